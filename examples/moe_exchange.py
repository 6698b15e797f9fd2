#!/usr/bin/env python3
"""One mixture-of-experts step with compressed exchanges, one GPU standing in for all ranks.

    python examples/moe_exchange.py [--tokens N] [--hidden H] [--inner F] [--experts E] [--ranks R]

The router's choices are sorted by expert; the rows of each rank's experts are compressed
straight from the token matrix by the sorted row lists and decoded as the receiving ranks
would; the experts (two products in 8 bits with a SiLU between) run on the received rows;
their outputs are compressed, sent back and decoded; each token sums its experts' outputs
with its weights.  Then the gradients of the combine and of the dispatch.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import torch  # noqa: E402

from lossless_bf16_exponent_codec_amd import moe  # noqa: E402
from lossless_bf16_exponent_codec_amd import zipccl as Z  # noqa: E402


def send(segments, cuts, length, status):
    """Compresses one segment per rank (by row lists, or whole rows) and decodes them into
    one buffer, as the receiving ranks would: (rows, compressed bytes)."""
    rows = cuts[-1][1]
    static = torch.empty(sum(Z.static_size((b - a) * length) for a, b in cuts), dtype=torch.uint8, device="cuda")
    esc = torch.empty(max(rows * length, 1), dtype=torch.uint8, device="cuda")
    space = torch.empty(Z.workspace_size(rows * length, len(cuts)), dtype=torch.uint8, device="cuda")
    n_esc = torch.zeros(len(cuts) + 1, dtype=torch.int64, device="cuda")
    if len(segments[0]) == 3:
        Z.compress_gather(segments, static, esc, space, n_esc, status)
    else:
        Z.compress(segments, static, esc, space, n_esc, status)
    got = torch.empty(rows, length, dtype=torch.bfloat16, device="cuda")
    Z.decompress(static, esc, [got[a:b] for a, b in cuts], status)
    return got, static.numel() + int(n_esc[-1])


def step(tokens=4096, hidden=1024, inner=512, experts=16, top_k=2, ranks=8, seed=0):
    """Returns the step's tensors by name."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").mul_(0.5).bfloat16()
    w1 = moe.QuantizedExperts(torch.randn(experts, inner, hidden, generator=g, device="cuda").mul_(hidden ** -0.5).bfloat16())
    w2 = moe.QuantizedExperts(torch.randn(experts, hidden, inner, generator=g, device="cuda").mul_(inner ** -0.5).bfloat16())
    top = torch.randn(tokens, experts, generator=g, device="cuda").topk(top_k)
    weights = torch.softmax(top.values, dim=1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    # there: rows by expert, one segment per rank
    routing = moe.route(top.indices, experts, status)
    ends = routing.splits()
    cuts = [(ends[r * experts // ranks], ends[(r + 1) * experts // ranks]) for r in range(ranks)]
    plan = Z.plan(sigma=0.5)
    sent, there = send([(x, routing.rows[a:b], plan) for a, b in cuts], cuts, hidden, status)

    # the experts' two products
    inside = torch.nn.functional.silu(w1(moe.quantize(sent), routing, status=status))
    made = w2(moe.quantize(inside), routing, status=status)

    # and back: each rank's rows as they lie
    scale = float(made.float().std())
    back, home = send([(made[a:b].reshape(-1), Z.plan(sigma=scale)) for a, b in cuts], cuts, hidden, status)
    out = moe.combine(back, routing, weights, status)

    # gradients: of the combine (rows and weights), and of the dispatch
    y, w, xg = back.detach().requires_grad_(), weights.detach().requires_grad_(), x.detach().requires_grad_()
    dout = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    dy, dw = torch.autograd.grad(moe.combine(y, routing, w, status), (y, w), dout)
    dx, = torch.autograd.grad(moe.dispatch(xg, routing, ends[-1], status), xg, dy)
    return dict(x=x, w1=w1, w2=w2, weights=weights, routing=routing, ends=ends, sent=sent, made=made, back=back,
                out=out, dout=dout, dy=dy, dw=dw, dx=dx, status=int(status.item()),
                ratio=2 * 2 * ends[-1] * hidden / (there + home))


def main():
    ap = argparse.ArgumentParser()
    for name, value in dict(tokens=4096, hidden=1024, inner=512, experts=16, top_k=2, ranks=8).items():
        ap.add_argument("--" + name.replace("_", "-"), type=int, default=value)
    args = ap.parse_args()
    s = step(**vars(args))
    same = bool(torch.equal(s["sent"].view(torch.int16), s["x"][s["routing"].rows[:s["ends"][-1]].long()].view(torch.int16)))
    print(f"{args.tokens} tokens x {args.top_k} of {args.experts} experts on {args.ranks} ranks: {s['ends'][-1]} rows each "
          f"way, {s['ratio']:.3f} times smaller, received rows {'equal' if same else 'DIFFERENT'}; "
          f"|out| {float(s['out'].float().abs().mean()):.4f}, |dx| {float(s['dx'].float().abs().mean()):.4f}, status {s['status']}")
    return 0 if same and s["status"] == 0 else 1


if __name__ == "__main__":
    sys.exit(main())
