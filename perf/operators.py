"""The measured cases of the mixture-of-experts operators: the router's choices sorted by
expert, tokens dispatched to their experts' rows and combined back with weights (each with
its gradient), and the experts' product in 8-bit integers.

`run` computes an operator either in its plain form (elementary torch operations in 32
bits, one rounding at the end) or, with `own` true, through the package's calls.
"""
import math

import torch

own = False

#: The router's skew: expert popularity follows k**-SKEW, the skew of the repository's MoE dispatch workload.
SKEW = 1.2
#: The widest listed case of each kind; a drawn case costs no more than this.
MOST_ASSIGNED = 16384 * 8
MOST_MOVED = 16384 * 8 * 7168
MOST_PRODUCT = 16384 * 7168 * 4096
MOST_WEIGHTS = 64 * 2048 * 7168


def listed():
    return [
        # One decode step of a batch of 64 sequences: the choices of 64 tokens, latency only.
        dict(name="sort_decode", op="sort", tokens=64, top_k=8, experts=256, drop=False),
        # A training batch of the repository's dispatch size, the choices past the experts' capacity dropped.
        dict(name="sort_batch", op="sort", tokens=16384, top_k=8, experts=256, drop=True),
        # The repository's dispatch matrix (16384 x 7168), every token sent to 8 experts: the forward pass
        # of training and of a long prompt.
        dict(name="dispatch_16384x7168", op="dispatch", tokens=16384, top_k=8, experts=64, row_len=7168,
             dtype="bf16", drop=False, backward=False),
        # The gradient of a dispatch with dropped choices (a few tokens have no row at all).
        dict(name="dispatch_backward_4096x2048", op="dispatch", tokens=4096, top_k=4, experts=32, row_len=2048,
             dtype="bf16", drop=True, backward=True),
        # Odd sizes in fp32: rows that start at any 4-byte address.
        dict(name="dispatch_fp32_odd", op="dispatch", tokens=1023, top_k=3, experts=7, row_len=1037, dtype="fp32",
             drop=False, backward=False),
        # The end of a decode step of 16 sequences: latency only.
        dict(name="combine_decode", op="combine", tokens=16, top_k=8, experts=64, row_len=7168, dtype="bf16",
             drop=False, backward=False),
        # The way back of the large dispatch.
        dict(name="combine_16384x7168", op="combine", tokens=16384, top_k=8, experts=64, row_len=7168,
             dtype="bf16", drop=False, backward=False),
        # The gradient of a combine in training: the experts' rows and the router's weights.
        dict(name="combine_backward_8192x4096", op="combine", tokens=8192, top_k=4, experts=16, row_len=4096,
             dtype="bf16", drop=False, backward=True),
        # Decode of one sequence: eight experts' weights are read for a row each.
        dict(name="product_one_token", op="product", tokens=1, top_k=8, experts=32, row_len=2048, outputs=1024,
             dtype="bf16", drop=False),
        # Decode of a batch: few rows for each expert, bound by the weights.
        dict(name="product_decode", op="product", tokens=64, top_k=4, experts=32, row_len=7168, outputs=2048,
             dtype="bf16", drop=False),
        # Odd sizes and uneven experts, fp32 out.
        dict(name="product_ragged", op="product", tokens=1501, top_k=2, experts=5, row_len=1000, outputs=1111,
             dtype="fp32", drop=True),
        # The repository's dispatch (16384 x 7168 to 8 skewed experts) multiplied by each expert's weights.
        dict(name="product_16384x7168", op="product", tokens=16384, top_k=1, experts=8, row_len=7168, outputs=4096,
             dtype="bf16", drop=False),
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], even over the logarithm; one in three is made odd."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    v = min(high, max(low, v))
    return v | 1 if rng.random() < 1 / 3 and v | 1 <= high else v


def draw(rng):
    op = rng.choice(["sort", "dispatch", "combine", "product"])
    while True:
        case = dict(op=op, tokens=_spread(rng, 1, 65536), top_k=rng.randint(1, 8), experts=_spread(rng, 4, 256),
                    drop=rng.random() < 0.3)
        if op == "sort":
            case["top_k"] = min(case["top_k"], case["experts"])
            if case["tokens"] * case["top_k"] <= MOST_ASSIGNED:
                return case
            continue
        case["row_len"] = _spread(rng, 64, 7168)
        case["dtype"] = rng.choice(["bf16", "bf16", "fp32"])
        if op == "product":
            case["experts"] = _spread(rng, 1, 64)
            case["outputs"] = _spread(rng, 64, 4096)
            rows = case["tokens"] * min(case["top_k"], case["experts"])
            fits = (rows * case["row_len"] * case["outputs"] <= MOST_PRODUCT and
                    case["experts"] * case["row_len"] * case["outputs"] <= MOST_WEIGHTS)
        else:
            case["backward"] = rng.random() < 0.5
            # the gradients move up to twice what the forward passes move, fp32 twice what bf16 does
            per = (2 if case["dtype"] == "fp32" else 1) * (2 if case["backward"] else 1)
            fits = per * case["tokens"] * case["top_k"] * case["row_len"] <= MOST_MOVED
        case["top_k"] = min(case["top_k"], case["experts"])
        if fits:
            return case


def _type(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _dropped(case):
    """Choices that find no place: none, or a fifth."""
    return case["tokens"] * case["top_k"] // 5 if case["drop"] else 0


def _sorted_by_expert(ids, experts):
    """offsets, rows and slots of the choices ids (negative: dropped), in torch operations."""
    flat = torch.where(ids < 0, experts, ids).reshape(-1)
    order = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(order.values, torch.arange(experts + 1, device=ids.device)).to(torch.int32)
    place = torch.empty_like(order.indices)
    place[order.indices] = torch.arange(flat.numel(), device=ids.device)
    rows = torch.where(order.values < experts, order.indices // ids.shape[1], -1).to(torch.int32)
    slots = torch.where(flat < experts, place, -1).to(torch.int32).reshape(ids.shape)
    return offsets, rows, slots


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, K, E, op = case["tokens"], case["top_k"], case["experts"], case["op"]
    # a router's choices: the K largest of skewed logits with Gumbel noise, softmax weights over them
    uniform = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    logits = -SKEW * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32)) - torch.log(-torch.log(uniform))
    top = torch.topk(logits, K, dim=1)
    ids = top.indices.clone()
    lost = torch.randperm(T * K, generator=g, device="cuda")[:_dropped(case)]
    ids.view(-1)[lost] = -1
    state = dict(case, ids=ids)
    if op == "sort":
        state["workspace"] = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        state["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        state["rows"] = torch.empty(T * K, dtype=torch.int32, device="cuda")
        state["slots"] = torch.empty(T, K, dtype=torch.int32, device="cuda")
        return state
    offsets, rows, slots = _sorted_by_expert(ids, E)
    # the program has copied the offsets to the host (all-to-all splits, sizes of its buffers)
    ends = offsets.tolist()
    H, M, dtype = case["row_len"], ends[-1], _type(case)
    state.update(offsets=offsets, rows=rows, slots=slots, ends=ends)

    def gaussian(n, length, scale=1.0):
        return torch.randn(n, length, generator=g, device="cuda").mul_(scale).to(dtype)

    if op == "dispatch":
        n_in, n_out = (M, T) if case["backward"] else (T, M)
        state["x"] = gaussian(n_in, H)
        state["out"] = torch.empty(n_out, H, dtype=dtype, device="cuda")
    elif op == "combine":
        state["weights"] = torch.softmax(top.values, dim=1)
        state["y"] = gaussian(M, H)
        if case["backward"]:
            state["grad"] = gaussian(T, H, 1e-2)
            state["grad_y"] = torch.empty(M, H, dtype=dtype, device="cuda")
            state["grad_weights"] = torch.empty(T, K, dtype=torch.float32, device="cuda")
        else:
            state["out"] = torch.empty(T, H, dtype=dtype, device="cuda")
    else:
        N, wide = case["outputs"], -(-H // 128) * 128
        # activations: a scale for each token, a few large channels, a few empty tokens; bf16 in any case
        x = torch.randn(T, H, generator=g, device="cuda")
        x *= torch.exp(torch.randn(T, 1, generator=g, device="cuda"))
        x[:, torch.randint(0, H, (max(1, H // 256),), generator=g, device="cuda")] *= 20.0
        x[torch.rand(T, generator=g, device="cuda") < 0.01] = 0.0
        state["x"] = x.to(torch.bfloat16)
        # 8-bit weights with a scale for each channel, laid out once: rows padded with zeros to 128 bytes
        w = torch.zeros(E, N, wide, dtype=torch.int8, device="cuda")
        for e in range(E):
            w[e, :, :H] = torch.randn(N, H, generator=g, device="cuda").mul_(32.0).round_().clamp_(-127, 127).to(torch.int8)
        state["weights"] = w
        state["weight_scales"] = torch.rand(E, N, generator=g, device="cuda").add_(0.5).mul_(H ** -0.5 / 32)
        state["q"] = torch.empty(M, wide, dtype=torch.int8, device="cuda")
        state["scales"] = torch.empty(M, dtype=torch.float32, device="cuda")
        state["out"] = torch.empty(M, N, dtype=dtype, device="cuda")
    return state


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from lossless_bf16_exponent_codec_amd import zipccl as Z

    op = s["op"]
    if op == "sort":
        Z.moe_sort(s["ids"], s["experts"], s["offsets"], s["rows"], s["slots"], s["workspace"])
        return s["offsets"], s["rows"], s["slots"]
    if op == "dispatch":
        if s["backward"]:
            Z.moe_dispatch_backward(s["x"], s["slots"], s["out"])
        else:
            Z.moe_dispatch(s["x"], s["slots"], s["out"])
        return s["out"]
    if op == "combine":
        if s["backward"]:
            Z.moe_combine_backward(s["grad"], s["y"], s["slots"], s["weights"], s["grad_y"], s["grad_weights"])
            return s["grad_y"], s["grad_weights"]
        Z.moe_combine(s["y"], s["slots"], s["weights"], s["out"])
        return s["out"]
    Z.quantize_rows(s["x"], s["q"], s["scales"], slots=s["slots"])
    Z.experts_product(s["q"], s["scales"], s["weights"], s["weight_scales"], s["row_len"], s["out"],
                      offsets=s["offsets"])
    return s["out"]


def _picked(rows, slots):
    """rows[slots] in 32 bits, [T, K, H], zeros where the slot is negative."""
    if rows.shape[0] == 0:
        return torch.zeros(*slots.shape, rows.shape[1], device=rows.device)
    return torch.where((slots >= 0).unsqueeze(-1), rows[slots.clamp(min=0)].float(), 0.0)


def _run_plain(s):
    op = s["op"]
    if op == "sort":
        return _sorted_by_expert(s["ids"], s["experts"])
    # token of each row, in sorted order
    tokens = s["rows"][:s["ends"][-1]]
    if op == "dispatch":
        if s["backward"]:
            return _picked(s["x"], s["slots"]).sum(1).to(s["x"].dtype)
        return s["x"][tokens]
    if op == "combine":
        if s["backward"]:
            grad = s["grad"].float()
            at = s["slots"].reshape(-1)
            spread = (s["weights"].unsqueeze(-1) * grad.unsqueeze(1)).reshape(at.numel(), -1)
            grad_y = torch.empty_like(s["y"])
            grad_y[at[at >= 0]] = spread[at >= 0].to(grad_y.dtype)
            return grad_y, (_picked(s["y"], s["slots"]) * grad.unsqueeze(1)).sum(-1)
        return (s["weights"].unsqueeze(-1) * _picked(s["y"], s["slots"])).sum(1).to(s["y"].dtype)
    x = s["x"].float()
    most = x.abs().amax(1, keepdim=True)
    q = torch.where(most > 0, torch.round(x * 127.0 / most), 0.0)[tokens]
    scale = (most / 127.0)[tokens]
    out = torch.empty_like(s["out"])
    ends = s["ends"]
    for e in range(s["experts"]):  # the experts with rows, one product each
        a, b = ends[e], ends[e + 1]
        if a < b:
            w = s["weights"][e, :, :s["row_len"]].float()
            out[a:b] = torch.matmul(q[a:b], w.t()) * scale[a:b] * s["weight_scales"][e]
    return out


def work(case):
    T, K, E, op = case["tokens"], case["top_k"], case["experts"], case["op"]
    rows = T * K - _dropped(case)
    if op == "sort":
        return dict(bytes=16 * T * K + 4 * (E + 1), flops=0)
    H, b = case["row_len"], 4 if case["dtype"] == "fp32" else 2
    if op == "dispatch":
        return dict(bytes=(T + rows) * H * b + 4 * T * K, flops=rows * H if case["backward"] else 0)
    if op == "combine":
        if case["backward"]:
            return dict(bytes=(T + 2 * rows) * H * b + 12 * T * K, flops=3 * rows * H)
        return dict(bytes=(T + rows) * H * b + 8 * T * K, flops=2 * rows * H)
    N = case["outputs"]
    # experts with rows, expected from their popularity
    mass = [k ** -SKEW for k in range(1, E + 1)]
    touched = sum(1 - (1 - min(1.0, K * m / sum(mass))) ** T for m in mass)
    return dict(bytes=T * H * 2 + touched * (N * H + 4 * N) + rows * N * b + 4 * T * K, flops=2 * rows * N * H)


def exact(case, seed):
    """The outputs in 64 bits, from the definitions: each row of the sorted order belongs to one assignment."""
    s = prepare(case, seed)
    op, K = case["op"], case["top_k"]
    if op == "sort":
        # whole numbers: counted on the host, choice by choice
        ids = s["ids"].reshape(-1).cpu()
        counts = torch.bincount(ids[ids >= 0], minlength=s["experts"])
        offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
        rows = torch.full((ids.numel(),), -1, dtype=torch.int64)
        slots = torch.full((ids.numel(),), -1, dtype=torch.int64)
        nxt, token_of, slot_of = offsets.tolist(), rows.numpy(), slots.numpy()
        for i, e in enumerate(ids.tolist()):
            if e >= 0:
                token_of[nxt[e]], slot_of[i] = i // K, nxt[e]
                nxt[e] += 1
        return offsets.int(), rows.int(), slots.int().reshape(s["ids"].shape)
    M = s["ends"][-1]
    # the assignment (token * K + choice) of each row, from the slots alone
    which = torch.empty(M, dtype=torch.int64, device="cuda")
    held = torch.nonzero(s["slots"].reshape(-1) >= 0).squeeze(1)
    which[s["slots"].reshape(-1)[held].long()] = held
    if op == "dispatch":
        if case["backward"]:
            out = torch.zeros(case["tokens"], case["row_len"], dtype=torch.float64, device="cuda")
            return out.index_add_(0, which // K, s["x"].double())
        return s["x"].double()[which // K]
    if op == "combine":
        w = s["weights"].double().reshape(-1)[which].unsqueeze(1)
        if case["backward"]:
            grad = s["grad"].double()[which // K]
            dot = torch.zeros(case["tokens"] * K, dtype=torch.float64, device="cuda")
            dot[which] = (grad * s["y"].double()).sum(1)
            return grad.mul_(w), dot.reshape(s["weights"].shape)
        out = torch.zeros(case["tokens"], case["row_len"], dtype=torch.float64, device="cuda")
        return out.index_add_(0, which // K, s["y"].double().mul_(w))
    x = s["x"].double()
    peak = x.abs().max(dim=1).values
    safe = torch.where(peak == 0, 1.0, peak)
    q = torch.round(127 * x / safe.unsqueeze(1))
    out = torch.empty(M, case["outputs"], dtype=torch.float64, device="cuda")
    for e in range(s["experts"]):
        part = which[s["ends"][e]:s["ends"][e + 1]] // K
        if part.numel():
            sums = q[part] @ s["weights"][e, :, :case["row_len"]].double().t()
            out[s["ends"][e]:s["ends"][e + 1]] = sums * (peak[part] / 127).unsqueeze(1) * s["weight_scales"][e].double()
    return out
