"""The measured cases of a mixture-of-experts layer's router and of its experts in 4 bits: a
router's choices and weights from its logits, the balance loss with the experts' counts (each
with its gradient), and the experts' product with 4-bit weights and group scales.

`run` computes an operator either in its plain form (elementary torch operations in 32
bits, one rounding at the end) or, with `own` true, through the package's calls.
"""
import math

import torch

own = False

#: The router's skew: expert popularity follows k**-SKEW, the skew of the repository's MoE dispatch workload.
SKEW = 1.2
#: The widest listed case of each kind; a drawn case costs no more than this.
MOST_LOGITS = 16384 * 256
MOST_PRODUCT = 8192 * 7168 * 4096
MOST_WEIGHTS = 32 * 2048 * 7168


def listed():
    return [
        # One decode step of a batch of 64 sequences: choices and weights only, latency.
        dict(name="gate_decode", op="gate", tokens=64, experts=256, top_k=8, dtype="bf16", renormalize=True,
             balance=False, masked=False, backward=False),
        # A training batch of the repository's dispatch size, with counts and loss, some tokens padding and some
        # experts closed.
        dict(name="gate_batch", op="gate", tokens=16384, experts=256, top_k=8, dtype="fp32", renormalize=True,
             balance=True, masked=True, backward=False),
        # Its gradient: of the weights and of the loss, into the logits.
        dict(name="gate_batch_backward", op="gate", tokens=16384, experts=256, top_k=8, dtype="fp32",
             renormalize=True, balance=True, masked=True, backward=True),
        # Odd sizes in bf16 (many equal logits), probabilities as weights.
        dict(name="gate_odd", op="gate", tokens=8191, experts=61, top_k=3, dtype="bf16", renormalize=False,
             balance=True, masked=True, backward=False),
        # The gradient of probabilities as weights, without a loss, of a small batch.
        dict(name="gate_raw_backward", op="gate", tokens=1023, experts=32, top_k=2, dtype="bf16", renormalize=False,
             balance=False, masked=False, backward=True),
        # Choices that the program made itself: counts, loss and gradient of a long batch over 64 experts.
        dict(name="balance_batch", op="balance", tokens=65536, experts=64, top_k=4, dtype="bf16", masked=True),
        # The same for one short sequence.
        dict(name="balance_short", op="balance", tokens=500, experts=16, top_k=2, dtype="fp32", masked=False),
        # Decode of one sequence: eight experts' weights are read for a row each.
        dict(name="product4_one_token", op="product4", tokens=1, top_k=8, experts=32, row_len=2048, outputs=1024,
             group=128, scales="bf16", dtype="bf16", drop=False),
        # Decode of a batch of 64: few rows for each expert, bound by the weights.
        dict(name="product4_decode", op="product4", tokens=64, top_k=4, experts=32, row_len=7168, outputs=2048,
             group=128, scales="bf16", dtype="bf16", drop=False),
        # Small groups with scales in fp32, a batch of 256, outputs that end inside a tile.
        dict(name="product4_groups_of_32", op="product4", tokens=256, top_k=2, experts=16, row_len=4096, outputs=1400,
             group=32, scales="fp32", dtype="bf16", drop=False),
        # Odd sizes and uneven experts, fp32 out.
        dict(name="product4_ragged", op="product4", tokens=1501, top_k=2, experts=5, row_len=1000, outputs=1111,
             group=64, scales="bf16", dtype="fp32", drop=True),
        # A prompt of 4096 tokens through the experts that decode uses: bound by the products.
        dict(name="product4_prompt", op="product4", tokens=4096, top_k=2, experts=8, row_len=7168, outputs=4096,
             group=128, scales="bf16", dtype="bf16", drop=False),
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], even over the logarithm; one in three is made odd."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    v = min(high, max(low, v))
    return v | 1 if rng.random() < 1 / 3 and v | 1 <= high else v


def draw(rng):
    op = rng.choice(["gate", "gate", "balance", "product4", "product4"])
    while True:
        if op == "product4":
            case = dict(op=op, tokens=_spread(rng, 1, 8192), top_k=rng.randint(1, 8), experts=_spread(rng, 1, 64),
                        row_len=_spread(rng, 64, 7168), outputs=_spread(rng, 64, 4096), group=rng.choice([32, 64, 128]),
                        scales=rng.choice(["bf16", "fp32"]), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                        drop=rng.random() < 0.3)
            case["top_k"] = min(case["top_k"], case["experts"])
            if (case["tokens"] * case["top_k"] * case["row_len"] * case["outputs"] <= MOST_PRODUCT and
                    case["experts"] * case["row_len"] * case["outputs"] <= MOST_WEIGHTS):
                return case
            continue
        case = dict(op=op, tokens=_spread(rng, 1, 65536), experts=_spread(rng, 4, 512), top_k=rng.randint(1, 8),
                    dtype=rng.choice(["bf16", "fp32"]), masked=rng.random() < 0.5)
        case["top_k"] = min(case["top_k"], case["experts"])
        if op == "gate":
            case.update(renormalize=rng.random() < 0.5, balance=rng.random() < 0.6, backward=rng.random() < 0.5)
        if case["tokens"] * case["experts"] <= MOST_LOGITS:
            return case


def _type(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _dropped(case):
    """Choices that find no place: none, or a fifth."""
    return case["tokens"] * case["top_k"] // 5 if case["drop"] else 0


def _router_logits(T, E, g):
    """Skewed logits with Gumbel noise: softmax over them spreads as the experts' popularity."""
    uniform = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    popular = -SKEW * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    return popular - torch.log(-torch.log(uniform))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, K, E = case["tokens"], case["top_k"], case["experts"]
    state = dict(case)
    if case["op"] == "product4":
        return _prepare_product(state, g)
    logits = _router_logits(T, E, g).to(_type(case["dtype"]))
    state["mask"] = None
    if case["masked"]:
        # closed experts, tokens that may go nowhere, and padding, which may hold anything
        closed = torch.rand(T, E, generator=g, device="cuda") < 0.05
        closed |= torch.rand(T, 1, generator=g, device="cuda") < 0.005
        logits.masked_fill_(closed, float("-inf"))
        state["mask"] = torch.rand(T, generator=g, device="cuda") >= 0.1
        logits.masked_fill_(~state["mask"].unsqueeze(1), float("nan"))
    state["logits"] = logits
    # choices that the forward pass has made (or the program itself): the largest K, the lowest index among equals
    live = logits.float()
    if case["masked"]:
        live = torch.where(state["mask"].unsqueeze(1), live, float("-inf"))
    if case["op"] == "balance" or case["backward"]:
        top = torch.sort(live, dim=1, descending=True, stable=True)
        state["experts_of"] = torch.where(top.values[:, :K] != float("-inf"), top.indices[:, :K], -1).to(torch.int32)
    else:
        state["experts_of"] = torch.empty(T, K, dtype=torch.int32, device="cuda")
        state["weights"] = torch.empty(T, K, dtype=torch.float32, device="cuda")
    if case["op"] == "balance" or case["balance"]:
        state["counts"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        state["sums"] = torch.empty(E, dtype=torch.float32, device="cuda")
        state["loss"] = torch.empty(1, dtype=torch.float32, device="cuda")
        state["workspace"] = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
        state["dloss"] = torch.rand(1, generator=g, device="cuda").add_(0.5).mul_(0.01 * T)
    if case["op"] == "balance" or case["backward"]:
        state["dlogits"] = torch.empty_like(logits)
    if case["op"] == "gate" and case["backward"]:
        state["dweights"] = torch.randn(T, K, generator=g, device="cuda")
        if case["balance"]:   # the forward pass has counted
            ids = state["experts_of"].reshape(-1).long()
            state["counts"][:E] = torch.bincount(torch.where(ids < 0, E, ids), minlength=E + 1)[:E]
            state["counts"][E] = (live != float("-inf")).any(1).sum()
    return state


def _prepare_product(state, g):
    T, K, E = state["tokens"], state["top_k"], state["experts"]
    H, N, G = state["row_len"], state["outputs"], state["group"]
    top = torch.topk(_router_logits(T, E, g), K, dim=1)
    ids = top.indices.clone()
    ids.view(-1)[torch.randperm(T * K, generator=g, device="cuda")[:_dropped(state)]] = -1
    # the choices sorted by expert; the program has the offsets on the host too
    flat = torch.where(ids < 0, E, ids).reshape(-1)
    order = torch.sort(flat, stable=True)
    state["offsets"] = torch.searchsorted(order.values, torch.arange(E + 1, device="cuda")).to(torch.int32)
    state["rows"] = torch.where(order.values < E, order.indices // K, -1).to(torch.int32)
    state["ends"] = state["offsets"].tolist()
    M = state["ends"][-1]
    # activations: a scale for each token, a few large channels, a few empty tokens
    x = torch.randn(T, H, generator=g, device="cuda")
    x *= torch.exp(torch.randn(T, 1, generator=g, device="cuda"))
    x[:, torch.randint(0, H, (max(1, H // 256),), generator=g, device="cuda")] *= 20.0
    x[torch.rand(T, generator=g, device="cuda") < 0.01] = 0.0
    state["x"] = x.to(torch.bfloat16)
    # weights from -8 to 7, laid out once: tiles of 16 outputs x 128 inputs, padded with zeros
    tiles, slabs = -(-N // 16), -(-H // 128)
    packed = torch.empty(E, tiles * slabs * 1024, dtype=torch.uint8, device="cuda")
    for e in range(E):
        w = torch.zeros(16 * tiles, 128 * slabs, device="cuda")
        w[:N, :H] = torch.randn(N, H, generator=g, device="cuda").mul_(2.6).round_().clamp_(-8, 7)
        packed[e] = _pack(w.to(torch.int32), tiles, slabs)
    state["weights"] = packed
    groups = -(-H // G)
    state["weight_scales"] = torch.rand(E, groups, N, generator=g, device="cuda").add_(0.5).mul_(H ** -0.5 / 2.6).to(_type(state["scales"]))
    state["out"] = torch.empty(M, N, dtype=_type(state["dtype"]), device="cuda")
    return state


def _pack(w, tiles, slabs):
    """A tile's 1024 bytes: output o and inputs 32 i + 8 q .. + 7 are dword i of lane 16 q + o, input j in bits 4 j."""
    w = (w & 15).view(tiles, 16, slabs, 4, 4, 4, 2)   # tile, output, slab, i, q, byte, half
    both = (w[..., 0] | w[..., 1] << 4).to(torch.uint8)
    return both.permute(0, 2, 4, 1, 3, 5).reshape(-1)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from lossless_bf16_exponent_codec_amd import zipccl as Z

    op = s["op"]
    if op == "product4":
        Z.experts_product4(s["x"], s["weights"], s["weight_scales"], s["group"], s["out"], rows=s["rows"],
                           offsets=s["offsets"])
        return s["out"]
    if op == "balance":
        Z.moe_balance(s["logits"], s["experts_of"], s["counts"], s["sums"], s["loss"], s["workspace"], mask=s["mask"])
        Z.moe_gate_backward(s["logits"], s["experts_of"], s["dlogits"], counts=s["counts"], dloss=s["dloss"],
                            mask=s["mask"])
        return s["counts"], s["sums"], s["loss"], s["dlogits"]
    if s["backward"]:
        Z.moe_gate_backward(s["logits"], s["experts_of"], s["dlogits"], dweights=s["dweights"],
                            counts=s.get("counts"), dloss=s.get("dloss"), renormalize=s["renormalize"], mask=s["mask"])
        return s["dlogits"]
    Z.moe_gate(s["logits"], s["experts_of"], s["weights"], renormalize=s["renormalize"], mask=s["mask"],
               counts=s.get("counts"), sums=s.get("sums"), loss=s.get("loss"), workspace=s.get("workspace"))
    if s["balance"]:
        return s["experts_of"], s["weights"], s["counts"], s["sums"], s["loss"]
    return s["experts_of"], s["weights"]


def _live(s):
    """Logits in 32 bits with nothing in padded rows, exp of them less their row's largest, its sum (1 in rows of
    nothing), and which rows have something."""
    logits = s["logits"].float()
    if s["mask"] is not None:
        logits = torch.where(s["mask"].unsqueeze(1), logits, float("-inf"))
    most = logits.amax(1, keepdim=True)
    some = most != float("-inf")
    e = torch.exp(logits - torch.where(some, most, 0.0))
    return logits, e, torch.where(some, e.sum(1, keepdim=True), 1.0), some


def _balance(s, p, some, ids):
    """Counts (with the number of tokens counted), sums of probabilities and the loss."""
    E, K = s["experts"], s["top_k"]
    at = torch.where(ids < 0, E, ids).reshape(-1).long()
    counts = torch.zeros(E + 1, dtype=torch.int64, device=p.device).scatter_add_(0, at, torch.ones_like(at))
    counts[E] = some.sum()
    sums = p.sum(0)
    n = counts[E].float()
    loss = E / K * (counts[:E].float() * sums).sum() / torch.where(n > 0, n * n, 1.0)
    return counts.to(torch.int32), sums, loss.reshape(1)


def _balance_gradient(s, p, counts):
    E, K = s["experts"], s["top_k"]
    n = counts[E].float()
    c = s["dloss"] * (E / K) * counts[:E].float() / torch.where(n > 0, n * n, 1.0)
    return p * (c - (p * c).sum(1, keepdim=True))


def _run_plain(s):
    if s["op"] == "product4":
        return _product_plain(s)
    K, ids = s["top_k"], s["experts_of"]
    logits, e, total, some = _live(s)
    p = e / total
    if s["op"] == "balance":
        counts, sums, loss = _balance(s, p, some, ids)
        return counts, sums, loss, _balance_gradient(s, p, counts).to(s["logits"].dtype)
    if s["backward"]:
        at = ids.clamp(min=0).long()
        chosen = torch.where(ids >= 0, torch.gather(e, 1, at), 0.0)
        if s["renormalize"]:
            w = chosen / torch.where(some, chosen.sum(1, keepdim=True), 1.0)
            dw = torch.where(ids >= 0, s["dweights"], 0.0)
            d = w * (dw - (w * dw).sum(1, keepdim=True))
            grad = torch.zeros_like(p).scatter_add_(1, at, d)
        else:
            dw = torch.where(ids >= 0, s["dweights"], 0.0)
            dot = (chosen / total * dw).sum(1, keepdim=True)
            grad = p * (torch.zeros_like(p).scatter_add_(1, at, dw) - dot)
        if s["balance"]:
            grad = grad + _balance_gradient(s, p, s["counts"])
        return grad.to(s["logits"].dtype)
    top = torch.sort(logits, dim=1, descending=True, stable=True)
    there = top.values[:, :K] != float("-inf")
    ids = torch.where(there, top.indices[:, :K], -1).to(torch.int32)
    chosen = torch.where(there, torch.gather(e, 1, top.indices[:, :K]), 0.0)
    weights = chosen / (torch.where(some, chosen.sum(1, keepdim=True), 1.0) if s["renormalize"] else total)
    if s["balance"]:
        return (ids, weights, *_balance(s, p, some, ids))
    return ids, weights


def _product_plain(s):
    H, N, G = s["row_len"], s["outputs"], s["group"]
    tiles, slabs = -(-N // 16), -(-H // 128)
    x, out, ends = s["x"].float(), torch.empty_like(s["out"]), s["ends"]
    for e in range(s["experts"]):  # the experts with rows, one product each
        a, b = ends[e], ends[e + 1]
        if a < b:
            both = s["weights"][e].view(tiles, slabs, 4, 16, 4, 4).permute(0, 3, 1, 4, 2, 5)
            w = torch.stack([both & 15, both >> 4], dim=-1).reshape(16 * tiles, 128 * slabs)[:N, :H]
            w = ((w ^ 8).float() - 8.0)
            scales = s["weight_scales"][e].float().t().repeat_interleave(G, dim=1)[:, :H]
            out[a:b] = torch.matmul(x[s["rows"][a:b]], (w * scales).t())
    return out


def work(case):
    T, K, E = case["tokens"], case["top_k"], case["experts"]
    b = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "product4":
        rows, H, N = T * K - _dropped(case), case["row_len"], case["outputs"]
        # experts with rows, expected from their popularity
        mass = [k ** -SKEW for k in range(1, E + 1)]
        touched = sum(1 - (1 - min(1.0, K * m / sum(mass))) ** T for m in mass)
        scales = -(-H // case["group"]) * N * (4 if case["scales"] == "fp32" else 2)
        return dict(bytes=T * H * 2 + touched * (N * H / 2 + scales) + rows * N * b + 4 * rows, flops=2 * rows * N * H)
    mask = T if case["masked"] else 0
    if case["op"] == "balance":
        return dict(bytes=2 * T * E * b + 4 * T * K + 12 * E + mask, flops=12 * T * E)
    if case["backward"]:
        return dict(bytes=2 * T * E * b + 8 * T * K + mask + (4 * E if case["balance"] else 0), flops=9 * T * E)
    return dict(bytes=T * E * b + 8 * T * K + mask + (8 * E if case["balance"] else 0), flops=4 * T * E)


def exact(case, seed):
    """The outputs in 64 bits, from the definitions."""
    s = prepare(case, seed)
    if case["op"] == "product4":
        return _product_exact(s)
    T, E, K = case["tokens"], case["experts"], case["top_k"]
    z = s["logits"].double()
    counted = torch.isfinite(z).any(1)   # padding holds NaN, closed experts minus infinity
    z = torch.where(counted.unsqueeze(1), z, 0.0)
    p = torch.softmax(z, dim=1) * counted.unsqueeze(1)
    if case["op"] == "gate" and not case["backward"]:
        # by descending logit, then by index: a stable sort of the negated logits
        index = torch.sort(-z, dim=1, stable=True).indices[:, :K]
        valid = counted.unsqueeze(1) & (torch.gather(z, 1, index) > float("-inf"))
        ids = torch.where(valid, index, -1)
    else:
        ids, valid = s["experts_of"].long(), s["experts_of"] >= 0
    chosen = torch.zeros(T, E + 1, dtype=torch.float64, device="cuda")   # one in the column of each choice
    chosen.scatter_(1, torch.where(valid, ids, E), 1.0)
    chosen = chosen[:, :E]
    picked = torch.where(valid, torch.gather(p, 1, ids.clamp(min=0)), 0.0)
    share = (p * chosen).sum(1, keepdim=True)
    share = torch.where(share > 0, share, 1.0)
    counts, n = chosen.sum(0), counted.sum().double()
    per = E / (K * n * n) if n > 0 else torch.zeros((), dtype=torch.float64, device="cuda")
    whole = torch.cat([counts, n.reshape(1)]).to(torch.int32)
    sums = p.sum(0)
    loss = (per * torch.dot(counts, sums)).reshape(1)
    grad = torch.zeros_like(p)
    if case["op"] == "balance" or case["balance"] and case["backward"]:
        f = s["dloss"].double() * per * counts
        grad += p * f - p * torch.mv(p, f).unsqueeze(1)
    if case["op"] == "balance":
        return whole, sums, loss, grad
    if case["backward"]:
        dw = torch.zeros(T, E + 1, dtype=torch.float64, device="cuda")
        dw.scatter_(1, torch.where(valid, ids, E), s["dweights"].double())
        dw = dw[:, :E]
        q = p * chosen / share if case["renormalize"] else p
        return grad + q * dw - q * (q * dw).sum(1, keepdim=True)
    weights = picked / share if case["renormalize"] else picked
    return (ids.int(), weights, whole, sums, loss) if case["balance"] else (ids.int(), weights)


def _product_exact(s):
    H, N, G = s["row_len"], s["outputs"], s["group"]
    slabs = -(-H // 128)
    n = torch.arange(N, device="cuda").unsqueeze(1)
    h = torch.arange(H, device="cuda").unsqueeze(0)
    # the byte of output n and input h
    at = (((n // 16 * slabs + h // 128) * 64 + h % 32 // 8 * 16 + n % 16) * 4 + h % 128 // 32) * 4 + h % 8 // 2
    out = torch.empty(s["ends"][-1], N, dtype=torch.float64, device="cuda")
    for e in range(s["experts"]):
        a, b = s["ends"][e], s["ends"][e + 1]
        if a < b:
            code = s["weights"][e][at].int() >> h % 2 * 4 & 15
            w = torch.where(code > 7, code - 16, code).double() * s["weight_scales"][e].double()[(h // G)[0]].t()
            out[a:b] = s["x"].double()[s["rows"][a:b].long()] @ w.t()
    return out
