"""Experts' weights in 4 bits on the GPU against plain 64-bit implementations.

Packing is compared for equality (a quotient of two fp32 numbers and its rounding have one
right value).  A product's fp32 sum over H inputs is off by at most H * 2^-23 of the sum of
the terms' magnitudes (products of a BF16 and a 4-bit number are exact, a group's scale
rounds once), then rounded once to its type (half a step).  Where x holds small whole
numbers and the scales powers of two every partial sum is exact in fp32: equality."""
import numpy as np
import pytest
import torch

from tests import router_reference as R

pytestmark = pytest.mark.gpu

POISON = 12345.0


@pytest.fixture(scope="module")
def Z():
    from lossless_bf16_exponent_codec_amd import zipccl
    return zipccl


@pytest.fixture(scope="module")
def moe():
    from lossless_bf16_exponent_codec_amd import moe
    return moe


def host(t):
    return t.double().cpu().numpy()


def round_to(dtype):
    def f(a):
        return torch.from_numpy(a).to(dtype).float().numpy() if dtype == torch.bfloat16 else a
    return f


# ------------------------------------------------------------------------------------
# packing
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("scale_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,N,H,group", [(1, 1, 1, 32), (2, 16, 128, 32), (3, 17, 129, 64), (2, 40, 300, 128),
                                         (1, 33, 1000, 64), (2, 20, 700, 256), (1, 18, 513, 512), (2, 5, 200, 1 << 30),
                                         (4, 64, 256, 32)])
def test_quantize(Z, E, N, H, group, scale_dtype):
    rng = np.random.default_rng(N + H)
    w = torch.from_numpy(rng.standard_normal((E, N, H)).astype(np.float32)).bfloat16()
    w[0, 0, : min(H, 32)] = 0                           # a group of zeros
    w[E - 1, N - 1, H - 1] = float("inf") if N % 2 else float("nan")
    w[0, N // 2] *= 1e-30
    if N > 2:
        w[0, 1] = w[0, 1] * 0 + 1e-40                   # scales that are subnormal
    groups = -(-H // group)
    q = torch.full((Z.weights4_size(E, N, H) + 64,), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((E, groups, N), POISON, dtype=scale_dtype, device="cuda")
    Z.quantize_weights4(w.cuda(), group, q, scales)
    assert bool((q[-64:] == 0xAA).all())
    values, clean = R.unpack4(q[:-64].cpu().numpy(), E, N, H)
    want, wscales = R.quantize4(w.float().numpy(), group, round_to(scale_dtype))
    assert clean and np.array_equal(host(scales), wscales, equal_nan=True)
    assert np.array_equal(values, want)


def test_quantize_strided_and_one_expert(Z):
    rng = np.random.default_rng(1)
    E, N, H = 3, 21, 150
    flat = torch.from_numpy(rng.standard_normal(E * N * 157 + 1).astype(np.float32)).bfloat16().cuda()
    w = flat[1:].view(E, N, 157)[:, :, :H]
    q = torch.empty(Z.weights4_size(E, N, H), dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, 3, N, dtype=torch.float32, device="cuda")
    Z.quantize_weights4(w, 64, q, scales)
    want, wscales = R.quantize4(w.float().cpu().numpy(), 64, round_to(torch.float32))
    values, clean = R.unpack4(q.cpu().numpy(), E, N, H)
    assert clean and np.array_equal(values, want) and np.array_equal(host(scales), wscales)
    q1, s1 = torch.empty(Z.weights4_size(1, N, H), dtype=torch.uint8, device="cuda"), torch.empty(1, 3, N, device="cuda")
    Z.quantize_weights4(w[2], 64, q1, s1)
    assert torch.equal(q1, q.view(E, -1)[2]) and torch.equal(s1[0], scales[2])


@pytest.mark.parametrize("E,N,H", [(1, 1, 1), (3, 17, 129), (2, 32, 256), (1, 50, 77)])
def test_pack4(moe, E, N, H):
    values = torch.from_numpy(np.random.default_rng(E + N).integers(-8, 8, (E, N, H)))
    for dtype in (torch.int8, torch.int32, torch.int64):
        q = moe.pack4(values.to(dtype).cuda())
        back, clean = R.unpack4(q.cpu().numpy(), E, N, H)
        assert clean and np.array_equal(back, values.numpy())


# ------------------------------------------------------------------------------------
# product
# ------------------------------------------------------------------------------------
def spread(rng, M, E, empty=0.3):
    """offsets of M rows over E experts, some of them empty."""
    mass = rng.random(E) * (rng.random(E) > empty) + 1e-9
    cuts = np.sort(rng.choice(E, M, p=mass / mass.sum()))
    return np.searchsorted(cuts, np.arange(E + 1)).astype(np.int32)


def make(rng, moe, T, M, E, N, H, group, scale_dtype, whole=False, stride=None, offset=0):
    stride = stride or H
    groups = -(-H // group)
    values = rng.integers(-8, 8, (E, N, H))
    if whole:
        flat = rng.integers(-4, 5, T * stride + offset).astype(np.float32)
        scales = 2.0 ** rng.integers(-2, 3, (E, groups, N))
    else:
        flat = rng.standard_normal(T * stride + offset).astype(np.float32)
        scales = rng.uniform(0.5, 1.5, (E, groups, N))
    x = torch.from_numpy(flat).bfloat16().cuda()[offset:].view(T, stride)[:, :H]
    s = torch.from_numpy(scales).to(scale_dtype).cuda()
    q = moe.pack4(torch.from_numpy(values).cuda())
    index = rng.integers(0, T, M).astype(np.int32)
    return x, torch.from_numpy(index).cuda(), q, s, values


def check(Z, x, index, q, s, values, group, offsets, dtype, whole=False, out=None):
    M, N, H = len(index), values.shape[1], values.shape[2]
    if out is None:
        out = torch.full((M, N), POISON, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Z.experts_product4(x, q, s, group, out, rows=index, offsets=torch.from_numpy(offsets).cuda(), status=status)
    want, size = R.product4(host(x), index.cpu().numpy(), values, host(s), group, offsets)
    got, inside = host(out), ~np.isnan(want).all(axis=1)
    assert np.all(got[~inside] == torch.tensor(POISON, dtype=dtype).item())
    assert int(status.item()) == 0
    want, size = want[inside], size[inside]
    if whole:
        assert np.array_equal(got[inside], torch.from_numpy(want).to(dtype).double().numpy())
    else:
        tol = (H * 2.0 ** -23) * size + torch.finfo(dtype).eps / 2 * (np.abs(want) + H * 2.0 ** -23 * size)
        assert np.all(np.abs(got[inside] - want) <= tol)


PRODUCTS = [(1, 1, 1, 1, 1, 32), (1, 8, 32, 64, 256, 128), (3, 5, 4, 16, 128, 64), (40, 33, 3, 17, 129, 32),
            (64, 100, 7, 50, 300, 128), (20, 16, 1, 70, 1000, 64), (90, 65, 2, 130, 384, 32), (200, 300, 5, 64, 640, 128),
            (30, 17, 1, 100, 2050, 128), (300, 900, 70, 20, 200, 64), (50, 130, 2, 65, 513, 256), (9, 40, 3, 33, 700, 512),
            (500, 1500, 4, 140, 260, 32), (16, 31, 2, 300, 4100, 128)]


@pytest.mark.parametrize("scale_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,M,E,N,H,group", PRODUCTS)
def test_product(Z, moe, T, M, E, N, H, group, dtype, scale_dtype):
    rng = np.random.default_rng(M + N + H)
    x, index, q, s, values = make(rng, moe, T, M, E, N, H, group, scale_dtype)
    offsets = spread(rng, M, E)
    check(Z, x, index, q, s, values, group, offsets, dtype)
    # sums that are exact: at most 32 * 8 * 4 * 4 * H below 2^24 in size
    x, index, q, s, values = make(rng, moe, T, M, E, N, H, group, scale_dtype, whole=True)
    check(Z, x, index, q, s, values, group, offsets, dtype, whole=True)


# enough rows for tiles of 64 (128 outputs wide, and 64), and enough outputs for workgroups of 32
# and 64 of them on few rows
MANY = [(300, 1200, 8, 1500, 130, 32), (700, 1100, 2, 2050, 257, 64), (90, 1200, 8, 1400, 640, 128),
        (300, 1200, 8, 2500, 300, 128), (64, 1100, 2, 3900, 515, 256), (200, 1300, 8, 2400, 128, 64),
        (1300, 1300, 1, 3200, 386, 32), (64, 640, 40, 160, 400, 64), (400, 1600, 4, 300, 260, 32),
        (1000, 1000, 100, 200, 700, 128)]


@pytest.mark.parametrize("scale_dtype,dtype", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("T,M,E,N,H,group", MANY)
def test_many_rows(Z, moe, T, M, E, N, H, group, dtype, scale_dtype):
    rng = np.random.default_rng(M + N + H)
    # rows that are loaded without registers, and rows at odd places
    for stride, offset in ((-(-H // 8) * 8, 0), (H + 1, 3)):
        x, index, q, s, values = make(rng, moe, T, M, E, N, H, group, scale_dtype, stride=stride, offset=offset)
        check(Z, x, index, q, s, values, group, spread(rng, M, E), dtype)
    x, index, q, s, values = make(rng, moe, T, M, E, N, H, group, scale_dtype, whole=True)
    check(Z, x, index, q, s, values, group, spread(rng, M, E, empty=0.0), dtype, whole=True)


@pytest.mark.parametrize("T,M,E,N,H,group", MANY[:8:3])
def test_many_rows_some_bad(Z, moe, T, M, E, N, H, group):
    # rows out of range, rows behind the last expert, NaN and infinity in a token
    rng = np.random.default_rng(N)
    x, index, q, s, values = make(rng, moe, T, M, E, N, H, group, torch.bfloat16, whole=True)
    index[3::50], index[4::70] = T, -1
    x[7, H - 1], x[8, 0] = float("nan"), float("inf")
    offsets = np.concatenate([[2], np.sort(rng.integers(2, M - 40, E - 1)), [M - 40]]).astype(np.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((M, N), POISON, device="cuda")
    Z.experts_product4(x, q, s, group, out, rows=index, offsets=torch.from_numpy(offsets).cuda(), status=status)
    assert int(status.item()) == Z.STATUS_BAD_INDEX
    want, _ = R.product4(host(x), index.cpu().numpy(), values, host(s), group, offsets)
    got, at = host(out), index.cpu().numpy()
    assert np.all(got[:2] == POISON) and np.all(got[M - 40:] == POISON)
    inside = slice(2, M - 40)
    assert not got[inside][(at[inside] < 0) | (at[inside] >= T)].any()
    assert np.array_equal(got[inside], want[inside], equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,stride,offset", [(64, 67, 1), (515, 520, 3), (128, 128, 7), (1000, 1001, 1)])
def test_strided_and_unaligned_rows(Z, moe, H, stride, offset, dtype):
    rng = np.random.default_rng(H)
    M, E, N = 45, 3, 37
    x, index, q, s, values = make(rng, moe, 30, M, E, N, H, 64, torch.bfloat16, whole=True, stride=stride, offset=offset)
    flat = torch.full((M * (N + 3) + offset,), POISON, dtype=dtype, device="cuda")
    out = flat[offset:].view(M, N + 3)[:, :N]
    check(Z, x, index, q, s, values, 64, spread(rng, M, E), dtype, whole=True, out=out)
    rest = flat[offset:].view(M, N + 3)[:, N:]
    assert bool((rest == rest.new_tensor(POISON)).all()) and bool((flat[:offset] == flat.new_tensor(POISON)).all())


def test_rows_past_the_last_expert_stay(Z, moe):
    rng = np.random.default_rng(2)
    M, E, N, H = 70, 4, 48, 200
    x, index, q, s, values = make(rng, moe, 20, M, E, N, H, 32, torch.float32, whole=True)
    check(Z, x, index, q, s, values, 32, np.array([3, 3, 20, 41, 60], np.int32), torch.float32, whole=True)
    check(Z, x, index, q, s, values, 32, np.zeros(5, np.int32), torch.bfloat16, whole=True)


def test_rows_as_they_lie_and_one_expert(Z, moe):
    rng = np.random.default_rng(3)
    M, N, H = 50, 40, 256
    x, _, q, s, values = make(rng, moe, M, M, 1, N, H, 128, torch.bfloat16, whole=True)
    out = torch.empty(M, N, dtype=torch.float32, device="cuda")
    Z.experts_product4(x, q, s, 128, out)
    want, _ = R.product4(host(x), np.arange(M), values, host(s), 128, [0, M])
    assert np.array_equal(host(out), want)


def test_bad_rows_and_offsets_are_reported(Z, moe):
    rng = np.random.default_rng(4)
    T, M, E, N, H = 12, 40, 3, 20, 130
    x, index, q, s, values = make(rng, moe, T, M, E, N, H, 64, torch.float32, whole=True)
    index[5], index[6] = T, -3
    offsets = np.array([0, 10, 25, 40], np.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((M, N), POISON, device="cuda")
    Z.experts_product4(x, q, s, 64, out, rows=index, offsets=torch.from_numpy(offsets).cuda(), status=status)
    assert int(status.item()) == Z.STATUS_BAD_INDEX
    want, _ = R.product4(host(x), index.cpu().numpy(), values, host(s), 64, offsets)
    assert np.array_equal(host(out), want) and not out[5:7].any()
    # offsets past the rows are clamped
    index[5], index[6] = 0, 0
    for bad in ([0, 10, 25, 41], [-2, 10, 25, 40], [0, 25, 10, 40]):
        status.zero_()
        Z.experts_product4(x, q, s, 64, out, rows=index, offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"),
                           status=status)
        assert int(status.item()) == Z.STATUS_BAD_INDEX


def test_nans_and_infinities_stay_in_their_rows(Z, moe):
    rng = np.random.default_rng(5)
    T, M, E, N, H = 40, 40, 2, 33, 300
    x, _, q, s, values = make(rng, moe, T, M, E, N, H, 32, torch.bfloat16)
    x[7, 3], x[20, 299] = float("nan"), float("inf")
    s[1, 2, 5] = float("nan")
    offsets = torch.tensor([0, 25, 40], dtype=torch.int32, device="cuda")
    rows = torch.arange(M, dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.empty(M, N, dtype=dtype, device="cuda")
        Z.experts_product4(x, q, s, 32, out, rows=rows, offsets=offsets)
        nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
        nan[7], nan[25:, 5] = True, True
        w20 = torch.from_numpy(values[0, :, 299]).cuda()
        nan[20] |= w20 == 0                             # infinity times nothing
        assert torch.equal(out.isnan(), nan)
        assert bool((out[20][w20 != 0].float() == torch.sign(w20[w20 != 0]).float() * float("inf")).all())
        if dtype == torch.bfloat16:
            assert bool((out.view(torch.int16)[nan] == 0x7FC0).all())


def test_no_rows(Z, moe):
    q, s = moe.pack4(torch.zeros(2, 16, 128, dtype=torch.int8, device="cuda")), torch.ones(2, 1, 16, device="cuda")
    out = torch.empty(0, 16, device="cuda")
    Z.experts_product4(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), q, s, 128, out,
                       rows=torch.empty(0, dtype=torch.int32, device="cuda"),
                       offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))


def test_captured_and_replayed(Z, moe):
    rng = np.random.default_rng(6)
    T, M, E, N, H = 16, 32, 4, 80, 512
    x, index, q, s, values = make(rng, moe, T, M, E, N, H, 128, torch.bfloat16)
    offsets = torch.from_numpy(spread(rng, M, E)).cuda()
    out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    Z.experts_product4(x, q, s, 128, out, rows=index, offsets=offsets)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z.experts_product4(x, q, s, 128, out, rows=index, offsets=offsets)
    for _ in range(4):
        x.copy_(torch.randn(T, H, device="cuda"))
        offsets.copy_(torch.from_numpy(spread(rng, M, E)))
        graph.replay()
        torch.cuda.synchronize()
        eager = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        Z.experts_product4(x, q, s, 128, eager, rows=index, offsets=offsets)
        torch.cuda.synchronize()
        lo, hi = int(offsets[0]), int(offsets[-1])
        assert torch.equal(out[lo:hi], eager[lo:hi])


# ------------------------------------------------------------------------------------
# the torch layer, and the operators together as a layer uses them
# ------------------------------------------------------------------------------------
def test_experts_of_existing_values(moe):
    g = torch.Generator(device="cuda").manual_seed(1)
    T, K, E, N, H = 30, 2, 5, 50, 200
    values = torch.randint(-8, 8, (E, N, H), generator=g, device="cuda", dtype=torch.int8)
    scales = torch.rand(E, N, 4, generator=g, device="cuda") + 0.5
    experts = moe.QuantizedExperts4.of(values, scales, 64)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    routing = moe.route(torch.rand(T, E, generator=g, device="cuda").topk(K).indices, E)
    got = experts(x, routing, dtype=torch.float32)
    ends = routing.splits()
    assert got.shape[0] == T * K
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        w = values[e].double() * scales[e].double().repeat_interleave(64, dim=1)[:, :H]
        rows = x[routing.rows[a:b].long()].double()
        want, size = rows @ w.T, rows.abs() @ w.abs().T
        assert bool(((got[a:b].double() - want).abs() <= H * 2.0 ** -23 * size).all())


@pytest.mark.parametrize("renormalize", [True, False])
def test_layer_in_training(moe, renormalize):
    # gate, balance loss, dispatch, dense experts, combine: gradients of the logits and of x
    # against autograd in 64 bits.  Values of size 1 or less and sums of at most 200 terms:
    # 400 * 2^-23 of the largest value, doubled for the library's products
    g = torch.Generator(device="cuda").manual_seed(2)
    T, K, E, H = 60, 2, 6, 24
    x, f = torch.randn(T, H, generator=g, device="cuda"), torch.randn(E, H, H, generator=g, device="cuda") * 0.2
    z, dout = torch.randn(T, E, generator=g, device="cuda"), torch.randn(T, H, generator=g, device="cuda")
    mask = torch.rand(T, generator=g, device="cuda") < 0.9
    z[4, :5] = float("-inf")
    leaves = [x.clone().requires_grad_(), z.clone().requires_grad_()]
    router = moe.gate(leaves[1], K, renormalize, mask, balance=True)
    routing = moe.route(router.experts, E)
    ends = routing.splits()
    y = moe.dispatch(leaves[0], routing, ends[-1])
    y = torch.cat([y[ends[e]:ends[e + 1]] @ f[e] for e in range(E)])
    out = moe.combine(y, routing, router.weights)
    got = torch.autograd.grad((out * dout).sum() + 0.3 * router.loss, leaves)

    wide = [x.double().cpu().requires_grad_(), z.double().cpu().requires_grad_()]
    m, fd = mask.cpu(), f.double().cpu()
    p = torch.softmax(wide[1], 1)
    ids = torch.sort(z.cpu(), dim=1, descending=True, stable=True).indices[:, :K]
    ok = m.unsqueeze(1) & (torch.gather(z.cpu(), 1, ids) > float("-inf"))
    assert torch.equal(router.experts.cpu().long(), torch.where(ok, ids, -1))
    w = torch.where(ok, torch.gather(p, 1, ids), torch.zeros((), dtype=torch.float64))
    if renormalize:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    each = torch.einsum("th,ehk->tek", wide[0], fd)
    ref = (w.unsqueeze(-1) * torch.gather(each, 1, ids.unsqueeze(-1).expand(-1, -1, H))).sum(1)
    counts = torch.bincount(ids[ok], minlength=E).double()
    n = m.sum().double()
    loss = E / (K * n * n) * (counts * (p * m.unsqueeze(1)).sum(0)).sum()
    assert torch.equal(router.counts.cpu().double(), torch.cat([counts, n.reshape(1)]))
    want = torch.autograd.grad((ref * dout.double().cpu()).sum() + 0.3 * loss, wide)
    bound = 2 * 400 * 2.0 ** -23
    assert abs(float(router.loss) - float(loss)) <= bound * float(loss)
    assert bool(((out.double().cpu() - ref).abs() <= bound * float(ref.abs().max())).all())
    for a, b in zip(got, want):
        assert bool(((a.double().cpu() - b).abs() <= bound * float(b.abs().max())).all())
    assert not got[1][~mask].any()


def test_balance_alone_and_unused_outputs(moe):
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.randn(40, 8, generator=g, device="cuda").requires_grad_()
    router = moe.gate(z, 2, balance=True)
    by_gate, = torch.autograd.grad(router.loss, z, retain_graph=True)
    loss, counts = moe.balance(z, router.experts.long())
    assert torch.equal(loss, router.loss) and torch.equal(counts, router.counts)
    alone, = torch.autograd.grad(loss * 1.0, z)
    assert torch.equal(alone, by_gate)
    # weights that sum to 1: expanded gradients of ones give nothing
    router.weights.sum().backward()
    assert bool((z.grad.abs() <= 8 * 2.0 ** -24).all())


def test_layer_in_serving(Z, moe):
    # decode: gate, sort, two 4-bit products with a SiLU between, combine; each step against the
    # same one in 64 bits from the step's own inputs
    g = torch.Generator(device="cuda").manual_seed(4)
    T, K, E, H, F = 5, 3, 8, 256, 144
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w1 = torch.randn(E, F, H, generator=g, device="cuda").mul_(H ** -0.5).bfloat16()
    w2 = torch.randn(E, H, F, generator=g, device="cuda").mul_(F ** -0.5).bfloat16()
    up, down = moe.QuantizedExperts4(w1), moe.QuantizedExperts4(w2, group=32, scale_dtype=torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    router = moe.gate(torch.randn(T, E, generator=g, device="cuda"), K, status=status)
    routing = moe.route(router.experts, E, status)
    inside = torch.nn.functional.silu(up(x, routing, status=status))
    made = down(inside, routing, by_expert=True, status=status)
    out = moe.combine(made, routing, router.weights, status)
    assert int(status.item()) == 0
    ends = routing.splits()
    for rows, experts, got in ((x[routing.rows.long()], up, None), (inside, down, made)):
        values, clean = R.unpack4(experts.q.cpu().numpy(), E, experts.outputs, experts.inputs)
        assert clean
        if got is None:
            continue
        want, size = R.product4(host(rows), np.arange(T * K), values, host(experts.scales), experts.group, ends)
        assert np.all(np.abs(host(got) - want) <= 2.0 ** -8 * np.abs(want) + 2 * F * 2.0 ** -23 * size)
    # a 4-bit weight is off by at most half a step: its scale / 2, and what the scale's rounding adds
    values, _ = R.unpack4(up.q.cpu().numpy(), E, F, H)
    step = np.repeat(host(up.scales).transpose(0, 2, 1), 128, axis=2)[:, :, :H]
    assert np.all(np.abs(values * step - host(w1)) <= step * (0.5 + 7 * 2.0 ** -8) + 1e-30)
    terms = host(router.weights)[:, :, None] * host(made)[routing.slots.cpu().numpy()]
    assert np.all(np.abs(host(out) - terms.sum(1)) <= 2.0 ** -8 * np.abs(terms.sum(1)) + K * 2.0 ** -23 * np.abs(terms).sum(1))
