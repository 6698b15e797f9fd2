"""Mixture-of-experts operators on the GPU against plain 64-bit implementations.

Tolerances follow from the arithmetic: a value rounded once to BF16 is off by at most
2^-8 of it; an fp32 sum of n terms by at most n * 2^-24 of the sum of their magnitudes
(taken as n * 2^-23 to cover the products' own rounding); whole numbers are equal."""
import numpy as np
import pytest
import torch

from tests import moe_reference as R

pytestmark = pytest.mark.gpu

POISON = 12345.0
BF16_REL = 2.0 ** -8
TINY = 1e-38


@pytest.fixture(scope="module")
def Z():
    from lossless_bf16_exponent_codec_amd import zipccl
    return zipccl


def rel(dtype):
    return BF16_REL if dtype == torch.bfloat16 else 2.0 ** -23


def values(rng, rows, length, dtype, stride=None, offset=0):
    """A rows x length device tensor, rows `stride` values apart, starting `offset` values
    into its memory."""
    stride = length if stride is None else stride
    flat = torch.from_numpy(rng.standard_normal(rows * stride + offset).astype(np.float32)).to(dtype).cuda()
    return flat[offset:offset + rows * stride].view(rows, stride)[:, :length]


def host(t):
    return t.double().cpu().numpy()


def choices(rng, T, K, E, drop=0.0):
    ids = np.stack([rng.choice(E, K, replace=K > E) for _ in range(T)]) if T else np.zeros((0, K), np.int64)
    ids[rng.random(ids.shape) < drop] = -1
    return ids.astype(np.int64)


def gpu_sort(Z, ids, E, status=None, dtype=torch.int64):
    T, K = ids.shape
    dev = torch.from_numpy(ids).to(dtype).cuda()
    off = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    rows = torch.full((T * K,), -7, dtype=torch.int32, device="cuda")
    slots = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    ws = torch.full((Z.MOE_SORT_WORKSPACE_BYTES,), 0xAA, dtype=torch.uint8, device="cuda")
    Z.moe_sort(dev, E, off, rows, slots, ws, status)
    return off, rows, slots


def check_sort(Z, ids, E, dtype=torch.int64):
    off, rows, slots = gpu_sort(Z, ids, E, dtype=dtype)
    woff, wrows, wslots = R.sort(ids, E)
    assert np.array_equal(off.cpu().numpy(), woff)
    assert np.array_equal(rows.cpu().numpy(), wrows)
    assert np.array_equal(slots.cpu().numpy(), wslots)
    return off, rows, slots


# ------------------------------------------------------------------------------------
# sort
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (1, 8, 8), (3, 2, 5), (63, 1, 2), (64, 8, 256), (65, 3, 1000),
                                   (1000, 4, 64), (2048, 8, 256), (2049, 8, 33), (5000, 7, 1024), (20011, 2, 3)])
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_sort(Z, T, K, E, drop):
    check_sort(Z, choices(np.random.default_rng(T * 31 + K), T, K, E, drop), E)


@pytest.mark.parametrize("T,K", [(7, 3), (9000, 2)])
def test_sort_one_expert_takes_all_or_none(Z, T, K):
    check_sort(Z, np.full((T, K), 4, np.int64), 9)
    check_sort(Z, np.full((T, K), -1, np.int64), 9)


def test_sort_int32_ids_strided(Z):
    rng = np.random.default_rng(5)
    ids = choices(rng, 3000, 5, 40, 0.1)
    check_sort(Z, ids, 40, dtype=torch.int32)
    wide = torch.full((3000, 9), 77, dtype=torch.int64, device="cuda")
    wide[:, :5] = torch.from_numpy(ids).cuda()
    off = torch.empty(41, dtype=torch.int32, device="cuda")
    rows, slots = torch.empty(15000, dtype=torch.int32, device="cuda"), torch.empty(3000, 5, dtype=torch.int32,
                                                                                      device="cuda")
    ws = torch.empty(Z.MOE_SORT_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    Z.moe_sort(wide[:, :5], 40, off, rows, slots, ws)
    woff, wrows, wslots = R.sort(ids, 40)
    assert np.array_equal(off.cpu().numpy(), woff) and np.array_equal(rows.cpu().numpy(), wrows)
    assert np.array_equal(slots.cpu().numpy(), wslots)


@pytest.mark.parametrize("T", [50, 30000])
def test_sort_out_of_range_ids_are_dropped_and_reported(Z, T):
    ids = choices(np.random.default_rng(6), T, 2, 16, 0.2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gpu_sort(Z, ids, 16, status)
    assert int(status.item()) == 0
    ids[T // 2, 1] = 16
    ids[1, 0] = 1 << 40
    off, rows, slots = gpu_sort(Z, ids, 16, status)
    assert int(status.item()) == Z.STATUS_BAD_INDEX
    woff, wrows, wslots = R.sort(ids, 16)
    assert np.array_equal(off.cpu().numpy(), woff) and np.array_equal(slots.cpu().numpy(), wslots)
    assert np.array_equal(rows.cpu().numpy(), wrows)


@pytest.mark.parametrize("T,E", [(1 << 18, 256), (300001, 1000), (700003, 77)])
def test_sort_large(Z, T, E):
    # 2^21 choices and more, the last past 256 workgroups of 16 groups per wave; against a
    # stable sort
    K = 8
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(-3, E, (T, K), generator=g, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    rows, slots = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (T * K, T * K))
    ws = torch.empty(Z.MOE_SORT_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    Z.moe_sort(ids, E, off, rows, slots, ws)
    flat = torch.where(ids < 0, E, ids).view(-1)
    order = torch.sort(flat, stable=True)
    M = int((flat < E).sum())
    assert int(off[E]) == M
    assert torch.equal(off.long(), torch.searchsorted(order.values, torch.arange(E + 1, device="cuda")))
    assert torch.equal(rows[:M].long(), order.indices[:M] // K) and bool((rows[M:] == -1).all())
    want = torch.empty_like(flat)
    want[order.indices] = torch.arange(T * K, device="cuda")
    assert torch.equal(slots.long(), torch.where(flat < E, want, -1))


def test_sort_no_tokens(Z):
    off, rows, slots = gpu_sort(Z, np.zeros((0, 3), np.int64), 6)
    assert not off.any()


# ------------------------------------------------------------------------------------
# dispatch and combine
# ------------------------------------------------------------------------------------
SHAPES = [(1, 1, 1, 1), (1, 8, 8, 7168), (2, 3, 4, 7), (5, 2, 3, 8), (5, 2, 3, 9), (33, 4, 16, 515), (64, 1, 8, 1024),
          (37, 64, 80, 130), (700, 3, 9, 83), (129, 8, 32, 2049), (9, 2, 4, 20001), (300, 2, 5, 4096)]


def setup(rng, T, K, E, drop):
    ids = choices(rng, T, K, E, drop)
    off, rows, slots = R.sort(ids, E)
    return slots, int(off[-1]), torch.from_numpy(slots.astype(np.int32)).cuda()


def poisoned(rows, length, dtype, stride=None):
    t = torch.full((rows, stride or length), POISON, dtype=dtype, device="cuda")
    return t[:, :length]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,E,H", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.5])
def test_dispatch_and_its_gradient(Z, T, K, E, H, dtype, drop):
    rng = np.random.default_rng(H * 7 + T)
    slots, M, dslots = setup(rng, T, K, E, drop)
    x = values(rng, T, H, dtype)
    y = poisoned(M, H, dtype)
    Z.moe_dispatch(x, dslots, y)
    assert np.array_equal(host(y), R.dispatch(host(x), slots, M))
    dy = values(rng, M, H, dtype)
    dx = poisoned(T, H, dtype)
    Z.moe_dispatch_backward(dy, dslots, dx)
    want, size = R.combine(host(dy), slots, None)
    assert np.all(np.abs(host(dx) - want) <= rel(dtype) * np.abs(want) + K * 2.0 ** -23 * size)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,E,H", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.5])
def test_combine_and_its_gradient(Z, T, K, E, H, dtype, drop):
    rng = np.random.default_rng(H * 5 + T)
    slots, M, dslots = setup(rng, T, K, E, drop)
    y = values(rng, M, H, dtype)
    w = torch.from_numpy(rng.random((T, K)).astype(np.float32)).cuda()
    out = poisoned(T, H, dtype)
    Z.moe_combine(y, dslots, w, out)
    want, size = R.combine(host(y), slots, host(w))
    assert np.all(np.abs(host(out) - want) <= rel(dtype) * np.abs(want) + K * 2.0 ** -23 * size)

    dout = values(rng, T, H, dtype)
    dy, dw = poisoned(M, H, dtype), torch.full((T, K), POISON, device="cuda")
    Z.moe_combine_backward(dout, y, dslots, w, dy, dw)
    wdy, wdw, size = R.combine_backward(host(dout), host(y), slots, host(w))
    assert np.all(np.abs(host(dy) - wdy) <= (rel(dtype) + 2.0 ** -23) * np.abs(wdy) + TINY)
    assert np.all(np.abs(host(dw) - wdw) <= H * 2.0 ** -23 * size)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,stride,offset", [(64, 67, 1), (515, 520, 3), (1024, 1024, 5), (8, 8, 1), (5, 6, 1)])
def test_strided_and_unaligned_rows(Z, dtype, H, stride, offset):
    # rows that start at any address of a value, and values beside them that stay
    rng = np.random.default_rng(H + stride)
    T, K, E = 41, 3, 7
    slots, M, dslots = setup(rng, T, K, E, 0.2)

    def holder(rows):
        flat = torch.full((rows * stride + offset,), POISON, dtype=dtype, device="cuda")
        return flat, flat[offset:].view(rows, stride)[:, :H]

    def beside(flat, rows):
        rest = flat[offset:].view(rows, stride)[:, H:]
        return bool((flat[:offset] == flat.new_tensor(POISON)).all()) and bool((rest == rest.new_tensor(POISON)).all())

    x = values(rng, T, H, dtype, stride, offset)
    yf, y = holder(M)
    Z.moe_dispatch(x, dslots, y)
    assert np.array_equal(host(y), R.dispatch(host(x), slots, M)) and beside(yf, M)
    w = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda()
    of, out = holder(T)
    Z.moe_combine(y, dslots, w, out)
    want, size = R.combine(host(y), slots, host(w))
    assert np.all(np.abs(host(out) - want) <= rel(dtype) * np.abs(want) + K * 2.0 ** -23 * size) and beside(of, T)
    df, dy = holder(M)
    dw = torch.full((T, K), POISON, device="cuda")
    Z.moe_combine_backward(x, y, dslots, w, dy, dw)
    wdy, wdw, size = R.combine_backward(host(x), host(y), slots, host(w))
    assert np.all(np.abs(host(dy) - wdy) <= (rel(dtype) + 2.0 ** -23) * np.abs(wdy)) and beside(df, M)
    assert np.all(np.abs(host(dw) - wdw) <= H * 2.0 ** -23 * size)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_against_differences(Z, dtype):
    # combine is linear in y and in the weights, dispatch in x: the difference of two
    # outputs along a direction equals the gradient's product with it.  Values are small
    # whole numbers, so both sides are exact.
    rng = np.random.default_rng(8)
    T, K, E, H = 29, 4, 9, 77
    slots, M, s = setup(rng, T, K, E, 0.3)

    def whole(*shape):
        return torch.from_numpy(rng.integers(-2, 3, shape).astype(np.float32)).cuda()

    y, d, g, x, dxd = (whole(n, H).to(dtype) for n in (M, M, T, T, T))
    w, dw_dir = whole(T, K), whole(T, K)

    def combine(rows, weights):
        out = torch.empty(T, H, dtype=dtype, device="cuda")
        Z.moe_combine(rows, s, weights, out)
        return host(out)

    gy, gw = torch.zeros(M, H, dtype=dtype, device="cuda"), torch.zeros(T, K, device="cuda")
    Z.moe_combine_backward(g, y, s, w, gy, gw)
    assert np.sum(host(g) * (combine(y + d, w) - combine(y, w))) == np.sum(host(gy) * host(d))
    assert np.sum(host(g) * (combine(y, w + dw_dir) - combine(y, w))) == np.sum(host(gw) * host(dw_dir))

    def dispatch(tokens):
        out = torch.zeros(M, H, dtype=dtype, device="cuda")
        Z.moe_dispatch(tokens, s, out)
        return host(out)

    gx = torch.empty(T, H, dtype=dtype, device="cuda")
    Z.moe_dispatch_backward(y, s, gx)
    assert np.sum(host(y) * (dispatch(x + dxd) - dispatch(x))) == np.sum(host(gx) * host(dxd))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dropped_choices_leave_no_trace(Z, dtype):
    # infinities and NaN in rows no choice names and in weights of dropped choices; tokens
    # with every choice dropped; special values in kept rows pass through
    rng = np.random.default_rng(9)
    H, M = 333, 20
    slots = np.array([[-1, -1], [3, -1], [-1, 7], [5, 6], [-5, -1 << 31]], np.int64)
    s = torch.from_numpy(slots.astype(np.int32)).cuda()
    y = values(rng, M, H, dtype)
    y[0], y[1], y[19] = float("nan"), float("inf"), float("-inf")
    y[5, 10], y[6, 11], y[7, 12] = float("inf"), float("nan"), float("-inf")
    w = torch.tensor([[float("nan"), float("inf")], [0.5, float("nan")], [float("-inf"), 2.0], [1.0, 0.0],
                      [float("nan"), 1.0]], device="cuda")
    out = poisoned(5, H, dtype)
    Z.moe_combine(y, s, w, out)
    o = host(out)
    assert not o[0].any() and not o[4].any()
    hy = host(y)
    assert np.all(np.abs(o[1] - 0.5 * hy[3]) <= rel(dtype) * np.abs(hy[3]))
    assert o[2, 12] == -np.inf and np.isfinite(np.delete(o[2], 12)).all()
    assert o[3, 10] == np.inf and np.isnan(o[3, 11])
    dout, dy, dw = values(rng, 5, H, dtype), poisoned(M, H, dtype), torch.full((5, 2), POISON, device="cuda")
    Z.moe_combine_backward(dout, y, s, w, dy, dw)
    d = host(dw)
    assert d[0, 0] == 0 and d[0, 1] == 0 and d[1, 1] == 0 and d[2, 0] == 0 and d[4, 0] == 0 and d[4, 1] == 0
    assert np.isfinite(d[1, 0]) and np.isnan(d[3, 1])
    untouched = [r for r in range(M) if r not in (3, 5, 6, 7)]
    assert bool((dy[untouched] == dy.new_tensor(POISON)).all())
    # a dispatch copies every bit pattern
    if dtype == torch.bfloat16:
        bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(64, 1024).cuda()
        perm = torch.randperm(64, dtype=torch.int32).view(64, 1).cuda()
        got = torch.zeros(64, 1024, dtype=dtype, device="cuda")
        Z.moe_dispatch(bits, perm, got)
        assert torch.equal(got[perm.view(-1).long()].view(torch.int16), bits.view(torch.int16))


def test_nothing_kept_and_no_tokens(Z):
    x = torch.randn(6, 40, device="cuda").bfloat16()
    s = torch.full((6, 3), -1, dtype=torch.int32, device="cuda")
    y = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    out = poisoned(6, 40, torch.bfloat16)
    w, dw = torch.ones(6, 3, device="cuda"), torch.full((6, 3), POISON, device="cuda")
    Z.moe_dispatch(x, s, y)
    Z.moe_combine(y, s, w, out)
    Z.moe_combine_backward(x, y, s, w, y.clone(), dw)
    assert not out.any() and not dw.any()
    none = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    ns = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    Z.moe_dispatch(none, ns, y)
    Z.moe_combine(y, ns, torch.empty(0, 3, device="cuda"), none)
    q = torch.empty(0, 128, dtype=torch.int8, device="cuda")
    scales = torch.empty(0, device="cuda")
    Z.quantize_rows(x, q, scales, slots=s)
    Z.quantize_rows(none, q, scales)
    Z.experts_product(q, scales, torch.zeros(2, 5, 128, dtype=torch.int8, device="cuda"), torch.zeros(2, 5, device="cuda"),
                      40, torch.empty(0, 5, device="cuda"), offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()


def test_slots_past_the_rows_are_dropped_and_reported(Z):
    rng = np.random.default_rng(10)
    H, M = 100, 6
    s = torch.tensor([[0, 6], [1 << 30, 2], [3, -1]], dtype=torch.int32, device="cuda")
    slots = s.cpu().numpy()
    x, y = values(rng, 3, H, torch.float32), values(rng, M, H, torch.float32)
    w = torch.ones(3, 2, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = poisoned(M, H, torch.float32)
    Z.moe_dispatch(x, s, got, status)
    want = R.dispatch(host(x), slots, M)
    kept = [0, 2, 3]
    assert int(status.item()) == Z.STATUS_BAD_INDEX and np.array_equal(host(got)[kept], want[kept])
    status.zero_()
    out = poisoned(3, H, torch.float32)
    Z.moe_combine(y, s, w, out, status)
    assert int(status.item()) == Z.STATUS_BAD_INDEX and np.array_equal(host(out), R.combine(host(y), slots, None)[0])
    status.zero_()
    dy, dw = poisoned(M, H, torch.float32), torch.empty(3, 2, device="cuda")
    Z.moe_combine_backward(x, y, s, w, dy, dw, status)
    assert int(status.item()) == Z.STATUS_BAD_INDEX and float(dw[0, 1]) == 0 and float(dw[1, 0]) == 0
    status.zero_()
    q, scales = torch.zeros(M, 128, dtype=torch.int8, device="cuda"), torch.zeros(M, device="cuda")
    Z.quantize_rows(x.bfloat16(), q, scales, slots=s, status=status)
    assert int(status.item()) == Z.STATUS_BAD_INDEX
    assert q[kept].any(1).all() and not q[[1, 4, 5]].any() and not scales[[1, 4, 5]].any()


def test_rows_past_32_bits(Z):
    # rows 2^21 + 3 values apart: the last of 1100 starts past 2^32 bytes in BF16 and 2^33 in fp32
    for dtype in (torch.bfloat16, torch.float32):
        rng = np.random.default_rng(11)
        T, K, H, stride = 1100, 1, 777, (1 << 21) + 3
        x = values(rng, T, H, dtype)
        s = torch.from_numpy(rng.permutation(T).astype(np.int32)).cuda().view(T, 1)
        y = torch.empty(T * stride, dtype=dtype, device="cuda").view(T, stride)[:, :H]
        Z.moe_dispatch(x, s, y)
        assert torch.equal(y[s.view(-1).long()], x)
        out = poisoned(T, H, dtype)
        Z.moe_combine(y, s, None, out)
        assert torch.equal(out, x)
        dy, dw = torch.empty(T * stride, dtype=dtype, device="cuda").view(T, stride)[:, :H], torch.empty(T, 1, device="cuda")
        Z.moe_combine_backward(x, y, s, torch.ones(T, 1, device="cuda"), dy, dw)
        assert torch.equal(dy[s.view(-1).long()], x)
        want = (host(x) ** 2).sum(1)
        assert np.all(np.abs(host(dw)[:, 0] - want) <= H * 2.0 ** -23 * want)


def test_many_tokens_step_over_the_grid(Z):
    # more token groups than a grid's second dimension holds
    T, H = 4 * 65535 + 9, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    s = torch.randperm(T, generator=g, device="cuda").int().view(T, 1)
    y = torch.empty_like(x)
    Z.moe_dispatch(x, s, y)
    assert torch.equal(y[s.view(-1).long()], x)
    out = torch.empty_like(x)
    Z.moe_combine(y, s, None, out)
    assert torch.equal(out, x)


@pytest.mark.parametrize("dtype,T,K,H", [
    (torch.bfloat16, 2000, 16, 4096), (torch.bfloat16, 9000, 3, 4096), (torch.bfloat16, 9000, 1, 16320),
    (torch.bfloat16, 2000, 16, 4099), (torch.float32, 1500, 20, 2048),
    (torch.float32, 1500, 20, 2051), (torch.bfloat16, 40000, 6, 515), (torch.bfloat16, 140000, 1, 1030),
    (torch.bfloat16, 3000000, 1, 7), (torch.float32, 6000000, 1, 3)])
def test_more_than_the_caches_and_one_slice(Z, dtype, T, K, H):
    # rows and tokens past the Infinity Cache, and more chunks than a slice of the grid
    g = torch.Generator(device="cuda").manual_seed(H)
    M = T * K - T // 3
    perm = torch.randperm(T * K, generator=g, device="cuda")
    s = torch.where(perm < M, perm, -1).int().view(T, K)
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    w = torch.rand(T, K, generator=g, device="cuda")
    flat = s.view(-1)
    kept = torch.nonzero(flat >= 0).squeeze(1)
    token, row = kept // K, flat[kept].long()
    y = poisoned(M, H, dtype)
    Z.moe_dispatch(x, s, y)
    assert torch.equal(y[row], x[token])
    y = torch.randn(M, H, generator=g, device="cuda").to(dtype)
    for weights, run in ((None, lambda out: Z.moe_dispatch_backward(y, s, out)), (w, lambda out: Z.moe_combine(y, s, w, out))):
        out = poisoned(T, H, dtype)
        run(out)
        for a in range(0, T, 1 << 19):   # in parts: 64-bit copies are large
            b = min(T, a + (1 << 19))
            terms = [torch.where((s[a:b, k] >= 0).unsqueeze(1), y[s[a:b, k].clamp(min=0).long()].double(), 0.0)
                     * (1.0 if weights is None else w[a:b, k:k + 1].double()) for k in range(K)]
            want, size = sum(terms), sum(t.abs() for t in terms)
            assert bool(((out[a:b].double() - want).abs() <= rel(dtype) * want.abs() + K * 2.0 ** -23 * size).all())
    dy, dw = poisoned(M, H, dtype), torch.full((T, K), POISON, device="cuda")
    Z.moe_combine_backward(x, y, s, w, dy, dw)
    for a in range(0, kept.numel(), 1 << 17):
        t, r, at = token[a:a + (1 << 17)], row[a:a + (1 << 17)], kept[a:a + (1 << 17)]
        want = x[t].double() * w.view(-1)[at].double().unsqueeze(1)
        assert bool(((dy[r].double() - want).abs() <= (rel(dtype) + 2.0 ** -23) * want.abs() + TINY).all())
        dots = x[t].double() * y[r].double()
        assert bool(((dw.view(-1)[at].double() - dots.sum(1)).abs() <= H * 2.0 ** -23 * dots.abs().sum(1)).all())
    assert not dw.view(-1)[flat < 0].any()


def test_dispatch_of_more_than_one_slice_of_streamed_rows(Z):
    T, H = 540000, 4096   # 8 KB a row: 2^22 parts are 524288 tokens
    x = torch.randint(-30000, 30000, (T, H), dtype=torch.int16, device="cuda").view(torch.bfloat16)
    s = torch.randperm(T, device="cuda").int().view(T, 1)
    s[7] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.zeros_like(x)
    Z.moe_dispatch(x, s, y, status)
    kept = torch.nonzero(s.view(-1) >= 0).squeeze(1)
    assert int(status.item()) == 0 and torch.equal(y[s.view(-1)[kept].long()].view(torch.int16), x[kept].view(torch.int16))
    s[9] = T
    Z.moe_dispatch(x, s, y, status)
    assert int(status.item()) == Z.STATUS_BAD_INDEX


# ------------------------------------------------------------------------------------
# 8-bit rows
# ------------------------------------------------------------------------------------
def gpu_quantize(Z, x, slots=None, nrows=None):
    H = x.shape[1]
    M = x.shape[0] if slots is None else nrows
    wide = -(-H // 128) * 128
    q = torch.full((M, wide), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((M,), POISON, device="cuda")
    Z.quantize_rows(x, q, scales, slots=slots)
    return q, scales


def same(a, b):
    return np.array_equal(a, b, equal_nan=True)


@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (2, 8), (65, 127), (5, 128), (4, 129), (17, 2048), (300, 1000),
                                 (9, 7168), (3, 8192), (2, 8193), (1, 50001)])
def test_quantize_rows(Z, T, H):
    rng = np.random.default_rng(H)
    x = values(rng, T, H, torch.bfloat16) * torch.from_numpy(10.0 ** rng.uniform(-30, 30, (T, 1))).cuda().bfloat16()
    x[T // 2] = 0
    q, scales = gpu_quantize(Z, x)
    wq, ws = R.quantize(host(x))
    assert np.array_equal(q.cpu().numpy()[:, :H], wq)
    assert not q[:, H:].any()
    assert np.array_equal(scales.cpu().numpy(), ws.astype(np.float32))


def test_quantize_every_pair_of_significands(Z):
    # every peak significand and every value of either sign down to 2^-9 of it, ties among
    # them, at ordinary, largest, smallest normal and subnormal exponents
    q_of, x_of = [], []
    for e in (0, 126, -120, -126, -130):
        for a in range(128, 256):
            row = [float(a) * 2.0 ** (e - 7)]
            for d in range(0, 10):
                row += [s * v * 2.0 ** (e - 7 - d) for v in range(128, 256) for s in (1.0, -1.0) if v * 2.0 ** -d <= a]
            row += [0.0] * (2561 - len(row))
            x_of.append(row)
    x = torch.tensor(x_of, dtype=torch.float64).to(torch.float32).to(torch.bfloat16).cuda()
    q, scales = gpu_quantize(Z, x)
    wq, ws = R.quantize(host(x))
    assert np.array_equal(q.cpu().numpy()[:, :x.shape[1]], wq)
    assert np.array_equal(scales.cpu().numpy(), ws.astype(np.float32))


def test_quantize_special_rows(Z):
    x = torch.randn(6, 300, device="cuda").bfloat16()
    x[1, 299], x[2, 0], x[3, 128] = float("inf"), float("nan"), float("-inf")
    x[4] = 0
    x[5] = 0
    x[5, 17] = -2.0 ** -133   # the smallest BF16 value
    q, scales = gpu_quantize(Z, x)
    wq, ws = R.quantize(host(x))
    assert np.array_equal(q.cpu().numpy()[:, :300], wq) and not q[:, 300:].any()
    assert same(scales.cpu().numpy(), ws.astype(np.float32))
    assert int(q[5, 17]) == -127


@pytest.mark.parametrize("T,K,E,H", [(1, 8, 8, 7168), (50, 3, 6, 515), (129, 2, 40, 2049), (7, 64, 70, 64)])
def test_quantize_to_slots(Z, T, K, E, H):
    rng = np.random.default_rng(T)
    slots, M, dslots = setup(rng, T, K, E, 0.3)
    x = values(rng, T, H, torch.bfloat16, H + 5, 3)
    q, scales = gpu_quantize(Z, x, dslots, M)
    wq, ws = R.quantize(host(x))
    for t in range(T):
        for s in slots[t]:
            if s >= 0:
                assert np.array_equal(q[s].cpu().numpy()[:H], wq[t]) and not q[s, H:].any()
                assert float(scales[s]) == np.float32(ws[t])


# ------------------------------------------------------------------------------------
# product
# ------------------------------------------------------------------------------------
def product_inputs(rng, M, E, N, H):
    wide = -(-H // 128) * 128
    q, w = np.zeros((M, wide), np.int8), np.zeros((E, N, wide), np.int8)
    q[:, :H] = rng.integers(-128, 128, (M, H))
    w[:, :, :H] = rng.integers(-128, 128, (E, N, H))
    return q, rng.uniform(0.5, 2, M).astype(np.float32), w, rng.uniform(-1, 1, (E, N)).astype(np.float32)


def check_product(Z, rng, counts, N, H, dtype, gap=0):
    """counts: rows of each expert; gap: rows after the last expert's."""
    offsets = np.concatenate([[0], np.cumsum(counts)])
    M, E = int(offsets[-1]) + gap, len(counts)
    q, s, w, ws = product_inputs(rng, M, E, N, H)
    dq, dsc, dw, dws = (torch.from_numpy(v).cuda() for v in (q, s, w, ws))
    out = poisoned(M, N, dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Z.experts_product(dq, dsc, dw, dws, H, out, offsets=torch.from_numpy(offsets.astype(np.int32)).cuda(), status=status)
    assert int(status.item()) == 0
    want = R.product(q, s, w, ws, offsets)
    got = host(out)
    filled = int(offsets[-1])
    assert np.all(np.abs(got[:filled] - want[:filled]) <= (rel(dtype) + 4 * 2.0 ** -24) * np.abs(want[:filled]))
    assert bool((out[filled:] == out.new_tensor(POISON)).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,N,H", [
    ([1], 1, 1), ([1], 16, 128), ([1] * 8, 100, 200), ([0, 3, 0, 1], 33, 129), ([5, 0, 0, 12, 7], 257, 1000),
    ([16, 17, 15], 64, 640), ([33, 64, 1, 0, 90], 130, 7168), ([128, 1, 127, 129], 128, 256), ([300, 2, 70], 511, 384),
    ([0] * 70 + [9] + [0] * 60 + [20, 1], 70, 300), ([1000, 255, 257], 300, 520), ([600], 1024, 1024),
    ([257, 600, 31], 513, 900)])
def test_product(Z, counts, N, H, dtype):
    check_product(Z, np.random.default_rng(N + H), counts, N, H, dtype)


@pytest.mark.parametrize("counts,N,H", [
    ([16640], 1280, 2000),                # 65 x 5 tiles of 256 x 256: a part round of 69, a total that is no multiple of 8
    ([8400], 2048, 2048),                 # a round of 256 and 8 tiles over
    ([5000, 3000, 300, 77], 2290, 2100),  # 35 x 9, 59 over; edges inside tiles on both sides
    ([100] * 3 + [40000], 513, 130),      # most rows with one expert
    ([300] * 70, 1024, 1930),             # more experts than lanes
    ([16640], 1280, 128), ([8400], 2048, 256), ([5000, 3000, 300, 77], 2050, 384),
    ([130] * 64, 300, 200), ([40] * 100, 200, 300), ([64] * 20, 2000, 128)])
def test_product_many_tiles(Z, counts, N, H):
    check_product(Z, np.random.default_rng(N), counts, N, H, torch.bfloat16)


def test_product_rows_outside_every_range_stay(Z):
    check_product(Z, np.random.default_rng(1), [4, 9], 70, 130, torch.float32, gap=5)
    check_product(Z, np.random.default_rng(1), [400, 90], 70, 130, torch.bfloat16, gap=300)


@pytest.mark.parametrize("M", [1, 3, 40, 200, 700])
def test_product_of_one_matrix(Z, M):
    rng = np.random.default_rng(2)
    q, s, w, ws = product_inputs(rng, M, 1, 333, 450)
    out = poisoned(M, 333, torch.float32, stride=340)
    Z.experts_product(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), torch.from_numpy(w[0]).cuda(),
                      torch.from_numpy(ws).cuda(), 450, out)
    want = R.product(q, s, w, ws, [0, M])
    assert np.all(np.abs(host(out) - want) <= 6 * 2.0 ** -24 * np.abs(want))


@pytest.mark.parametrize("M", [2, 100, 600])
def test_product_largest_sums(Z, M):
    # every product -128 * -128 over the longest row: 2147467264, 16384 below 2^31
    H = 131071
    wide = 131072
    q = torch.full((M, wide), -128, dtype=torch.int8, device="cuda")
    w = torch.full((3, wide), -128, dtype=torch.int8, device="cuda")
    q[:, H:], w[:, H:] = 0, 0
    out = torch.empty(M, 3, device="cuda")
    Z.experts_product(q, torch.ones(M, device="cuda"), w, torch.ones(3, device="cuda"), H, out)
    assert bool((out == float(np.float32(16384 * H))).all())


def test_product_offsets_out_of_range_are_clamped(Z):
    rng = np.random.default_rng(4)
    M, E, N, H = 50, 4, 40, 256
    q, s, w, ws = product_inputs(rng, M, E, N, H)
    dev = [torch.from_numpy(v).cuda() for v in (q, s, w, ws)]
    for offsets in ([-5, 10, 20, 30, 1000], [0, 60, 70, 80, 90], [40, 30, 20, 10, 0], [-9, -8, -7, -6, -5]):
        out = poisoned(M, N, torch.float32)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        Z.experts_product(*dev, H, out, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), status=status)
        assert int(status.item()) == Z.STATUS_BAD_INDEX
        clean = [min(max(o, 0), M) for o in offsets]
        if all(a <= b for a, b in zip(clean, clean[1:])):
            want = R.product(q, s, w, ws, clean)
            got = host(out)
            held = ~np.isnan(want[:, 0])
            assert np.all(np.abs(got[held] - want[held]) <= 6 * 2.0 ** -24 * np.abs(want[held]))
            assert np.all(got[~held] == POISON)


def test_product_rows_with_nan_scale(Z):
    x = torch.randn(5, 200, device="cuda").bfloat16()
    x[3, 7] = float("nan")
    x[1] = 0
    q, scales = gpu_quantize(Z, x)
    w = torch.randint(-127, 128, (30, 256), dtype=torch.int8, device="cuda")
    out = torch.empty(5, 30, device="cuda")
    Z.experts_product(q, scales, w, torch.ones(30, device="cuda"), 200, out)
    assert bool(out[3].isnan().all()) and not out[1].any() and bool(out[[0, 2, 4]].isfinite().all())


@pytest.mark.parametrize("counts", [[3, 1], [700, 300]])
def test_product_strided_and_unaligned_out(Z, counts):
    rng = np.random.default_rng(12)
    M, N, H = sum(counts), 77, 300
    q, s, w, ws = product_inputs(rng, M, 2, N, H)
    flat = torch.full((M * 83 + 1,), POISON, dtype=torch.bfloat16, device="cuda")
    out = flat[1:].view(M, 83)[:, :N]
    wide = torch.zeros(M, 512, dtype=torch.int8, device="cuda")
    wide[:, :384] = torch.from_numpy(q).cuda()
    wide[:, 384:] = 55   # past the padding: never part of a sum
    Z.experts_product(wide, torch.from_numpy(s).cuda(), torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda(), H, out,
                      offsets=torch.tensor([0, counts[0], M], dtype=torch.int32, device="cuda"))
    want = R.product(q, s, w, ws, [0, counts[0], M])
    assert np.all(np.abs(host(out) - want) <= (BF16_REL + 4 * 2.0 ** -24) * np.abs(want))
    assert bool((flat[1:].view(M, 83)[:, N:] == flat.new_tensor(POISON)).all()) and float(flat[0]) == float(flat.new_tensor(POISON))


def test_product_past_32_bits(Z):
    # q rows and weights that end past 2^32 bytes, out past 2^32 values
    M, H, stride = 600, 200, 8 << 20
    q = torch.empty(M, stride, dtype=torch.int8, device="cuda")
    q[:, :256] = 0
    q[:, :H] = torch.randint(-127, 128, (M, H), dtype=torch.int8, device="cuda")
    w = torch.empty(3, 200, stride, dtype=torch.int8, device="cuda")
    w[:, :, :256] = 0
    w[:, :, :H] = torch.randint(-127, 128, (3, 200, H), dtype=torch.int8, device="cuda")
    out = torch.empty(M, stride, dtype=torch.bfloat16, device="cuda")[:, :200]
    offsets = [0, 5, 300, 600]
    ones, wones = torch.ones(M, device="cuda"), torch.ones(3, 200, device="cuda")
    Z.experts_product(q, ones, w, wones, H, out, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    want = R.product(q[:, :H].cpu().numpy(), np.ones(M), w[:, :, :H].cpu().numpy(), np.ones((3, 200)), offsets)
    assert np.all(np.abs(host(out) - want) <= (BF16_REL + 4 * 2.0 ** -24) * np.abs(want))


# ------------------------------------------------------------------------------------
# all together
# ------------------------------------------------------------------------------------
class Layer:
    """Buffers of one pass: sort, quantise to the experts, product, combine, gradient."""

    def __init__(self, Z, T, K, E, H, N):
        self.Z, self.T, self.K, self.E, self.H = Z, T, K, E, H
        dev, M = dict(device="cuda"), T * K
        wide = -(-H // 128) * 128
        self.ids = torch.zeros(T, K, dtype=torch.int64, **dev)
        self.x = torch.zeros(T, H, dtype=torch.bfloat16, **dev)
        self.weights = torch.zeros(T, K, **dev)
        self.w = torch.zeros(E, N, wide, dtype=torch.int8, **dev)
        self.w[:, :, :H] = torch.randint(-127, 128, (E, N, H), dtype=torch.int8, **dev)
        self.ws = torch.rand(E, N, **dev) * 1e-3
        self.off = torch.zeros(E + 1, dtype=torch.int32, **dev)
        self.rows, self.slots = torch.zeros(M, dtype=torch.int32, **dev), torch.zeros(T, K, dtype=torch.int32, **dev)
        self.space = torch.zeros(Z.MOE_SORT_WORKSPACE_BYTES, dtype=torch.uint8, **dev)
        self.q, self.scales = torch.zeros(M, wide, dtype=torch.int8, **dev), torch.zeros(M, **dev)
        self.y, self.dy = (torch.zeros(M, N, dtype=torch.bfloat16, **dev) for _ in range(2))
        self.copy, self.dx = torch.zeros(M, H, dtype=torch.bfloat16, **dev), torch.zeros_like(self.x)
        self.out, self.dw = torch.zeros(T, N, dtype=torch.bfloat16, **dev), torch.zeros(T, K, **dev)

    def fill(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ids.copy_(torch.rand(self.T, self.E, generator=g, device="cuda").topk(self.K).indices)
        self.x.copy_(torch.randn(self.T, self.H, generator=g, device="cuda"))
        self.weights.copy_(torch.rand(self.T, self.K, generator=g, device="cuda"))

    def run(self):
        Z = self.Z
        Z.moe_sort(self.ids, self.E, self.off, self.rows, self.slots, self.space)
        Z.quantize_rows(self.x, self.q, self.scales, slots=self.slots)
        Z.experts_product(self.q, self.scales, self.w, self.ws, self.H, self.y, offsets=self.off)
        Z.moe_combine(self.y, self.slots, self.weights, self.out)
        Z.moe_combine_backward(self.out, self.y, self.slots, self.weights, self.dy, self.dw)
        Z.moe_dispatch(self.x, self.slots, self.copy)
        Z.moe_dispatch_backward(self.copy, self.slots, self.dx)

    def results(self):
        return [t.clone() for t in (self.off, self.rows, self.slots, self.q, self.scales, self.y, self.out, self.dy,
                                    self.dw, self.copy, self.dx)]


def equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T,K,E,H,N", [(5, 2, 4, 200, 100), (4000, 8, 32, 200, 136), (1100, 2, 3, 1000, 520)])
def test_same_bits_on_every_run_and_stream(Z, T, K, E, H, N):
    L = Layer(Z, T, K, E, H, N)
    L.fill(1)
    L.run()
    first = L.results()
    L.fill(2)
    L.run()
    L.fill(1)
    L.run()
    assert equal(first, L.results())
    # another stream, right behind the work there that makes the inputs
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.fill(2)
        L.fill(1)
        L.run()
        again = L.results()
    torch.cuda.current_stream().wait_stream(side)
    assert equal(first, again)


@pytest.mark.parametrize("T,K,E,H,N", [(5, 2, 4, 200, 100), (4000, 8, 32, 200, 136)])
def test_graph_replays_equal_eager_runs(Z, T, K, E, H, N):
    L = Layer(Z, T, K, E, H, N)
    want = []
    for seed in (1, 2, 3):
        L.fill(seed)
        L.run()
        want.append(L.results())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        L.run()
    for rep in range(3):
        for seed in (1, 2, 3):
            L.fill(seed)
            graph.replay()
            torch.cuda.synchronize()
            assert equal(want[seed - 1], L.results()), (rep, seed)


def test_row_lists_feed_the_gathered_compress(Z):
    # the sorted rows, cut by destination, compress straight from the token matrix; decoded
    # they are the dispatched rows, bit for bit
    from lossless_bf16_exponent_codec_amd import workloads as W
    T, K, E, H, ranks = 600, 2, 16, 1024, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.from_numpy(W.gaussian_bf16(T * H, 0.5, 4).view(np.int16)).cuda().view(torch.bfloat16).view(T, H)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(K).indices
    off, rows, slots = gpu_sort(Z, ids.cpu().numpy(), E)
    ends = off.tolist()
    M = ends[-1]
    cuts = [(ends[r * E // ranks], ends[(r + 1) * E // ranks]) for r in range(ranks)]
    static = torch.empty(sum(Z.static_size((b - a) * H) for a, b in cuts), dtype=torch.uint8, device="cuda")
    esc = torch.empty(M * H, dtype=torch.uint8, device="cuda")
    ws = torch.empty(Z.workspace_size(M * H, ranks), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = Z.plan(sigma=0.5)
    Z.compress_gather([(x, rows[a:b], plan) for a, b in cuts], static, esc, ws, status=status)
    got = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    Z.decompress(static, esc, [got[a:b] for a, b in cuts], status)
    y = torch.empty_like(got)
    Z.moe_dispatch(x, slots, y)
    assert int(status.item()) == 0 and torch.equal(got.view(torch.int16), y.view(torch.int16))
