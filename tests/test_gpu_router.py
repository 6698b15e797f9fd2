"""The router's operators on the GPU (choices, weights, balance loss, gradients) against plain
64-bit implementations.

Tolerances follow from the arithmetic, in units u = 2^-24.  exp(z - max) by the hardware's
exp2: the difference, the product and its constant are off by u each, times |z - max| <= R,
the range of the row's open logits, and the exp2 by 2 u.  A probability divides one such
value by a sum of them, of E terms in a tree of at most 16 + 6 steps, over one more rounded
division and product: (6 R + 64) u of it covers all.  A sum over tokens adds as many u as it
has steps in a row (tokens of a lane, waves, the rounding of the result).  A gradient
multiplies a probability's error by the sums of magnitudes of its terms, and those sums
have the tree's steps; then it is rounded once to its type (half a step)."""
import numpy as np
import pytest
import torch

from tests import router_reference as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -125          # exp2 and products that underflow
POISON = 777.0


@pytest.fixture(scope="module")
def Z():
    from lossless_bf16_exponent_codec_amd import zipccl
    return zipccl


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def host(t):
    return t.double().cpu().numpy()


def make_logits(rng, T, E, dtype, spread=3.0, closed=0.0, stride=None, offset=0):
    """tokens x experts on the device, rows `stride` values apart, starting `offset` values into
    their memory; the fp64 values with them."""
    stride = stride or E
    v = rng.standard_normal((T, E)) * spread
    v[rng.random((T, E)) < closed] = -np.inf
    flat = torch.full((T * stride + offset,), POISON, dtype=dtype)
    rows = flat[offset:offset + T * stride].view(T, stride)
    rows[:, :E] = torch.from_numpy(v).to(dtype)
    flat = flat.cuda()
    z = flat[offset:offset + T * stride].view(T, stride)[:, :E]
    return z, host(z)


def spread_of(z, live):
    """R: the largest range of a counted token's open logits."""
    best = 0.0
    for t in np.flatnonzero(live):
        row = z[t][np.isfinite(z[t])]
        if row.size:
            best = max(best, row.max() - row.min())
    return best


def delta(z, live):
    return (6 * spread_of(z, live) + 64) * U


def outputs(T, K, E):
    f, i = torch.float32, torch.int32
    return (torch.full((T, K), -9, dtype=i, device="cuda"), torch.full((T, K), POISON, dtype=f, device="cuda"),
            torch.full((E + 1,), -9, dtype=i, device="cuda"), torch.full((E,), POISON, dtype=f, device="cuda"),
            torch.full((1,), POISON, dtype=f, device="cuda"))


def space(Z):
    return torch.full((Z.MOE_GATE_WORKSPACE_BYTES,), 0xAA, dtype=torch.uint8, device="cuda")


def check_balance(z, mask, ids, counts, sums, loss):
    live = R.counted(z, mask)
    wcounts, wsums, wloss = R.balance(z, mask, ids)
    assert np.array_equal(counts.cpu().numpy(), wcounts)
    d = delta(z, live) + (z.shape[0] // 256 + 64) * U    # tokens in a row: at most those of a workgroup
    assert np.all(np.abs(host(sums) - wsums) <= d * wsums + TINY * max(1, z.shape[0]))
    assert abs(float(loss.double()) - wloss) <= (d + 4 * U) * wloss


def check_gate(Z, z, logits, K, renormalize, mask=None, with_balance=True):
    T, E = z.shape
    ids, w, counts, sums, loss = outputs(T, K, E)
    more = dict(counts=counts, sums=sums, loss=loss, workspace=space(Z)) if with_balance else {}
    dmask = None if mask is None else torch.from_numpy(mask).cuda()
    Z.moe_gate(logits, ids, w, renormalize=renormalize, mask=dmask, **more)
    want = R.choices(z, mask, K)
    assert np.array_equal(ids.cpu().numpy(), want)
    ww = R.weights(z, mask, want, renormalize)
    d = 2 * delta(z, R.counted(z, mask))
    assert np.all(np.abs(host(w) - ww) <= d * ww + TINY)
    if with_balance:
        check_balance(z, mask, want, counts, sums, loss)
    return want, ids


SHAPES = [(1, 1, 1), (1, 8, 256), (5, 2, 3), (7, 3, 16), (64, 8, 64), (65, 1, 17), (33, 4, 33), (100, 16, 100),
          (41, 5, 128), (130, 8, 129), (257, 2, 256), (37, 6, 257), (50, 64, 64), (19, 17, 200), (30, 64, 512),
          (23, 8, 513), (12, 64, 1024), (1500, 3, 61), (9000, 2, 5), (40, 12, 40), (31, 10, 130), (70, 16, 256)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,K,E", SHAPES)
def test_gate(Z, T, K, E, renormalize, dtype):
    rng = np.random.default_rng(T * 7 + E)
    logits, z = make_logits(rng, T, E, dtype)
    check_gate(Z, z, logits, K, renormalize)
    check_gate(Z, z, logits, K, renormalize, with_balance=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,E", [(70, 4, 9), (300, 8, 61), (40, 3, 300), (1, 2, 4)])
def test_closed_experts_and_padding(Z, T, K, E, dtype):
    rng = np.random.default_rng(T + E)
    logits, z = make_logits(rng, T, E, dtype, closed=0.6)
    mask = rng.random(T) < 0.7
    z[~mask] = np.nan                                   # padding may hold anything
    for t in range(0, T, 9):                            # tokens with nowhere to go, and with one place
        z[t] = -np.inf
        if t % 2:
            z[t, E - 1] = 0.5
    z[T // 2] = torch.finfo(dtype).min                  # the type's lowest value is a number: an even spread
    logits.copy_(torch.from_numpy(z).to(dtype))
    z = host(logits)
    for renormalize in (True, False):
        check_gate(Z, z, logits, K, renormalize, mask)
    check_gate(Z, z, logits, K, True, np.zeros(T, bool))
    check_gate(Z, z, logits, K, True, mask.astype(np.uint8) * 7)


def test_equal_logits_go_to_the_lowest_expert(Z):
    z = np.zeros((6, 40))
    z[1] = np.arange(40) // 10                          # ties in tens
    z[2, ::2] = -0.0                                    # both zeros are one value
    z[3, 5:] = -np.inf
    z[4] = -1e30
    z[5, 17] = 1e30
    for dtype in (torch.float32, torch.bfloat16):
        logits = torch.from_numpy(z).to(dtype).cuda()
        ids, w, *_ = outputs(6, 8, 40)
        Z.moe_gate(logits, ids, w)
        assert ids[0].tolist() == list(range(8)) and ids[2].tolist() == list(range(8))
        assert ids[1].tolist() == list(range(30, 38)) and ids[4].tolist() == list(range(8))
        assert ids[3].tolist() == [0, 1, 2, 3, 4, -1, -1, -1] and ids[5].tolist() == [17, 0, 1, 2, 3, 4, 5, 6]
        assert bool((w[0] == 0.125).all()) and w[5].tolist() == [1.0] + [0.0] * 7


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nans_and_infinities_show(Z, dtype):
    inf, nan = float("inf"), float("nan")
    z = torch.zeros(5, 20, dtype=dtype)
    z[0, 7], z[1, 3], z[2, 4], z[2, 9], z[3, 2] = nan, inf, inf, nan, -nan
    z[4, 1] = 2.0
    logits = z.cuda()
    ids, w, counts, sums, loss = outputs(5, 3, 20)
    Z.moe_gate(logits, ids, w, counts=counts, sums=sums, loss=loss, workspace=space(Z))
    assert ids.tolist() == [[7, 0, 1], [3, 0, 1], [9, 4, 0], [2, 0, 1], [1, 0, 2]]
    assert bool(w[:4].isnan().all()) and not bool(w[4].isnan().any())
    assert bool(sums.isnan().all()) and bool(loss.isnan().all()) and int(counts[20]) == 5
    # and in the gradient: the rows that hold them, no others
    d = torch.empty_like(logits)
    dw = torch.ones(5, 3, device="cuda")
    dw[4, 0] = 3.0
    for renormalize in (True, False):
        Z.moe_gate_backward(logits, ids, d, dweights=dw, renormalize=renormalize)
        chosen = torch.zeros(5, 20, dtype=torch.bool, device="cuda").scatter_(1, ids.long(), True)
        assert bool(d[:4][chosen[:4]].isnan().all()) and not bool(d[4].isnan().any()) and bool(d[4, 1] > 0)
        if dtype == torch.bfloat16:
            bits = d.view(torch.int16)[d.isnan()]
            assert bool((bits == 0x7FC0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,stride,offset", [(61, 64, 1), (64, 67, 3), (256, 260, 2), (5, 9, 1), (300, 301, 1)])
def test_strided_and_unaligned_logits(Z, E, stride, offset, dtype):
    rng = np.random.default_rng(E)
    T, K = 77, 4
    logits, z = make_logits(rng, T, E, dtype, stride=stride, offset=offset, closed=0.1)
    _, ids = check_gate(Z, z, logits, K, True)
    flat = torch.full((T * stride + offset,), POISON, dtype=dtype, device="cuda")
    d = flat[offset:].view(T, stride)[:, :E]
    check_backward(Z, z, logits, ids, True, rng, d=d)
    rest = flat[offset:].view(T, stride)[:, E:]
    assert bool((rest == POISON).all()) and bool((flat[:offset] == POISON).all())


@pytest.mark.parametrize("id_dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (70, 2, 16), (500, 4, 64), (333, 20, 8), (4000, 8, 61), (90, 3, 700)])
def test_balance_of_given_choices(Z, T, K, E, id_dtype):
    # any choices: dropped ones, an expert twice, more choices than experts, strided
    rng = np.random.default_rng(T + K)
    logits, z = make_logits(rng, T, E, torch.float32, closed=0.1)
    mask = rng.random(T) < 0.8
    ids = rng.integers(-1, E, (T, K))
    wide = torch.full((T, K + 3), 5, dtype=id_dtype, device="cuda")
    wide[:, :K] = torch.from_numpy(ids).cuda()
    _, _, counts, sums, loss = outputs(T, K, E)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Z.moe_balance(logits, wide[:, :K], counts, sums, loss, space(Z), mask=torch.from_numpy(mask).cuda(), status=status)
    check_balance(z, mask, ids, counts, sums, loss)
    assert int(status.item()) == 0
    ids[T // 2, K // 2] = E
    mask[T // 2] = True
    wide[:, :K] = torch.from_numpy(ids).cuda()
    Z.moe_balance(logits, wide[:, :K], counts, sums, loss, space(Z), mask=torch.from_numpy(mask).cuda(), status=status)
    check_balance(z, mask, ids, counts, sums, loss)
    assert int(status.item()) == (Z.STATUS_BAD_INDEX if R.counted(z, mask)[T // 2] else 0)


def test_balance_of_many_tokens(Z):
    # more tokens than one grid takes at once, against torch in 64 bits
    T, K, E = 200003, 2, 24
    g = torch.Generator(device="cuda").manual_seed(4)
    logits = torch.randn(T, E, generator=g, device="cuda")
    ids, w, counts, sums, loss = outputs(T, K, E)
    Z.moe_gate(logits, ids, w, counts=counts, sums=sums, loss=loss, workspace=space(Z))
    top = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :K]
    assert torch.equal(ids.long(), top)
    p = torch.softmax(logits.double(), 1).sum(0)
    c = torch.bincount(top.reshape(-1), minlength=E)
    assert torch.equal(counts[:E].long(), c) and int(counts[E]) == T
    d = (6 * float(logits.max() - logits.min()) + 64 + T // 256 + 64) * U
    assert bool(((sums.double() - p).abs() <= d * p).all())
    want = E / (K * T * T) * float((c * p).sum())
    assert abs(float(loss) - want) <= (d + 4 * U) * want


def test_no_tokens(Z):
    E, K = 12, 3
    logits = torch.empty(0, E, device="cuda")
    ids, w, counts, sums, loss = outputs(0, K, E)
    Z.moe_gate(logits, ids, w)
    Z.moe_gate(logits, ids, w, counts=counts, sums=sums, loss=loss, workspace=space(Z))
    assert not counts.any() and not sums.any() and float(loss) == 0.0
    Z.moe_gate_backward(logits, ids, logits, counts=counts, dloss=loss)


def check_backward(Z, z, logits, ids, renormalize, rng, mask=None, weights=True, loss=True, d=None):
    T, E = z.shape
    K = ids.shape[1]
    dtype = logits.dtype
    hids = ids.cpu().numpy()
    dw = rng.standard_normal((T, K)).astype(np.float32) if weights else None
    if dw is not None:
        dw[hids < 0] = np.nan                           # a dropped choice's is not read into a sum
    counts, dl = None, None
    if loss:
        counts = R.balance(z, mask, hids)[0]
        dl = np.float32(rng.uniform(0.5, 2.0) * T)
    if d is None:
        d = torch.full((T, E), POISON, dtype=dtype, device="cuda")
    Z.moe_gate_backward(logits, ids, d, dweights=None if dw is None else torch.from_numpy(dw).cuda(),
                        counts=None if counts is None else torch.from_numpy(counts.astype(np.int32)).cuda(),
                        dloss=None if dl is None else torch.tensor([dl], device="cuda"), renormalize=renormalize,
                        mask=None if mask is None else torch.from_numpy(mask).cuda())
    want, size = R.backward(z, mask, hids, renormalize, None if dw is None else np.where(hids < 0, 0, dw), counts, dl)
    live = R.counted(z, mask)
    # three factors of a term have a probability's error; f and dw a rounding each; K terms may meet
    tol = (3 * delta(z, live) + (64 + K) * U) * size + half_step(dtype) * np.abs(want) + TINY * (1 + (dl or 0))
    got = host(d)
    assert np.all(np.abs(got - want) <= tol)
    assert not got[~live].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,K,E", SHAPES)
def test_gradient(Z, T, K, E, renormalize, dtype):
    rng = np.random.default_rng(T * 3 + E)
    logits, z = make_logits(rng, T, E, dtype, closed=0.05)
    mask = rng.random(T) < 0.9
    ids = torch.from_numpy(R.choices(z, mask, K).astype(np.int32)).cuda()
    check_backward(Z, z, logits, ids, renormalize, rng, mask)
    check_backward(Z, z, logits, ids, renormalize, rng, mask, loss=False)
    check_backward(Z, z, logits, ids.long(), renormalize, rng, mask, weights=False)


@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_of_any_choices(Z, renormalize):
    # choices made elsewhere: an expert twice, closed experts, dropped and out of range ones
    rng = np.random.default_rng(12)
    T, K, E = 120, 6, 10
    logits, z = make_logits(rng, T, E, torch.float32, closed=0.3)
    ids = rng.integers(-1, E, (T, K))
    ids[3], ids[4, 1:] = 2, ids[4, 0]
    z[5] = np.where(np.arange(E) < 5, -np.inf, z[5])
    ids[5] = rng.integers(0, 5, K)                      # all closed: no weights, no gradient through them
    logits.copy_(torch.from_numpy(z).float())
    z = host(logits)
    check_backward(Z, z, logits, torch.from_numpy(ids).cuda(), renormalize, rng)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = ids.copy()
    bad[np.flatnonzero(R.counted(z, None))[0], 0] = E
    d, e = (torch.empty(T, E, device="cuda") for _ in range(2))
    dw = torch.randn(T, K, device="cuda")
    Z.moe_gate_backward(logits, torch.from_numpy(bad).cuda(), d, dweights=dw, renormalize=renormalize, status=status)
    assert int(status.item()) == Z.STATUS_BAD_INDEX
    Z.moe_gate_backward(logits, torch.from_numpy(np.where(bad == E, -1, bad)).cuda(), e, dweights=dw,
                        renormalize=renormalize)
    assert torch.equal(d, e)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,E", [(60, 3, 20), (50, 8, 100), (30, 20, 300)])
def test_gradient_of_choices_far_below_the_largest(Z, T, K, E, dtype):
    # exp of what lies 90 to 200 below is nothing beside the row's largest; the weights over such
    # choices are ordinary ones
    rng = np.random.default_rng(E)
    logits, z = make_logits(rng, T, E, dtype)
    logits[:, 0] = torch.from_numpy(rng.uniform(90, 200, T)).to(dtype)
    z = host(logits)
    ids = np.stack([rng.permutation(E - 1)[:K] + 1 for _ in range(T)])
    ids[::5, 0] = 0
    check_backward(Z, z, logits, torch.from_numpy(ids).cuda(), True, rng)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_experts_closed_by_the_lowest_value(Z, dtype):
    # beside open experts the type's lowest value closes one as minus infinity does; a row that
    # holds nothing else is open everywhere
    rng = np.random.default_rng(31)
    T, K, E = 80, 3, 24
    logits, z = make_logits(rng, T, E, dtype, closed=0.5)
    z[:, :K] = np.where(np.isinf(z[:, :K]), 0.0, z[:, :K])
    logits.copy_(torch.from_numpy(z))
    low = torch.where(logits.isinf(), torch.finfo(dtype).min, logits)
    a, b = outputs(T, K, E), outputs(T, K, E)
    dw, dl = torch.randn(T, K, device="cuda"), torch.ones(1, device="cuda")
    grads = []
    for renormalize in (True, False):
        for o, x in ((a, logits), (b, low)):
            Z.moe_gate(x, o[0], o[1], renormalize=renormalize, counts=o[2], sums=o[3], loss=o[4], workspace=space(Z))
            grads.append(torch.empty_like(x))
            Z.moe_gate_backward(x, o[0], grads[-1], dweights=dw, counts=o[2], dloss=dl, renormalize=renormalize)
        assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(*grads[-2:])
    low.fill_(torch.finfo(dtype).min)
    Z.moe_gate(low, b[0], b[1], counts=b[2], sums=b[3], loss=b[4], workspace=space(Z))
    assert b[0].tolist() == [[0, 1, 2]] * T and bool(((b[1] - 1 / 3).abs() <= 4 * U).all())
    assert b[2].tolist() == [T] * K + [0] * (E - K) + [T]


def test_two_calls_at_once(Z):
    # on two streams, each with a workspace of its own, against the same calls one after the other
    g = torch.Generator(device="cuda").manual_seed(11)
    T, K, E = 6000, 4, 130
    logits = [torch.randn(T, E, generator=g, device="cuda") for _ in range(2)]
    made, spaces, streams = [], [space(Z), space(Z)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for rep in range(10):
        o = [outputs(T, K, E) for _ in range(2)]
        torch.cuda.synchronize()
        for i in range(2):
            Z.moe_gate(logits[i], o[i][0], o[i][1], counts=o[i][2], sums=o[i][3], loss=o[i][4], workspace=spaces[i],
                       stream=streams[i] if rep else None)
            if not rep:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        made.append(o)
    for o in made[1:]:
        assert all(torch.equal(x, y) for i in range(2) for x, y in zip(o[i], made[0][i]))


@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_against_differences(Z, renormalize):
    # (F(z + h v) - F(z - h v)) / 2h in 64 bits, F = <dw, weights> + dl loss, choices and counts
    # held: the next term is h^2 / 6 of a third derivative, below 20 in size along a
    # direction of length 1 for values and factors of size 1 here
    rng = np.random.default_rng(3)
    T, K, E, h = 12, 3, 14, 1e-4
    logits, z = make_logits(rng, T, E, torch.float32, spread=1.0)
    ids = R.choices(z, None, K)
    counts = R.balance(z, None, ids)[0]
    dw, dl = rng.uniform(-1, 1, (T, K)).astype(np.float32), np.float32(0.75)

    def f(at):
        sums = np.stack([R.softmax(r) for r in at]).sum(0)
        loss = E / (K * T * T) * (counts[:E] * sums).sum()
        return (R.weights(at, None, ids, renormalize) * dw).sum() + float(dl) * loss

    d = torch.empty(T, E, device="cuda")
    Z.moe_gate_backward(logits, torch.from_numpy(ids).cuda(), d, dweights=torch.from_numpy(dw).cuda(),
                        counts=torch.from_numpy(counts.astype(np.int32)).cuda(), dloss=torch.tensor([dl], device="cuda"),
                        renormalize=renormalize)
    for _ in range(8):
        v = rng.standard_normal((T, E))
        v /= np.linalg.norm(v)
        slope = (f(z + h * v) - f(z - h * v)) / (2 * h)
        # the gradient's own rounding: T * E values of size 1, 200 u each, along a unit direction
        assert abs((host(d) * v).sum() - slope) <= 20 * h * h / 6 + 200 * U * np.sqrt(T * E) + 1e-11


def test_ranks_counts_add_up(Z):
    # two ranks' tokens, counts added: the gradient is that of all tokens' loss
    rng = np.random.default_rng(7)
    T, K, E = 60, 2, 9
    logits, z = make_logits(rng, T, E, torch.float32)
    ids, w, counts, sums, loss = outputs(T, K, E)
    Z.moe_gate(logits, ids, w, counts=counts, sums=sums, loss=loss, workspace=space(Z))
    parts = []
    for a, b in ((0, 25), (25, T)):
        i, _, c, s, _ = o = outputs(b - a, K, E)
        Z.moe_gate(logits[a:b], o[0], o[1], counts=c, sums=s, loss=o[4], workspace=space(Z))
        parts.append((i, c, s))
    assert torch.equal(parts[0][1] + parts[1][1], counts)
    assert bool(((parts[0][2] + parts[1][2] - sums).abs() <= 1e-5 * sums).all())
    dl, d = torch.tensor([2.0], device="cuda"), torch.empty(T, E, device="cuda")
    Z.moe_gate_backward(logits, ids, d, counts=counts, dloss=dl)
    half = torch.empty(T - 25, E, device="cuda")
    Z.moe_gate_backward(logits[25:], parts[1][0], half, counts=parts[0][1] + parts[1][1], dloss=dl)
    assert torch.equal(half, d[25:])


def test_same_bits_on_every_run_and_other_streams(Z):
    g = torch.Generator(device="cuda").manual_seed(9)
    T, K, E = 5000, 4, 100
    logits = torch.randn(T, E, generator=g, device="cuda").bfloat16()
    got = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for rep in range(6):
        o = outputs(T, K, E)
        ws = space(Z)
        torch.cuda.synchronize()
        stream = streams[rep % 2] if rep > 1 else None
        Z.moe_gate(logits, o[0], o[1], counts=o[2], sums=o[3], loss=o[4], workspace=ws, stream=stream)
        torch.cuda.synchronize()
        got.append(o)
    for o in got[1:]:
        for x, y in zip(o, got[0]):
            assert torch.equal(x.view(torch.int32), y.view(torch.int32))


def test_captured_and_replayed(Z):
    g = torch.Generator(device="cuda").manual_seed(10)
    T, K, E = 700, 3, 33
    logits = torch.randn(T, E, generator=g, device="cuda")
    o, ws, d = outputs(T, K, E), space(Z), torch.empty(T, E, device="cuda")
    dw, dl = torch.randn(T, K, generator=g, device="cuda"), torch.tensor([3.0], device="cuda")

    def step(o, d):
        Z.moe_gate(logits, o[0], o[1], counts=o[2], sums=o[3], loss=o[4], workspace=ws)
        Z.moe_gate_backward(logits, o[0], d, dweights=dw, counts=o[2], dloss=dl)

    step(o, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(o, d)
    for rep in range(4):
        logits.copy_(torch.randn(T, E, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        e, ed = outputs(T, K, E), torch.empty(T, E, device="cuda")
        step(e, ed)
        torch.cuda.synchronize()
        for x, y in zip((*o, d), (*e, ed)):
            assert torch.equal(x, y)
