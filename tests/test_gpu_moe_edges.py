"""Mixture-of-experts operators on the GPU where calls are largest and where their inputs are
wrong: loops over more work than a grid has workgroups, offsets that are out of range, NaN
scales, rows that no choice has.  Tolerances as in the other tests of these operators: a value
rounded once to BF16 is off by at most 2^-8 of it, an fp32 sum of n terms by at most n * 2^-23
of the sum of their magnitudes; whole numbers are equal."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16_REL = 2.0 ** -8
SHAPES = [  # experts, rows, outputs, row length: a call of each tile shape
    (4, 50, 40, 256), (128, 1, 40, 200), (128, 40, 40, 130), (70, 3000, 300, 200), (70, 3000, 700, 200),
    (70, 9000, 300, 200), (5, 9000, 300, 200), (100, 22000, 1024, 2048)]


@pytest.fixture(scope="module")
def Z():
    from lossless_bf16_exponent_codec_amd import zipccl
    return zipccl


def operands(E, M, N, H):
    g = torch.Generator(device="cuda").manual_seed(E + M + N)
    wide = -(-H // 128) * 128
    q = torch.zeros(M, wide, dtype=torch.int8, device="cuda")
    w = torch.zeros(E, N, wide, dtype=torch.int8, device="cuda")
    q[:, :H] = torch.randint(-127, 128, (M, H), generator=g, device="cuda", dtype=torch.int8)
    w[:, :, :H] = torch.randint(-127, 128, (E, N, H), generator=g, device="cuda", dtype=torch.int8)
    return q, torch.rand(M, generator=g, device="cuda") + 0.5, w, torch.rand(E, N, generator=g, device="cuda") + 0.5


def even(E, M):
    return [M * e // E for e in range(E + 1)]


@pytest.mark.parametrize("E,M,N,H", SHAPES)
def test_every_offset_out_of_range_is_reported(Z, E, M, N, H):
    q, scales, w, w_scales = operands(E, M, N, H)
    good = even(E, M)

    def run(offsets):
        out = torch.full((M, N), 12345.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        Z.experts_product(q, scales, w, w_scales, H, out, status=status,
                          offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
        return out, int(status.item())

    def check(out, offsets):
        held = torch.zeros(M, dtype=torch.bool)
        for e in range(E):
            a, b = offsets[e], offsets[e + 1]
            if a < b:
                held[a:b] = True
                sums = q[a:b].double() @ w[e].double().t().contiguous()
                want = sums * scales[a:b, None].double() * w_scales[e].double()
                assert bool(((out[a:b].double() - want).abs() <= 4 * 2.0 ** -24 * want.abs()).all())
        assert bool((out[~held.cuda()] == 12345.0).all())

    out, status = run(good)
    assert status == 0
    check(out, good)
    for at in 0, E // 3, E - 1, E:   # out of range, the others ascending where they are clamped
        for value in -5, M + 1000:
            offsets = [min(v, value) if i < at else max(v, value) if i > at else value for i, v in enumerate(good)]
            out, status = run(offsets)
            assert status == Z.STATUS_BAD_INDEX, (at, value)
            check(out, [min(max(v, 0), M) for v in offsets])
    for rest in good, [0] + [M] * E:  # one alone; the rows with all experts or with the first
        for at in 1, E // 3 + 1, E - 1:
            for value in -5, M + 1000:
                offsets = list(rest)
                offsets[at] = value
                assert run(offsets)[1] == Z.STATUS_BAD_INDEX, (rest[1], at, value)
    for at in 0, E // 3, E - 1:      # in range, descending
        offsets = [M] * (at + 1) + [0] + [M] * (E - at - 1)
        assert run(offsets)[1] == Z.STATUS_BAD_INDEX, at


@pytest.mark.parametrize("E,M,N,H", SHAPES)
def test_nan_products_are_one_bit_pattern(Z, E, M, N, H):
    # NaNs of either sign and any payload, quiet and signalling, in rows' and channels' scales,
    # and infinity times zero: 0x7FC0 in BF16
    q, scales, w, w_scales = operands(E, M, N, H)
    nans = torch.tensor([-0x400000, 0x7FFFFFFF, 0x7FA12345, 0x7F800001, -1], dtype=torch.int32, device="cuda")   # bits
    rows, zero_rows, columns = slice(0, M, 7), slice(3, M, 7), slice(1, N, 9)
    scales.view(torch.int32)[rows] = nans[torch.arange(0, M, 7, device="cuda") % 5]
    w_scales.view(torch.int32)[:, columns] = nans[torch.arange(1, N, 9, device="cuda") % 5]
    q[zero_rows], scales[zero_rows] = 0, float("inf")
    out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    Z.experts_product(q, scales, w, w_scales, H, out,
                      offsets=torch.tensor(even(E, M), dtype=torch.int32, device="cuda"))
    want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    want[rows], want[:, columns], want[zero_rows] = True, True, True
    assert bool((out.view(torch.int16)[want] == 0x7FC0).all())
    assert bool(out[~want].isfinite().all())


# ------------------------------------------------------------------------------------
# more work than a grid: the kernels' loops take a second turn
# ------------------------------------------------------------------------------------
def parts(n, size):
    return [slice(a, min(n, a + size)) for a in range(0, n, size)]


def test_combine_by_waves_of_more_tokens_than_a_grid(Z):
    # whole 1 KB parts at aligned addresses, past the Infinity Cache: groups of 4 tokens, 65535 in a grid
    T, H = 4 * 65535 + 9, 512
    g = torch.Generator(device="cuda").manual_seed(1)
    y = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    slots = torch.randperm(T, generator=g, device="cuda").int().view(T, 1)
    weights = torch.rand(T, 1, generator=g, device="cuda")
    out = torch.full_like(y, 12345.0)
    Z.moe_combine(y, slots, weights, out)
    for s in parts(T, 1 << 17):
        want = y[slots[s, 0].long()].double() * weights[s].double()
        assert bool(((out[s].double() - want).abs() <= (BF16_REL + 2.0 ** -23) * want.abs()).all())


@pytest.mark.parametrize("T,H", [((1 << 20) + 5, 1025), (4 * (1 << 20) + 7, 264)])
def test_combine_gradient_of_more_tokens_than_a_grid(Z, T, H):
    # 2^20 workgroups: of a token each, and of four
    g = torch.Generator(device="cuda").manual_seed(2)
    y, dout = (torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    slots = torch.randperm(T, generator=g, device="cuda").int().view(T, 1)
    weights = torch.rand(T, 1, generator=g, device="cuda")
    dy, dw = torch.full_like(y, 12345.0), torch.full((T, 1), 12345.0, device="cuda")
    Z.moe_combine_backward(dout, y, slots, weights, dy, dw)
    for s in parts(T, 1 << 17):
        at, d = slots[s, 0].long(), dout[s].double()
        want = d * weights[s].double()
        assert bool(((dy[at].double() - want).abs() <= (BF16_REL + 2.0 ** -23) * want.abs()).all())
        terms = d * y[at].double()
        assert bool(((dw[s, 0].double() - terms.sum(1)).abs() <= H * 2.0 ** -23 * terms.abs().sum(1)).all())


@pytest.mark.parametrize("T,H", [((1 << 20) + 5, 2049), (4 * (1 << 20) + 7, 72)])
def test_quantize_more_tokens_than_a_grid(Z, T, H):
    # 2^20 workgroups: of a token each, and of four
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    x[::1000] = 0
    q = torch.full((T, -(-H // 128) * 128), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((T,), 12345.0, device="cuda")
    Z.quantize_rows(x, q, scales)
    for s in parts(T, 1 << 17):
        wide = x[s].double()
        peak = wide.abs().amax(1, keepdim=True)
        want = torch.round(127 * wide / torch.where(peak == 0, 1.0, peak))
        assert torch.equal(q[s, :H].double(), want) and not q[s, H:].any()
        assert bool(((scales[s].double() - peak[:, 0] / 127).abs() <= 2.0 ** -24 * peak[:, 0] / 127).all())


# ------------------------------------------------------------------------------------
# the torch layer with more rows than kept choices
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("count_first,apart", [(True, 0), (False, 0), (False, 1 << 40)])
def test_layer_with_rows_of_no_choice(count_first, apart, monkeypatch):
    from lossless_bf16_exponent_codec_amd import moe
    monkeypatch.setattr(moe, "CLEAR_APART", apart)
    T, K, E, H, rows = 50, 2, 4, 96, 130
    g = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(K).indices
    ids[5], ids[9, 1] = -1, -1
    routing = moe.route(ids, E)
    if count_first:
        assert routing.splits()[-1] == 97
    x, f, w, dout = (torch.randn(*s, generator=g, device="cuda") for s in ((T, H), (H, H), (T, K), (T, H)))
    leaves = [t.requires_grad_() for t in (x, f, w)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    del_me = torch.full((rows, H), float("nan"), device="cuda")   # memory that the layer's buffers may be made of
    del del_me
    y = moe.dispatch(x, routing, rows, status)
    assert not y[97:].any()
    out = moe.combine(y @ f, routing, w, status)
    got = torch.autograd.grad(out, leaves, dout)
    wide = [t.detach().double().cpu().requires_grad_() for t in leaves]
    kept = (ids >= 0).double().cpu()
    ref = ((wide[2] * kept).sum(1, keepdim=True)) * (wide[0] @ wide[1])
    want = torch.autograd.grad(ref, wide, dout.double().cpu())
    # sums of fewer than 200 terms, two in a row, doubled for the library's products, relative to the largest value
    for a, b in zip((out.detach(), *got), (ref.detach(), *want)):
        assert float((a.double().cpu() - b).abs().max()) <= 4 * 200 * 2.0 ** -23 * float(b.abs().max())
    assert int(status.item()) == 0
