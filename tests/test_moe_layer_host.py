"""The torch layer of the mixture-of-experts calls on the CPU: the calls themselves are
stand-ins in plain torch, so that what is tested is the layer's buffers, gradients and
refusals."""
import pytest
import torch


def picked(rows, slots):
    kept = ((slots >= 0) & (slots < rows.shape[0])).unsqueeze(-1)
    return torch.where(kept, rows[slots.clamp(0, max(rows.shape[0] - 1, 0)).long()], torch.zeros(()))


def sort(experts, num_experts, offsets, rows, slots, workspace, status=None):
    flat = torch.where(experts < 0, num_experts, experts).reshape(-1)
    order = torch.sort(flat, stable=True)
    offsets.copy_(torch.searchsorted(order.values, torch.arange(num_experts + 1)))
    rows.copy_(torch.where(order.values < num_experts, order.indices // experts.shape[1], -1))
    place = torch.empty_like(flat)
    place[order.indices] = torch.arange(flat.numel())
    slots.copy_(torch.where(flat < num_experts, place, -1).view(experts.shape))


def dispatch(x, slots, y, status=None):
    for t, k in (slots >= 0).nonzero().tolist():
        if slots[t, k] < y.shape[0]:
            y[slots[t, k]] = x[t]
        elif status is not None:
            status |= 4


def combine(y, slots, weights, out, status=None):
    w = torch.ones(slots.shape) if weights is None else weights.reshape(slots.shape)
    out.copy_((w.unsqueeze(-1) * picked(y, slots)).sum(1))
    if status is not None and bool((slots >= y.shape[0]).any()):
        status |= 4


def combine_backward(dout, y, slots, weights, dy, dweights, status=None):
    weights = weights.reshape(slots.shape)
    dweights.copy_((dout.unsqueeze(1) * picked(y, slots)).sum(-1).view(dweights.shape))
    for t, k in (slots >= 0).nonzero().tolist():
        if slots[t, k] < y.shape[0]:
            dy[slots[t, k]] = weights[t, k] * dout[t]
        elif status is not None:
            status |= 4


@pytest.fixture
def moe(monkeypatch):
    from lossless_bf16_exponent_codec_amd import moe

    def dispatch_backward(dy, slots, dx, status=None):
        combine(dy, slots, None, dx, status)

    for name, plain in dict(moe_sort=sort, moe_dispatch=dispatch, moe_dispatch_backward=dispatch_backward,
                            moe_combine=combine, moe_combine_backward=combine_backward).items():
        monkeypatch.setattr(moe.Z, name, torch.no_grad()(plain))   # autograd does not see what a kernel writes
    return moe


IDS = torch.tensor([[0, 2], [1, -1], [2, 0]])


def test_second_order_gradients_are_an_error_not_zero(moe):
    # the gradients are written by kernels that autograd does not see: differentiating them
    # again has to fail, not to drop the terms
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 4, generator=g, requires_grad=True)
    w = torch.rand(3, 2, generator=g, requires_grad=True)
    routing = moe.route(IDS, 3)
    M = routing.splits()[-1]
    y = moe.dispatch(x, routing, M)
    dx, = torch.autograd.grad((y ** 2).sum(), x, create_graph=True)
    assert torch.equal(dx.detach(), 2 * x.detach() * torch.tensor([[2.0], [1.0], [2.0]]))
    with pytest.raises(RuntimeError, match="twice"):
        (dx ** 2).sum().backward()
    rows = torch.randn(M, 4, generator=g, requires_grad=True)
    out = moe.combine(rows, routing, w)
    for leaf in rows, w:
        grad, = torch.autograd.grad((out ** 2).sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="twice"):
            (out.sum() + (grad ** 2).sum()).backward(retain_graph=True)


def test_products_of_rows_of_another_length_are_refused(moe, monkeypatch):
    asked = []
    monkeypatch.setattr(moe.Z, "quantize_rows", lambda *a, **kw: None)
    monkeypatch.setattr(moe.Z, "experts_product", lambda *a, **kw: asked.append(a))
    experts = moe.QuantizedExperts(torch.zeros(3, 5, 250, dtype=torch.bfloat16))
    routing = moe.route(IDS, 3)
    for length in 200, 249, 256, 1000:
        with pytest.raises(ValueError, match="250"):
            experts(moe.quantize(torch.zeros(5, length, dtype=torch.bfloat16)), routing)
    assert not asked
    experts(moe.quantize(torch.zeros(5, 250, dtype=torch.bfloat16)), routing)
    assert len(asked) == 1


def test_products_with_offsets_of_other_experts_are_refused(moe, monkeypatch):
    # with more offsets than experts the rows of the others would be memory as it was found
    asked = []
    monkeypatch.setattr(moe.Z, "quantize_rows", lambda *a, **kw: None)
    monkeypatch.setattr(moe.Z, "experts_product", lambda *a, **kw: asked.append(a))
    experts = moe.QuantizedExperts(torch.zeros(3, 5, 250, dtype=torch.bfloat16))
    rows = moe.quantize(torch.zeros(5, 250, dtype=torch.bfloat16))
    for other in 2, 4:
        with pytest.raises(ValueError, match="experts"):
            experts(rows, moe.route(IDS.clamp(max=1), other))
    assert not asked
    experts(rows, moe.route(IDS, 3))
    assert len(asked) == 1


@pytest.fixture
def poison():
    """Memory that is not written holds NaN (whole numbers: their largest)."""
    torch.use_deterministic_algorithms(True)
    yield
    torch.use_deterministic_algorithms(False)


@pytest.mark.parametrize("apart", [0, 1 << 40])
def test_rows_of_no_choice_are_zero(moe, poison, monkeypatch, apart):
    # 5 kept choices in a buffer of 8 rows, with the kept count on the host and without: the
    # rows past them are read by a dense expert and by its weights' gradient
    g = torch.Generator().manual_seed(3)
    x, f = torch.randn(3, 4, generator=g), torch.randn(4, 4, generator=g)
    assert bool(torch.empty(3).isnan().all())
    monkeypatch.setattr(moe, "CLEAR_APART", apart)
    for count_first in True, False:
        routing = moe.route(IDS, 3)
        if count_first:
            assert routing.splits() == [0, 2, 3, 5]
        xs, fs = x.clone().requires_grad_(), f.clone().requires_grad_()
        y = moe.dispatch(xs, routing, 8)
        assert not y[5:].any() and torch.equal(y[:5], x[[0, 2, 1, 0, 2]])
        out = moe.combine(y @ fs, routing, torch.ones(3, 2))
        out.sum().backward()
        kept = torch.tensor([[2.0], [1.0], [2.0]])
        torch.testing.assert_close(fs.grad, (kept * x).sum(0).unsqueeze(1).expand(4, 4))
        torch.testing.assert_close(xs.grad, kept * f.sum(1))
        # no rows past the kept ones: nothing to clear
        assert torch.equal(moe.dispatch(x, routing, 5), x[[0, 2, 1, 0, 2]])


def test_status_word_of_each_call(moe, monkeypatch):
    # slots past the rows are dropped; the caller's status word says so, forward and backward
    for name in "quantize_rows", "experts_product":
        monkeypatch.setattr(moe.Z, name, lambda *a, status=None, **kw: status is None or status.fill_(64))
    routing = moe.route(IDS, 3)
    x = torch.zeros(3, 4, requires_grad=True)
    status = torch.zeros(1, dtype=torch.int32)
    y = moe.dispatch(x, routing, 4, status)
    assert int(status) == 4
    status.zero_()
    y.sum().backward()
    assert int(status) == 4
    rows = torch.zeros(4, 4, requires_grad=True)
    status.zero_()
    out = moe.combine(rows, routing, torch.ones(3, 2), status)
    assert int(status) == 4
    status.zero_()
    out.sum().backward()
    assert int(status) == 4
    moe.quantize(torch.zeros(3, 250, dtype=torch.bfloat16), routing.slots, 4, status)
    assert int(status) == 64
    status.zero_()
    status.zero_()
    experts = moe.QuantizedExperts(torch.zeros(3, 5, 250, dtype=torch.bfloat16))
    experts(moe.QuantizedRows(torch.zeros(4, 256, dtype=torch.int8), torch.zeros(4), 250), routing, status=status)
    assert int(status) == 64


def test_weights_of_other_choices_are_refused(moe):
    # a weight for each choice; more would be read at the wrong places, and their gradients
    # would be memory as it was found
    routing = moe.route(IDS, 3)
    rows = torch.randn(5, 4)
    want = moe.combine(rows, routing, torch.arange(6.0).view(3, 2))
    for shape in (6,), (6, 1), (1, 6), (3, 2, 1):
        assert torch.equal(moe.combine(rows, routing, torch.arange(6.0).view(shape)), want)
    for shape in (3, 3), (2, 3), (4, 2), (7,), (3, 1), (5,):
        with pytest.raises(ValueError, match="weights"):
            moe.combine(rows, routing, torch.ones(shape))
