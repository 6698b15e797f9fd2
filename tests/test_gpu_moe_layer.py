"""The torch layer over the mixture-of-experts calls, and the example that runs them with the
codec, against plain torch in 64 bits."""
import os
import runpy

import pytest
import torch

pytestmark = pytest.mark.gpu

EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_exchange.py")


@pytest.fixture(scope="module")
def moe():
    from lossless_bf16_exponent_codec_amd import moe
    return moe


def plain_layer(x, ids, weights, f):
    """sum over k of weights * f_e(x), in 64 bits; f: list of per-expert matrices."""
    out = torch.zeros_like(x)
    for k in range(ids.shape[1]):
        for e in range(len(f)):
            m = (ids[:, k] == e).unsqueeze(1)
            out = out + torch.where(m, weights[:, k:k + 1] * (x @ f[e]), torch.zeros_like(x))
    return out


def test_gradients_through_experts(moe):
    # a layer of dense fp32 experts: the gradients of x, of the router's weights and of the
    # experts against autograd in 64 bits.  Every sum here has fewer than 200 terms, so
    # relative to the largest value 200 * 2^-23 bounds its rounding (twice: two sums in a
    # row), doubled again for the library's products.
    g = torch.Generator(device="cuda").manual_seed(1)
    T, K, E, H = 70, 2, 5, 36
    x, f = torch.randn(T, H, generator=g, device="cuda"), torch.randn(E, H, H, generator=g, device="cuda") * 0.2
    ids = torch.rand(T, E, generator=g, device="cuda").topk(K).indices
    ids[3] = -1
    ids[5, 1] = -1
    w, dout = torch.rand(T, K, generator=g, device="cuda"), torch.randn(T, H, generator=g, device="cuda")
    leaves = [t.clone().requires_grad_() for t in (x, w, f)]
    routing = moe.route(ids, E)
    ends = routing.splits()
    y = moe.dispatch(leaves[0], routing, ends[-1])
    y = torch.cat([y[ends[e]:ends[e + 1]] @ leaves[2][e] for e in range(E)])
    out = moe.combine(y, routing, leaves[1])
    got = [out.detach(), *torch.autograd.grad(out, leaves, dout)]
    wide = [t.double().cpu().requires_grad_() for t in (x, w, f)]
    ref = plain_layer(wide[0], ids.cpu(), wide[1], [wide[2][e] for e in range(E)])
    want = [ref.detach(), *torch.autograd.grad(ref, wide, dout.double().cpu())]
    for a, b in zip(got, want):
        assert float((a.double().cpu() - b).abs().max()) <= 4 * 200 * 2.0 ** -23 * float(b.abs().max())
    assert not got[1][3].any() and not got[2][3].any() and float(got[2][5, 1]) == 0


def test_expanded_gradient(moe):
    # sum().backward() hands an expanded tensor down
    x = torch.randn(9, 40, device="cuda").requires_grad_()
    routing = moe.route(torch.arange(18, device="cuda").view(9, 2) % 4, 4)
    moe.dispatch(x, routing, 18).sum().backward()
    assert bool((x.grad == 2).all())
    y, w = torch.randn(18, 40, device="cuda").requires_grad_(), torch.rand(9, 2, device="cuda").requires_grad_()
    moe.combine(y, routing, w).sum().backward()
    assert torch.equal(y.grad[routing.slots.view(-1).long()], w.detach().reshape(-1, 1).expand(18, 40))


def test_quantized_experts(moe):
    # against the dequantised product in 64 bits: one BF16 rounding (2^-8) of the result
    # and a few fp32 ones
    g = torch.Generator(device="cuda").manual_seed(2)
    T, K, E, H, N = 90, 2, 6, 300, 110
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    experts = moe.QuantizedExperts(torch.randn(E, N, H, generator=g, device="cuda").bfloat16())
    routing = moe.route(torch.rand(T, E, generator=g, device="cuda").topk(K).indices, E)
    ends = routing.splits()
    rows = moe.quantize(x, routing.slots, ends[-1])
    got = experts(rows, routing)
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        want = (rows.q[a:b, :H].double() @ experts.q[e, :, :H].double().T) * rows.scales[a:b, None].double() * \
            experts.scales[e].double()
        assert bool(((got[a:b].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -21) * want.abs()).all())
    # and the quantisation itself: half a step of either factor, summed over the row
    exact = x.double()[routing.rows[:ends[-1]].long()]
    assert bool(((rows.q[:, :H].double() * rows.scales[:, None].double() - exact).abs()
                 <= 0.5001 * rows.scales[:, None].double()).all())


@pytest.mark.parametrize("sizes", [dict(), dict(tokens=300, hidden=520, inner=136, experts=5, top_k=3, ranks=2)])
def test_example(sizes):
    s = runpy.run_path(EXAMPLE)["step"](**sizes)
    assert s["status"] == 0 and 1.3 < s["ratio"] < 1.5
    x, routing, M = s["x"], s["routing"], s["ends"][-1]
    rows, slots = routing.rows[:M].long(), routing.slots.long()
    # both exchanges give back what was sent, bit for bit
    assert torch.equal(s["sent"].view(torch.int16), x[rows].view(torch.int16))
    assert torch.equal(s["back"].view(torch.int16), s["made"].view(torch.int16))
    # combine and the gradients: one BF16 rounding each, and an fp32 sum of top_k terms
    K = slots.shape[1]
    y, w, dout = s["back"].double(), s["weights"].double(), s["dout"].double()

    def near(got, want, size):
        return bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + K * 2.0 ** -23 * size).all())

    terms = w.unsqueeze(-1) * y[slots]
    assert near(s["out"], terms.sum(1), terms.abs().sum(1))
    want = torch.empty_like(y)
    want[slots.view(-1)] = (w.unsqueeze(-1) * dout.unsqueeze(1)).view(-1, y.shape[1])
    assert near(s["dy"], want, want.abs())
    dots = dout.unsqueeze(1) * y[slots]
    assert bool(((s["dw"].double() - dots.sum(-1)).abs() <= y.shape[1] * 2.0 ** -23 * dots.abs().sum(-1)).all())
    back = s["dy"].double()[slots]
    assert near(s["dx"], back.sum(1), back.abs().sum(1))
