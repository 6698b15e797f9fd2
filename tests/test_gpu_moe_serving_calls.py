"""A served layer through the torch calls: captured and replayed, and with no tokens at all."""
import pytest
import torch

from tests.test_gpu_experts4 import moe  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def layer(moe, x, logits, up, down, K, mask=None):
    router = moe.gate(logits, K, mask=mask, balance=True)
    routing = moe.route(router.experts, logits.shape[1])
    inside = torch.nn.functional.silu(up(x, routing))
    out = moe.combine(down(inside, routing, by_expert=True), routing, router.weights)
    return router.experts, router.weights, router.loss, router.counts, out


def experts(moe, E, H, F, g):
    return (moe.QuantizedExperts4(torch.randn(E, F, H, generator=g, device="cuda").mul_(H ** -0.5).bfloat16()),
            moe.QuantizedExperts4(torch.randn(E, H, F, generator=g, device="cuda").mul_(F ** -0.5).bfloat16(), group=64))


def test_captured_and_replayed(moe):
    # two graphs of the same layer, replayed in turn with eager calls between
    g = torch.Generator(device="cuda").manual_seed(1)
    T, K, E, H, F = 12, 2, 40, 192, 130
    up, down = experts(moe, E, H, F, g)
    inputs = [(torch.randn(T, H, generator=g, device="cuda").bfloat16(), torch.randn(T, E, generator=g, device="cuda"),
               torch.rand(T, generator=g, device="cuda") < 0.8) for _ in range(2)]
    layer(moe, *inputs[0][:2], up, down, K, inputs[0][2])
    torch.cuda.synchronize()
    graphs, made = [], []
    for x, logits, mask in inputs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            made.append(layer(moe, x, logits, up, down, K, mask))
    for _ in range(4):
        for x, logits, mask in inputs:
            x.copy_(torch.randn(T, H, generator=g, device="cuda"))
            logits.copy_(torch.randn(T, E, generator=g, device="cuda"))
            mask.copy_(torch.rand(T, generator=g, device="cuda") < 0.8)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (x, logits, mask), got in zip(inputs, made):
            want = layer(moe, x, logits, up, down, K, mask)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_tokens(moe):
    g = torch.Generator(device="cuda").manual_seed(2)
    E, H, F, K = 6, 64, 48, 2
    up, down = experts(moe, E, H, F, g)
    logits = torch.empty(0, E, device="cuda", requires_grad=True)
    ids, w, loss, counts, out = layer(moe, torch.empty(0, H, dtype=torch.bfloat16, device="cuda"), logits, up, down, K)
    assert ids.shape == w.shape == (0, K) and out.shape == (0, H) and float(loss.detach()) == 0.0 and not counts.any()
    grad, = torch.autograd.grad(loss + w.sum(), logits)
    assert grad.shape == (0, E)


def test_tokens_that_are_all_padding(moe):
    g = torch.Generator(device="cuda").manual_seed(3)
    T, E, H, F, K = 9, 6, 64, 48, 2
    up, down = experts(moe, E, H, F, g)
    logits = torch.full((T, E), float("nan"), device="cuda", requires_grad=True)
    x = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    ids, w, loss, counts, out = layer(moe, x, logits, up, down, K, torch.zeros(T, dtype=torch.bool, device="cuda"))
    assert bool((ids == -1).all()) and not w.any() and float(loss.detach()) == 0.0 and not counts.any() and not out.any()
    grad, = torch.autograd.grad(loss + w.sum(), logits)
    assert not grad.any() and not grad.isnan().any()
