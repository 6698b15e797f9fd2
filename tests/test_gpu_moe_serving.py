"""A layer in serving, step by step: the router's choices and weights, both products with 4-bit
experts and the combine, each against 64 bits from the step's own inputs.  Tolerances as in the
operators' own tests."""
import numpy as np
import pytest
import torch

from tests import router_reference as R
from tests.test_gpu_experts4 import host, moe  # noqa: F401  (moe: a fixture)
from tests.test_gpu_router import TINY, delta

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,E,H,F", [(1, 2, 4, 200, 72), (5, 3, 8, 256, 144), (90, 4, 6, 384, 300)])
def test_every_step(moe, T, K, E, H, F):
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    logits = torch.randn(T, E, generator=g, device="cuda")
    up = moe.QuantizedExperts4(torch.randn(E, F, H, generator=g, device="cuda").mul_(H ** -0.5).bfloat16())
    down = moe.QuantizedExperts4(torch.randn(E, H, F, generator=g, device="cuda").mul_(F ** -0.5).bfloat16(), group=32,
                                 scale_dtype=torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    router = moe.gate(logits, K, status=status)
    routing = moe.route(router.experts, E, status)
    first = up(x, routing, status=status)
    inside = torch.nn.functional.silu(first)
    made = down(inside, routing, by_expert=True, status=status)
    out = moe.combine(made, routing, router.weights, status)
    assert int(status.item()) == 0

    z = host(logits)
    ids = R.choices(z, None, K)
    assert np.array_equal(router.experts.cpu().numpy(), ids)
    w = R.weights(z, None, ids, True)
    assert np.all(np.abs(host(router.weights) - w) <= 2 * delta(z, R.counted(z, None)) * w + TINY)
    ends, rows = routing.splits(), routing.rows.cpu().numpy()
    assert ends[-1] == T * K == first.shape[0]
    for e in range(E):      # the tokens that chose an expert, in order
        assert rows[ends[e]:ends[e + 1]].tolist() == [t for t in range(T) for k in range(K) if ids[t, k] == e]
    for source, index, experts, got in ((x, rows, up, first), (inside, np.arange(T * K), down, made)):
        values, clean = R.unpack4(experts.q.cpu().numpy(), E, experts.outputs, experts.inputs)
        want, size = R.product4(host(source), index, values, host(experts.scales), experts.group, ends)
        tol = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * experts.inputs * 2.0 ** -23 * size
        assert clean and np.all(np.abs(host(got) - want) <= tol)
    slots = routing.slots.cpu().numpy()
    assert np.array_equal(np.sort(slots.reshape(-1)), np.arange(T * K))
    terms = host(router.weights)[:, :, None] * host(made)[slots]
    assert np.all(np.abs(host(out) - terms.sum(1)) <= 2.0 ** -8 * np.abs(terms.sum(1)) + K * 2.0 ** -23 * np.abs(terms).sum(1))
