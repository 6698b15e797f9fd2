"""The router past what one grid of its kernels takes at once."""
import pytest
import torch

from tests.test_gpu_router import Z  # noqa: F401  (Z: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renormalize", [True, False])
def test_more_tokens_than_a_grid(Z, renormalize):
    # 2^20 workgroups of 4 tokens take 2^22 of them; a token's results are those of a call on fewer
    T, K, E, part = (1 << 22) + 4099, 3, 257, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.randn(T, E, generator=g, device="cuda", dtype=torch.bfloat16)
    mask = torch.rand(T, generator=g, device="cuda") < 0.9
    dw = torch.randn(T, K, generator=g, device="cuda")
    counts = torch.randint(0, 50000, (E + 1,), generator=g, device="cuda", dtype=torch.int32)
    dl = torch.full((1,), 1e4, device="cuda")
    ids, w = torch.full((T, K), -9, dtype=torch.int32, device="cuda"), torch.full((T, K), 7.0, device="cuda")
    d = torch.full((T, E), 7.0, device="cuda", dtype=torch.bfloat16)
    Z.moe_gate(logits, ids, w, renormalize=renormalize, mask=mask)
    Z.moe_gate_backward(logits, ids, d, dweights=dw, counts=counts, dloss=dl, renormalize=renormalize, mask=mask)
    for a in range(0, T, part):
        at = slice(a, min(T, a + part))
        i, v, e = torch.empty_like(ids[at]), torch.empty_like(w[at]), torch.empty_like(d[at])
        Z.moe_gate(logits[at], i, v, renormalize=renormalize, mask=mask[at])
        Z.moe_gate_backward(logits[at], i, e, dweights=dw[at], counts=counts, dloss=dl, renormalize=renormalize,
                            mask=mask[at])
        assert torch.equal(i, ids[at]) and torch.equal(v, w[at]) and torch.equal(e, d[at])
