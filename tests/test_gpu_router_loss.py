"""The balance loss joined over many workgroups."""
import pytest
import torch

from tests.test_gpu_router import U, Z, outputs, space  # noqa: F401  (Z: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,E", [(3000, 4, 1024), (700, 2, 33), (5000, 8, 256)])
def test_loss_of_many_workgroups_on_every_call(Z, T, K, E):
    # the parts of the loss that workgroups hand to the last of them: all there on every call, in memory
    # that held NaNs, beside another call at work
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn(T, E, generator=g, device="cuda")
    other, ws, beside = torch.cuda.Stream(), space(Z), space(Z)
    made = []
    for _ in range(60):
        ws.fill_(0xFF)
        o, p = outputs(T, K, E), outputs(T, K, E)
        torch.cuda.synchronize()
        Z.moe_gate(logits, p[0], p[1], counts=p[2], sums=p[3], loss=p[4], workspace=beside, stream=other)
        Z.moe_gate(logits, o[0], o[1], counts=o[2], sums=o[3], loss=o[4], workspace=ws)
        torch.cuda.synchronize()
        made += [o, p]
    for o in made[1:]:
        assert all(torch.equal(x, y) for x, y in zip(o, made[0]))
    _, _, counts, sums, loss = made[0]
    n = int(counts[E])
    assert n == T
    want = E / (K * n * n) * float((counts[:E].double() * sums.double()).sum())
    assert abs(float(loss) - want) <= 2 * U * want      # of the sums' rounding, and the loss's
