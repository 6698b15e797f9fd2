"""The router's probabilities and weights far below a row's largest logit, where an exponential
whose argument was rounded once more would be off by the rounding of a number of that size.

Logits are multiples of 2^-8 below 128 in size, so their differences are exact.  In units u = 2^-24,
an exponential at a distance of at most R is off by 2 u of its power of two (one place), u of the
correction's sum, and R / 20 u of the correction's constant: 4 + R / 20 with the terms of second order.
A quotient of one by a sum of them has twice that, the sum's steps and its own rounding: a lane
adds at most 16 (1 where there are at most 16 experts, or of choices), at most 6 steps join lanes."""
import numpy as np
import pytest
import torch

from tests import router_reference as R
from tests.test_gpu_router import TINY, U, Z, host, outputs, space  # noqa: F401  (Z: a fixture)

pytestmark = pytest.mark.gpu


def quotient(reach, added):
    return (2 * (4 + reach / 20) + (1 if added <= 16 else 16) + 6 + 1) * U


def far_logits(rng, T, E, near, far, dtype):
    """A largest logit for each token, the others from `near` to `far` below it."""
    z = rng.uniform(-far, -near, (T, E)).astype(np.float64)
    z[np.arange(T), rng.integers(0, E, T)] = 0.0
    z = np.round((z + rng.integers(0, 20, (T, 1))) * 256) / 256
    logits = torch.from_numpy(z).to(dtype).cuda()
    return logits, host(logits)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,E,far", [(400, 8, 8, 20), (400, 8, 8, 80), (300, 6, 40, 60), (300, 12, 300, 50)])
def test_weights_far_below_the_largest(Z, T, K, E, far, dtype):
    rng = np.random.default_rng(E + far)
    logits, z = far_logits(rng, T, E, 1, far, dtype)
    ids, w, *_ = outputs(T, K, E)
    for renormalize in (False, True):
        Z.moe_gate(logits, ids, w, renormalize=renormalize)
        want = R.choices(z, None, K)
        assert np.array_equal(ids.cpu().numpy(), want)
        ww = R.weights(z, None, want, renormalize)
        worst = (np.abs(host(w) - ww) / ww).max()
        assert worst <= quotient(far + 1, K if renormalize else E), worst / U


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,far", [(8, 20), (60, 60), (200, 70)])
def test_sums_far_below_the_largest(Z, E, far, dtype):
    # one token: the sums are its probabilities; and the gradient of one of them, held to their precision
    rng = np.random.default_rng(E)
    for _ in range(20):
        logits, z = far_logits(rng, 1, E, 1, far, dtype)
        ids, w, counts, sums, loss = outputs(1, 2, E)
        Z.moe_gate(logits, ids, w, counts=counts, sums=sums, loss=loss, workspace=space(Z))
        p = R.softmax(z[0])
        assert (np.abs(host(sums) - p) / p).max() <= quotient(far + 1, E) + U


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,E", [(300, 4, 20), (300, 8, 60), (200, 8, 250), (200, 20, 300)])
def test_gradient_of_choices_below_the_largest(Z, T, K, E, dtype):
    # choices 30 to 60 below the row's largest: the gradient's weights are as exact as the forward's.
    # w (dw - sum w dw): two factors of w in a term, and the roundings of its products, the sum's 6
    # steps and the difference
    rng = np.random.default_rng(E)
    logits, z = far_logits(rng, T, E, 30, 60, dtype)
    low = z < z.max(axis=1, keepdims=True)
    ids = np.stack([rng.permutation(np.flatnonzero(low[t]))[:K] for t in range(T)])
    dw = rng.standard_normal((T, K)).astype(np.float32)
    d = torch.empty(T, E, device="cuda")
    wide = logits.float()
    Z.moe_gate_backward(wide, torch.from_numpy(ids).cuda(), d, dweights=torch.from_numpy(dw).cuda())
    want, size = R.backward(z, None, ids, True, dw, None, None)
    tol = (2 * quotient(61, 1) + 12 * U) * size + TINY
    assert np.all(np.abs(host(d) - want) <= tol), (np.abs(host(d) - want) / np.maximum(size, 1e-30)).max() / U


@pytest.mark.parametrize("renormalize", [True, False])
def test_what_is_no_number_or_past_the_range(Z, renormalize):
    # an exponential of a distance past its range is 0 and of an infinite one too; NaNs stay
    inf, nan, top = float("inf"), float("nan"), torch.finfo(torch.float32).max
    z = torch.tensor([[0.0, -200.0, -inf, -1e38], [top, -top, 0.0, -inf], [-top, -inf, -top, -inf], [1.0, nan, -inf, 0.0],
                      [inf, 0.0, -inf, -top]], device="cuda")
    ids, w, counts, sums, loss = outputs(5, 4, 4)
    Z.moe_gate(z[:3], ids[:3], w[:3], renormalize=renormalize, counts=counts, sums=sums, loss=loss, workspace=space(Z))
    assert w[:3].tolist() == [[1.0, 0.0, 0.0, 0.0], [1.0, 0.0, 0.0, 0.0], [0.5, 0.5, 0.0, 0.0]]
    assert sums.tolist() == [2.5, 0.0, 0.5, 0.0]
    Z.moe_gate(z, ids, w, renormalize=renormalize)
    assert ids[3:].tolist() == [[1, 0, 3, -1], [0, 1, 3, -1]] and bool(w[3:, :3].isnan().all()) and not w[3:, 3].any()
    d, dw = torch.empty(5, 4, device="cuda"), torch.ones(5, 4, device="cuda")
    dw[:, 0] = 2.0
    Z.moe_gate_backward(z, ids, d, dweights=dw, renormalize=renormalize)
    assert d[:3].tolist() == [[0.0] * 4, [0.0] * 4, [0.25, 0.0, -0.25, 0.0]] and bool(d[3:].isnan().any(1).all())
