"""The product with 4-bit weights in every kernel that its rule picks: rows long enough for each
wave's steady loop, and rows that end where the last slab's groups do not.

Tolerances as in test_gpu_experts4: an fp32 sum over H inputs is off by at most H * 2^-23 of the sum
of its terms' magnitudes, the result by half a step of its type; whole numbers with scales that are
powers of two give exact sums and are compared for equality."""
import numpy as np
import pytest
import torch

from tests import product4_shapes as S
from tests.test_gpu_experts4 import POISON, Z, check, host, make, moe, spread  # noqa: F401  (Z, moe: fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale_dtype,dtype", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("T,M,E,N,H,group", S.STREAMED)
def test_long_streamed_rows(Z, moe, T, M, E, N, H, group, dtype, scale_dtype):
    rng = np.random.default_rng(M + N + H)
    x, index, q, s, values = make(rng, moe, T, M, E, N, H, group, scale_dtype)
    check(Z, x, index, q, s, values, group, spread(rng, M, E), dtype)
    # exact: a term is at most 4 * 8 * 4 and a multiple of 1 / 4, so sums of 3300 are below 2^21 quarters
    x, index, q, s, values = make(rng, moe, T, M, E, N, H, group, scale_dtype, whole=True)
    check(Z, x, index, q, s, values, group, spread(rng, M, E), dtype, whole=True)


@pytest.mark.parametrize("scale_dtype,dtype", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("T,M,E,N,H,group", S.PART_SLABS)
def test_infinite_scale_of_a_part_slab(Z, moe, T, M, E, N, H, group, dtype, scale_dtype):
    # a last group whose scale is infinite: an infinity of its sum's sign, NaN where that is 0
    rng = np.random.default_rng(N + H)
    x, index, q, s, values = make(rng, moe, T, M, E, N, H, group, scale_dtype, whole=True)
    last = s.shape[1] - 1
    s[:, last, ::3] = float("inf")
    s[:, last, 1::3] = -float("inf")
    offsets = spread(rng, M, E)
    out = torch.full((M, N), POISON, dtype=dtype, device="cuda")
    Z.experts_product4(x, q, s, group, out, rows=index, offsets=torch.from_numpy(offsets).cuda())
    want = np.full((M, N), float(torch.tensor(POISON, dtype=dtype)))
    scales, rows = host(s), host(x)[index.cpu().numpy()]
    for e in range(E):
        at = slice(int(offsets[e]), int(offsets[e + 1]))
        want[at] = 0.0
        for g in range(last + 1):
            part = slice(g * group, min(H, (g + 1) * group))
            with np.errstate(invalid="ignore"):
                want[at] += (rows[at, part] @ values[e][:, part].T) * scales[e, g]
    want = torch.from_numpy(want).to(dtype).double().numpy()
    assert np.isposinf(want).any() and np.isneginf(want).any()
    assert np.array_equal(host(out), want, equal_nan=True)
