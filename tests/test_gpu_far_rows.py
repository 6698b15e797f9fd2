"""The router's rows, 4-bit products' rows and experts' weights that lie past 4 GB from their
tensors' starts: results are those of the same values close together."""
import pytest
import torch

from tests.test_gpu_experts4 import Z, moe  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

FAR = 1 << 21       # values from row to row: 1100 rows are past 2^31 values, in BF16 past 4 GB


def far(values):
    """The same rows, FAR values apart in memory that holds NaNs beside the last ones."""
    rows, length = values.shape
    space = torch.empty(rows * FAR, dtype=values.dtype, device="cuda").view(rows, FAR)
    space[:, :length + 64] = float("nan")
    view = space[:, :length]
    view.copy_(values)
    return view


@pytest.mark.parametrize("T,K,E", [(1100, 3, 61), (1100, 8, 256), (1100, 4, 300)])
def test_logits(Z, T, K, E):
    g = torch.Generator(device="cuda").manual_seed(E)
    z = torch.randn(T, E, generator=g, device="cuda").bfloat16()
    dw, dl = torch.randn(T, K, generator=g, device="cuda"), torch.full((1,), 50.0, device="cuda")
    made = []
    for x, d in ((z, torch.empty_like(z)), (far(z), far(torch.zeros_like(z)))):
        ids, w = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
        counts, sums = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(E, device="cuda")
        loss, space = torch.empty(1, device="cuda"), torch.empty(Z.MOE_GATE_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
        Z.moe_gate(x, ids, w, counts=counts, sums=sums, loss=loss, workspace=space)
        Z.moe_gate_backward(x, ids, d, dweights=dw, counts=counts, dloss=dl)
        made.append((ids, w, counts, sums, loss, d))
    assert all(torch.equal(a, b) for a, b in zip(*made))


def test_given_choices(Z):
    T, K, E = 1100, 2, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn(T, E, generator=g, device="cuda")
    ids = torch.randint(-1, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    space = torch.zeros(T * FAR, dtype=torch.int32, device="cuda").view(T, FAR)[:, :K]
    space.copy_(ids)
    made = []
    for choices in (ids, space):
        counts, sums = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(E, device="cuda")
        loss, d = torch.empty(1, device="cuda"), torch.empty_like(z)
        Z.moe_balance(z, choices, counts, sums, loss, torch.empty(Z.MOE_GATE_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda"))
        Z.moe_gate_backward(z, choices, d, dweights=torch.ones(T, K, device="cuda"), counts=counts, dloss=loss,
                            renormalize=False)
        made.append((counts, sums, loss, d))
    assert all(torch.equal(a, b) for a, b in zip(*made))


# streamed, and in tiles of 64 rows by 64 outputs (aligned rows, which go straight to LDS)
@pytest.mark.parametrize("M,E,N,H", [(1100, 300, 50, 200), (1100, 3, 1400, 256)])
def test_rows_of_a_product(Z, moe, M, E, N, H):
    g = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn(M, H, generator=g, device="cuda").bfloat16()
    q = moe.pack4(torch.randint(-8, 8, (E, N, H), generator=g, device="cuda", dtype=torch.int8))
    s = torch.rand(E, -(-H // 64), N, generator=g, device="cuda")
    offsets = torch.linspace(0, M, E + 1, device="cuda").to(torch.int32)
    rows = torch.randint(0, M, (M,), generator=g, device="cuda", dtype=torch.int32)
    rows[-1] = M - 1
    close, wide = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), far(torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"))
    Z.experts_product4(x, q, s, 64, close, rows=rows, offsets=offsets)
    Z.experts_product4(far(x), q, s, 64, wide, rows=rows, offsets=offsets)
    assert torch.equal(close, wide)


def test_weights_of_many_experts(Z):
    # 1024 experts' weights are 4.3 GB: the last ones' products against the same experts alone
    E, N, H, group = 1024, 2048, 4096, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    size = Z.weights4_size(1, N, H)
    q = torch.zeros(E, size, dtype=torch.uint8, device="cuda")
    q[-3:] = torch.randint(0, 256, (3, size), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.rand(E, H // group, N, generator=g, device="cuda").bfloat16()
    M = 24
    x = torch.randn(M, H, generator=g, device="cuda").bfloat16()
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[-3:] = torch.tensor([10, 11, M], dtype=torch.int32)
    got, want = (torch.zeros(M, N, device="cuda") for _ in range(2))
    Z.experts_product4(x, q, s, group, got, offsets=offsets)
    # the same three experts as rows of a call that has no others
    few = torch.tensor([0, 10, 11, M], dtype=torch.int32, device="cuda")
    Z.experts_product4(x, q[-3:].contiguous(), s[-3:].contiguous(), group, want, offsets=few)
    # (other kernels may add in another order: H 2^-23 of the magnitudes, twice)
    bound = 2 * H * 2.0 ** -23 * x.abs().float().sum(1, keepdim=True) * 8
    assert bool(((got - want).abs() <= bound).all()) and bool((got.abs().amax(1) > 0).all())


def test_quantised_rows_of_weights(Z):
    N, H, group = 1100, 300, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    made = []
    for x in (w, far(w)):
        q = torch.empty(Z.weights4_size(1, N, H), dtype=torch.uint8, device="cuda")
        s = torch.empty(1, -(-H // group), N, device="cuda")
        Z.quantize_weights4(x, group, q, s)
        made.append((q, s))
    assert all(torch.equal(a, b) for a, b in zip(*made))
