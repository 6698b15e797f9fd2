"""The binding of the router's calls and of those with 4-bit weights: whose memory it passes
on, and where a call goes.  The library's calls are recorded, not made; no call here reaches
a GPU."""
import pytest
import torch

from tests.test_moe_binding import Elsewhere, Placed, Stream, placed, zeros

BF, I32 = torch.bfloat16, torch.int32
T, K, E, H, N, M = 6, 2, 3, 40, 7, 12
LOGITS, CHOICES, WEIGHTS, MASK = zeros(T, E), zeros(T, K, dtype=I32), zeros(T, K), zeros(T, dtype=torch.bool)
COUNTS, SUMS, ONE, SPACE = zeros(E + 1, dtype=I32), zeros(E), zeros(1), zeros(300, dtype=torch.uint8)
ALL = {
    "moe_gate": (lambda Z, a, **kw: Z.moe_gate(*a[:3], mask=a[3], counts=a[4], sums=a[5], loss=a[6], workspace=a[7], **kw),
                 [LOGITS, CHOICES, WEIGHTS, MASK, COUNTS, SUMS, ONE, SPACE]),
    "moe_balance": (lambda Z, a, **kw: Z.moe_balance(*a[:6], mask=a[6], **kw),
                    [LOGITS, CHOICES, COUNTS, SUMS, ONE, SPACE, MASK]),
    "moe_gate_backward": (lambda Z, a, **kw: Z.moe_gate_backward(*a[:6], mask=a[6], **kw),
                          [LOGITS, CHOICES, LOGITS, WEIGHTS, COUNTS, ONE, MASK]),
    "quantize_weights4": (lambda Z, a, **kw: Z.quantize_weights4(a[0], 32, *a[1:], **kw),
                          [zeros(E, N, H, dtype=BF), zeros(E * 1024, dtype=torch.uint8), zeros(E, 2, N)]),
    "experts_product4": (lambda Z, a, **kw: Z.experts_product4(*a[:3], 32, *a[3:], **kw),
                         [zeros(T, H, dtype=BF), zeros(E * 1024, dtype=torch.uint8), zeros(E, 2, N), zeros(M, N),
                          zeros(M, dtype=I32), zeros(E + 1, dtype=I32)]),
}
WITH_STATUS = [name for name in ALL if name != "quantize_weights4"]


@pytest.fixture
def Z(monkeypatch):
    """The binding with its library's calls recorded in Z.calls: (name, arguments,
    current GPU)."""
    from lossless_bf16_exponent_codec_amd import zipccl
    calls, current = [], [0]
    for name in ALL:
        def record(*args, name=name):
            calls.append((name, args, current[-1]))
            return zipccl.OK
        monkeypatch.setattr(zipccl.lib(), "zipccl_" + name, record)

    class On:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *_):
            current.pop()

    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(zipccl, "_current_device", lambda: current[-1])
    monkeypatch.setattr(zipccl, "_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(zipccl, "calls", calls, raising=False)
    return zipccl


@pytest.mark.parametrize("name", ALL)
def test_tensors_of_the_host_or_of_two_gpus_are_refused(Z, name):
    call, makers = ALL[name]
    for place in torch.Tensor, Elsewhere:
        for i in range(len(makers)):
            with pytest.raises(ValueError, match="one GPU"):
                call(Z, [placed(m(), place if j == i else Placed) for j, m in enumerate(makers)])
    with pytest.raises(ValueError, match="one GPU"):
        call(Z, [m() for m in makers])
    if name in WITH_STATUS:
        for status in torch.zeros(1, dtype=I32), placed(torch.zeros(1, dtype=I32), Elsewhere), \
                placed(torch.zeros(1, dtype=torch.int16)):
            with pytest.raises(ValueError):
                call(Z, [placed(m()) for m in makers], status=status)
    assert not Z.calls


@pytest.mark.parametrize("name", ALL)
def test_calls_go_to_the_gpu_that_holds_the_tensors(Z, name):
    call, makers = ALL[name]
    for device, place in enumerate((Placed, Elsewhere)):
        tensors = [placed(m(), place) for m in makers]
        call(Z, tensors)
        call(Z, tensors, stream=Stream(device))
        call(Z, tensors, stream=99)
        with pytest.raises(ValueError, match="stream"):
            call(Z, tensors, stream=Stream(1 - device))
        assert [(args[-1], where) for _, args, where in Z.calls] == [(1000 + device, device), (77, device), (99, device)]
        if name in WITH_STATUS:
            status = placed(torch.zeros(1, dtype=I32), place)
            call(Z, tensors, status=status)
            assert Z.calls.pop()[1][-2] == status.data_ptr()
            assert all(args[-2] is None for _, args, _ in Z.calls)
        Z.calls.clear()


def test_workspaces_and_vectors_are_their_own_memory(Z):
    call, makers = ALL["moe_gate"]
    t = [placed(m()) for m in makers]
    with pytest.raises(ValueError, match="workspace"):
        call(Z, t[:7] + [placed(torch.zeros(1, dtype=torch.uint8)).expand(300)])
    with pytest.raises(ValueError, match="mask"):
        call(Z, t[:3] + [placed(torch.zeros(1, dtype=torch.bool)).expand(T)] + t[4:])
    with pytest.raises(ValueError, match="experts"):
        call(Z, [t[0], placed(torch.zeros(1, K, dtype=I32)).expand(T, K)] + t[2:])
    call, makers = ALL["experts_product4"]
    t = [placed(m()) for m in makers]
    with pytest.raises(ValueError, match="q is"):
        call(Z, [t[0], placed(torch.zeros(1, dtype=torch.uint8)).expand(E * 1024)] + t[2:])
    assert not Z.calls


def test_weights_of_experts_one_after_another(Z):
    w = placed(torch.zeros(E, N, 64, dtype=BF))
    q, s = placed(torch.zeros(E * 1024, dtype=torch.uint8)), placed(torch.zeros(E, 2, N))
    Z.quantize_weights4(w[:, :, :H], 32, q, s)
    assert Z.calls.pop()[1][1:6] == (64, E, N, H, 32)
    Z.quantize_weights4(placed(torch.zeros(E, 5, H, dtype=BF))[:, :1], 32, q, placed(torch.zeros(E, 2, 1)))
    assert Z.calls.pop()[1][1:6] == (5 * H, E, 1, H, 32)
    for bad in (w[:, :5, :H], w[:, :, :H].transpose(0, 1), w.transpose(1, 2)):
        with pytest.raises(ValueError):
            Z.quantize_weights4(bad, 32, q, placed(torch.zeros(bad.shape[0], -(-bad.shape[2] // 32), bad.shape[1])))
    assert not Z.calls
