"""The binding of the mixture-of-experts calls: which tensors it passes on, and which it
refuses before the library is called.  The library's calls are recorded, not made; no call
here reaches a GPU."""
import pytest
import torch

NAMES = ("moe_sort", "moe_dispatch", "moe_dispatch_backward", "moe_combine", "moe_combine_backward", "quantize_rows",
         "experts_product")


class Placed(torch.Tensor):
    """A host tensor that says it lies on GPU 0."""
    place = 0

    def get_device(self):
        return self.place


class Elsewhere(Placed):
    place = 1


def placed(t, place=Placed):
    return t.as_subclass(place)


@pytest.fixture
def Z(monkeypatch):
    """The binding with its library's calls recorded in Z.calls: (name, arguments,
    current GPU)."""
    from lossless_bf16_exponent_codec_amd import zipccl
    calls, current = [], [0]
    for name in NAMES:
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


def rows8(rows, stride, columns=slice(None)):
    """Columns of an int8 matrix."""
    return placed(torch.zeros(rows, stride, dtype=torch.int8))[:, columns]


def quantize(Z, q, length):
    T = q.shape[0]
    Z.quantize_rows(placed(torch.zeros(T, length, dtype=torch.bfloat16)), q, placed(torch.zeros(T)))


def product(Z, q, length):
    M, wide = q.shape[0], -(-length // 128) * 128
    Z.experts_product(q, placed(torch.zeros(M)), placed(torch.zeros(7, wide, dtype=torch.int8)),
                      placed(torch.zeros(7)), length, placed(torch.zeros(M, 7)))


def test_rows_whose_padding_lies_elsewhere_are_refused(Z):
    # 8-bit rows are written and read up to the next multiple of 128 bytes.  100 values from
    # column 16 on of 128: the padding is the next row's first 16 columns and, after the last
    # row, no memory of the tensor.
    for call in quantize, product:
        with pytest.raises(ValueError, match="padding"):
            call(Z, rows8(5, 128, slice(16, 116)), 100)
        # the last columns of a wider matrix
        with pytest.raises(ValueError, match="padding"):
            call(Z, rows8(5, 256, slice(192, 256)), 64)
    # the last row's padding lies past the memory
    cut = torch.zeros(4 * 128 + 100, dtype=torch.int8)
    cut = placed(cut).as_strided((5, 100), (128, 1))
    for call in quantize, product:
        with pytest.raises(ValueError, match="padding"):
            call(Z, cut, 100)
    assert not Z.calls


def test_rows_with_their_padding_behind_them_are_taken(Z):
    for q in rows8(5, 128), rows8(5, 128, slice(0, 100)), rows8(5, 256, slice(128, 228)), rows8(5, 384, slice(16, 144)):
        quantize(Z, q, 100)
        product(Z, q, 100)
        assert [name for name, *_ in Z.calls] == ["quantize_rows", "experts_product"]
        assert Z.calls[0][1][6] == q.data_ptr() and Z.calls[0][1][8] == q.stride(0)
        Z.calls.clear()


# Each call as a function of its tensors, by position: (binding, tensors, the rest).
T, K, E, H, M = 6, 2, 3, 40, 12
BF = torch.bfloat16


def zeros(*shape, dtype=torch.float32):
    return lambda: torch.zeros(*shape, dtype=dtype)


SLOTS, ROWS, TOKENS, WEIGHTS = zeros(T, K, dtype=torch.int32), zeros(M, H, dtype=BF), zeros(T, H, dtype=BF), zeros(T, K)
ALL = {
    "moe_sort": (lambda Z, a, **kw: Z.moe_sort(a[0], E, *a[1:], **kw),
                 [SLOTS, zeros(E + 1, dtype=torch.int32), zeros(M, dtype=torch.int32), SLOTS,
                  zeros(1 << 20, dtype=torch.uint8)]),
    "moe_dispatch": (lambda Z, a, **kw: Z.moe_dispatch(*a, **kw), [TOKENS, SLOTS, ROWS]),
    "moe_dispatch_backward": (lambda Z, a, **kw: Z.moe_dispatch_backward(*a, **kw), [ROWS, SLOTS, TOKENS]),
    "moe_combine": (lambda Z, a, **kw: Z.moe_combine(*a, **kw), [ROWS, SLOTS, WEIGHTS, TOKENS]),
    "moe_combine_backward": (lambda Z, a, **kw: Z.moe_combine_backward(*a, **kw),
                             [TOKENS, ROWS, SLOTS, WEIGHTS, ROWS, WEIGHTS]),
    "quantize_rows": (lambda Z, a, **kw: Z.quantize_rows(*a[:3], slots=a[3], **kw),
                      [TOKENS, zeros(M, 128, dtype=torch.int8), zeros(M), SLOTS]),
    "experts_product": (lambda Z, a, **kw: Z.experts_product(*a[:4], H, a[4], offsets=a[5], **kw),
                        [zeros(M, 128, dtype=torch.int8), zeros(M), zeros(E, 7, 128, dtype=torch.int8), zeros(E, 7),
                         zeros(M, 7), zeros(E + 1, dtype=torch.int32)]),
}


@pytest.mark.parametrize("name", ALL)
def test_tensors_of_the_host_or_of_two_gpus_are_refused(Z, name):
    call, makers = ALL[name]
    for place in torch.Tensor, Elsewhere:
        for i in range(len(makers)):
            with pytest.raises(ValueError, match="one GPU"):
                call(Z, [placed(m(), place if j == i else Placed) for j, m in enumerate(makers)])
    host = [m() for m in makers]
    with pytest.raises(ValueError, match="one GPU"):
        call(Z, host)
    with pytest.raises(ValueError):
        call(Z, [placed(m()) for m in makers], status=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        call(Z, [placed(m()) for m in makers], status=placed(torch.zeros(1, dtype=torch.int32), Elsewhere))
    assert not Z.calls


class Stream:
    def __init__(self, device_index):
        self.device_index, self.cuda_stream = device_index, 77


@pytest.mark.parametrize("name", ALL)
def test_calls_go_to_the_gpu_that_holds_the_tensors(Z, name):
    call, makers = ALL[name]
    for device, place in enumerate((Placed, Elsewhere)):
        tensors = [placed(m(), place) for m in makers]
        status = placed(torch.zeros(1, dtype=torch.int32), place)
        call(Z, tensors)
        call(Z, tensors, status=status)
        call(Z, tensors, status=status, stream=Stream(device))
        call(Z, tensors, status=4096, stream=99)
        with pytest.raises(ValueError, match="stream"):
            call(Z, tensors, stream=Stream(1 - device))
        at = status.data_ptr()
        assert [(args[-2:], where) for _, args, where in Z.calls] == [
            ((None, 1000 + device), device), ((at, 1000 + device), device), ((at, 77), device), ((4096, 99), device)]
        assert all(n == name and args[:-2] == Z.calls[0][1][:-2] for n, args, _ in Z.calls)
        Z.calls.clear()


def test_workspace_and_status_hold_what_is_written(Z):
    # 2^20 bytes by their count, one by their memory; a status word of two bytes, and of one
    # byte four times
    call, makers = ALL["moe_sort"]
    tensors = [placed(m()) for m in makers]
    with pytest.raises(ValueError, match="workspace"):
        call(Z, tensors[:4] + [placed(torch.zeros(1, dtype=torch.uint8)).expand(1 << 20)])
    for name, (call, makers) in ALL.items():
        tensors = [placed(m()) for m in makers]
        for status in torch.zeros(1, dtype=torch.int16), torch.zeros(0, dtype=torch.int32), \
                torch.zeros(1, dtype=torch.uint8).expand(4):
            with pytest.raises(ValueError, match="status"):
                call(Z, tensors, status=placed(status))
        assert not Z.calls
        for status in torch.zeros(1, dtype=torch.int64), torch.zeros(4, dtype=torch.uint8), \
                torch.zeros(4, 4, dtype=torch.int32)[:, 1]:
            call(Z, tensors, status=placed(status))
        assert len(Z.calls) == 3
        Z.calls.clear()


def test_strides_whose_last_row_has_no_64_bit_address_are_refused():
    # 2^30 rows 2^39 values apart
    from lossless_bf16_exponent_codec_amd import zipccl as Z
    L, A, far, many = Z.lib(), 1 << 20, 1 << 39, 1 << 30
    for rc in (L.zipccl_moe_sort(A, 8, far, many, 1, 4, A, A, A, A, Z.MOE_SORT_WORKSPACE_BYTES, None, None),
               L.zipccl_moe_dispatch(A, far, A, many, 1, 8, 0, A, 4, 8, None, None),
               L.zipccl_moe_dispatch(A, 8, A, 4, 1, 8, 1, A, many, far, None, None),
               L.zipccl_moe_combine(A, many, far, A, A, 4, 1, 8, 0, A, 8, None, None),
               L.zipccl_moe_combine(A, 4, 8, A, A, many, 1, 8, 1, A, far, None, None),
               L.zipccl_moe_dispatch_backward(A, many, far, A, 4, 1, 8, 0, A, 8, None, None),
               L.zipccl_moe_combine_backward(A, far, A, 4, 8, A, A, many, 1, 8, 0, A, 8, A, None, None),
               L.zipccl_moe_combine_backward(A, 8, A, many, far, A, A, 4, 1, 8, 0, A, 8, A, None, None),
               L.zipccl_moe_combine_backward(A, 8, A, many, 8, A, A, 4, 1, 8, 0, A, far, A, None, None),
               L.zipccl_quantize_rows(A, far, many, 8, A, 1, A, 4, 128, A, None, None),
               L.zipccl_quantize_rows(A, 8, 4, 8, A, 1, A, many, far, A, None, None),
               L.zipccl_experts_product(A, 128, A, 1 << 24, A, 128, A, 1, 8, 100, None, A, far, 0, None, None)):
        assert rc == Z.ERR_SIZE


def test_host_calls_need_no_gpu_build_of_torch():
    # a torch without GPU support has no call for a stream's handle: the package loads, and
    # its host calls work
    import subprocess
    import sys
    code = ("import torch\n"
            "for name in '_cuda_getCurrentRawStream', '_cuda_getDevice':\n"
            "    if hasattr(torch._C, name): delattr(torch._C, name)\n"
            "from lossless_bf16_exponent_codec_amd import zipccl as Z\n"
            "assert Z.static_size(100) > 0 and len(Z.plan(sigma=1.0).exponents) == 7\n")
    root = __file__.rsplit("/tests/", 1)[0]
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=300)
