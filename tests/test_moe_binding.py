"""The binding of the mixture-of-experts calls: which tensors it passes on, and which it
refuses before the library is called.  The library's calls are recorded, not made; no call
here reaches a GPU."""
import pytest
import torch

NAMES = ("moe_sort", "moe_dispatch", "moe_dispatch_backward", "moe_combine", "moe_combine_backward", "quantize_rows",
         "experts_product")


class Placed(torch.Tensor):
    """A host tensor that says it lies on GPU `place`."""
    place = 0

    def get_device(self):
        return self.place


def placed(t, place=0):
    t = t.as_subclass(Placed)
    t.place = place
    return t


@pytest.fixture
def Z(monkeypatch):
    """The binding with its library's calls recorded in Z.calls: (name, arguments)."""
    from lossless_bf16_exponent_codec_amd import zipccl
    calls = []
    for name in NAMES:
        def record(*args, name=name):
            calls.append((name, args))
            return zipccl.OK
        monkeypatch.setattr(zipccl.lib(), "zipccl_" + name, record)
    monkeypatch.setattr(zipccl, "_current_device", lambda: 0)
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
    Z.experts_product(q, placed(torch.zeros(M)), placed(torch.zeros(7, wide, dtype=torch.int8)), placed(torch.zeros(7)), length,
                      placed(torch.zeros(M, 7)))


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
        assert [name for name, _ in Z.calls] == ["quantize_rows", "experts_product"]
        assert Z.calls[0][1][6] == q.data_ptr() and Z.calls[0][1][8] == q.stride(0)
        Z.calls.clear()
