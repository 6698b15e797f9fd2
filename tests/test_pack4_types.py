"""4-bit values of every integer type, packed on the host."""
import numpy as np
import pytest
import torch

from tests import router_reference as R

UNSIGNED = [torch.uint8, torch.uint16, torch.uint32, torch.uint64]
SIGNED = [torch.int8, torch.int16, torch.int32, torch.int64]


@pytest.fixture(scope="module")
def moe():
    from lossless_bf16_exponent_codec_amd import moe
    return moe


@pytest.mark.parametrize("dtype", UNSIGNED + SIGNED)
def test_values_of_any_integer_type(moe, dtype):
    E, N, H = 2, 18, 130
    values = np.random.default_rng(3).integers(0 if dtype in UNSIGNED else -8, 8, (E, N, H))
    given = torch.from_numpy(values).to(dtype)
    back, clean = R.unpack4(moe.pack4(given).numpy(), E, N, H)
    assert clean and np.array_equal(back, values)
    strided = torch.from_numpy(values.transpose(2, 1, 0).copy()).to(dtype).permute(2, 1, 0)
    assert torch.equal(moe.pack4(strided), moe.pack4(given))
    experts = moe.QuantizedExperts4.of(given, torch.ones(E, N, 2), 128)
    assert torch.equal(experts.q, moe.pack4(given)) and experts.scales.shape == (E, 2, N)
    assert torch.equal(given.to(torch.int64), torch.from_numpy(values))      # as they were


@pytest.mark.parametrize("dtype", UNSIGNED + SIGNED)
def test_values_that_need_more_bits_are_refused(moe, dtype):
    top = 2 ** (8 * dtype.itemsize) - 1 if dtype in UNSIGNED else 2 ** (8 * dtype.itemsize - 1) - 1
    wrong = [8, top, top // 2 + 1] if dtype in UNSIGNED else [8, top, -9, -top - 1]
    for value in wrong:
        values = np.zeros((1, 3, 5), str(dtype).split(".")[1])
        values[0, 1, 2] = value
        with pytest.raises(ValueError, match="-8 to 7"):
            moe.pack4(torch.from_numpy(values))


def test_truth_values(moe):
    values = torch.tensor([[[True, False, True]]])
    back, clean = R.unpack4(moe.pack4(values).numpy(), 1, 1, 3)
    assert clean and back.tolist() == [[[1, 0, 1]]]
