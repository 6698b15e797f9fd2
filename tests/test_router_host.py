"""Refusals of the router's calls and of those with 4-bit weights: every bad argument is an
error before anything is enqueued; what the binding passes on, and the torch layer's shapes.
No call here reaches a GPU."""
import numpy as np
import pytest
import torch

from tests import router_reference as R

P = 1 << 20   # an aligned stand-in for a device address: every call below is refused


@pytest.fixture(scope="module")
def Z():
    from lossless_bf16_exponent_codec_amd import zipccl
    return zipccl


@pytest.fixture(scope="module")
def moe():
    from lossless_bf16_exponent_codec_amd import moe
    return moe


def check(Z, fn, good, changes):
    for want, change in changes:
        args = dict(good)
        args.update(change)
        assert fn(*args.values()) == getattr(Z, "ERR_" + want), change


LOGITS = [("INVALID", dict(logits=None)), ("INVALID", dict(dtype=2)), ("INVALID", dict(stride=15)),
          ("INVALID", dict(E=0)), ("INVALID", dict(E=1025, stride=1025)), ("INVALID", dict(K=0)),
          ("INVALID", dict(K=65)), ("SIZE", dict(tokens=1 << 31)), ("SIZE", dict(tokens=1 << 30)),
          ("SIZE", dict(stride=1 << 40)), ("ALIGN", dict(logits=P + 1)), ("ALIGN", dict(logits=P + 2, dtype=1)),
          ("ALIGN", dict(status=P + 2))]
BALANCE = [("INVALID", dict(sums=None)), ("INVALID", dict(loss=None)), ("INVALID", dict(ws=None)),
           ("SIZE", dict(ws_bytes=100)), ("ALIGN", dict(ws=P + 128)), ("ALIGN", dict(counts=P + 2)),
           ("ALIGN", dict(sums=P + 2)), ("ALIGN", dict(loss=P + 1))]
CHOICES = [("INVALID", dict(experts=None)), ("INVALID", dict(id_bytes=2)), ("INVALID", dict(id_stride=3)),
           ("SIZE", dict(id_stride=1 << 40)), ("ALIGN", dict(experts=P + 4))]


def test_gate_refusals(Z):
    good = dict(logits=P, dtype=0, stride=16, tokens=10, E=16, mask=P, K=4, renormalize=1, experts=P, weights=P,
                counts=P, sums=P, loss=P, ws=P, ws_bytes=Z.MOE_GATE_WORKSPACE_BYTES, status=None, stream=None)
    check(Z, Z.lib().zipccl_moe_gate, good, LOGITS + BALANCE + [
        ("INVALID", dict(K=17)), ("INVALID", dict(experts=None)), ("INVALID", dict(weights=None)),
        ("INVALID", dict(counts=None)), ("INVALID", dict(counts=None, sums=None)),
        ("SIZE", dict(ws_bytes=Z.MOE_GATE_WORKSPACE_BYTES - 1)), ("ALIGN", dict(experts=P + 2)),
        ("ALIGN", dict(weights=P + 2))])
    assert Z.lib().zipccl_moe_gate(None, 0, 16, 0, 16, None, 4, 1, None, None, None, None, None, None, 0, None,
                                   None) == Z.OK


def test_balance_refusals(Z):
    good = dict(logits=P, dtype=1, stride=16, tokens=10, E=16, mask=None, experts=P, id_bytes=8, id_stride=4, K=4,
                counts=P, sums=P, loss=P, ws=P, ws_bytes=Z.MOE_GATE_WORKSPACE_BYTES, status=None, stream=None)
    check(Z, Z.lib().zipccl_moe_balance, good, LOGITS + BALANCE + CHOICES + [("INVALID", dict(counts=None))])


def test_backward_refusals(Z):
    good = dict(logits=P, dtype=0, stride=16, tokens=10, E=16, mask=P, experts=P, id_bytes=8, id_stride=4, K=4,
                renormalize=1, dweights=P, counts=P, dloss=P, dlogits=P, dstride=16, status=None, stream=None)
    check(Z, Z.lib().zipccl_moe_gate_backward, good, LOGITS + CHOICES + [
        ("INVALID", dict(counts=None)), ("INVALID", dict(dloss=None)),
        ("INVALID", dict(dweights=None, counts=None, dloss=None)), ("INVALID", dict(dlogits=None)),
        ("INVALID", dict(dstride=15)), ("SIZE", dict(dstride=1 << 40)), ("ALIGN", dict(dlogits=P + 1)),
        ("ALIGN", dict(dweights=P + 2)), ("ALIGN", dict(counts=P + 1)), ("ALIGN", dict(dloss=P + 2))])
    assert Z.lib().zipccl_moe_gate_backward(None, 0, 16, 0, 16, None, None, 8, 4, 4, 1, None, None, None, None, 16,
                                            None, None) == Z.OK


def test_quantize4_refusals(Z):
    good = dict(w=P, w_stride=100, E=4, N=50, H=100, group=32, q=P, scales=P, dtype=0, stream=None)
    check(Z, Z.lib().zipccl_quantize_weights4, good, [
        ("INVALID", dict(w=None)), ("INVALID", dict(q=None)), ("INVALID", dict(scales=None)), ("INVALID", dict(E=0)),
        ("INVALID", dict(E=1025)), ("INVALID", dict(N=0)), ("INVALID", dict(H=0)), ("INVALID", dict(group=0)),
        ("INVALID", dict(group=16)), ("INVALID", dict(group=96)), ("INVALID", dict(group=192)),
        ("INVALID", dict(dtype=2)), ("INVALID", dict(w_stride=99)), ("SIZE", dict(N=1 << 24)),
        ("SIZE", dict(H=(1 << 24) + 1, w_stride=1 << 25)), ("SIZE", dict(w_stride=1 << 40)),
        ("SIZE", dict(N=1 << 16, H=1 << 20, w_stride=1 << 20)), ("ALIGN", dict(w=P + 1)),
        ("ALIGN", dict(q=P + 8)), ("ALIGN", dict(scales=P + 1)), ("ALIGN", dict(scales=P + 2, dtype=1))])


def test_product4_refusals(Z):
    good = dict(x=P, x_stride=100, x_rows=30, index=P, rows=20, q=P, scales=P, s_dtype=0, group=64, E=4, N=50, H=100,
                offsets=P, out=P, out_stride=50, dtype=0, status=None, stream=None)
    check(Z, Z.lib().zipccl_experts_product4, good, [
        ("INVALID", dict(x=None)), ("INVALID", dict(q=None)), ("INVALID", dict(scales=None)), ("INVALID", dict(out=None)),
        ("INVALID", dict(offsets=None)), ("INVALID", dict(index=None)), ("INVALID", dict(E=0)),
        ("INVALID", dict(E=1025)), ("INVALID", dict(N=0)), ("INVALID", dict(H=0)), ("INVALID", dict(group=48)),
        ("INVALID", dict(s_dtype=2)), ("INVALID", dict(dtype=-1)), ("INVALID", dict(x_stride=99)),
        ("INVALID", dict(out_stride=49)), ("SIZE", dict(rows=1 << 31)), ("SIZE", dict(x_rows=1 << 31)),
        ("SIZE", dict(N=1 << 24, out_stride=1 << 24)), ("SIZE", dict(H=(1 << 24) + 1, x_stride=1 << 25)),
        ("SIZE", dict(rows=(1 << 31) - 1, N=1 << 20, out_stride=1 << 20)), ("SIZE", dict(x_stride=1 << 40)),
        ("SIZE", dict(N=1 << 18, out_stride=1 << 18, H=1 << 20, x_stride=1 << 20, group=128)),
        ("ALIGN", dict(x=P + 1)), ("ALIGN", dict(index=P + 2)), ("ALIGN", dict(q=P + 8)), ("ALIGN", dict(scales=P + 1)),
        ("ALIGN", dict(scales=P + 2, s_dtype=1)), ("ALIGN", dict(offsets=P + 2)), ("ALIGN", dict(out=P + 1)),
        ("ALIGN", dict(out=P + 2, dtype=1)), ("ALIGN", dict(status=P + 2))])
    good.update(x=None, x_rows=0, index=None, rows=0, out=None)
    assert Z.lib().zipccl_experts_product4(*good.values()) == Z.OK


def test_weights4_size(Z):
    assert Z.weights4_size(1, 1, 1) == 1024 and Z.weights4_size(3, 17, 129) == 3 * 2 * 2 * 1024
    assert Z.weights4_size(0, 16, 128) == 0 and Z.weights4_size(1, 1 << 24, 1) == 0


def test_binding_refuses_shapes_and_types(Z):
    z, i32, f = torch.zeros(6, 8), torch.zeros(6, 2, dtype=torch.int32), torch.zeros(6, 2)
    counts, sums, loss = torch.zeros(9, dtype=torch.int32), torch.zeros(8), torch.zeros(1)
    ws = torch.zeros(16, dtype=torch.uint8)
    bf, q, s = torch.zeros(6, 100, dtype=torch.bfloat16), torch.zeros(2048, dtype=torch.uint8), torch.zeros(2, 1, 16)
    off = torch.zeros(3, dtype=torch.int32)
    out = torch.zeros(5, 16)
    for call in [
            lambda: Z.moe_gate(z.double(), i32, f), lambda: Z.moe_gate(z.t(), i32, f),
            lambda: Z.moe_gate(z, i32.long(), f), lambda: Z.moe_gate(z, i32[:5], f),
            lambda: Z.moe_gate(z, torch.zeros(6, 5, dtype=torch.int32)[:, :2], f),
            lambda: Z.moe_gate(z, i32, f[:5]), lambda: Z.moe_gate(z, i32, f.double()),
            lambda: Z.moe_gate(z, i32, f, mask=torch.zeros(5, dtype=torch.bool)),
            lambda: Z.moe_gate(z, i32, f, mask=torch.zeros(6)),
            lambda: Z.moe_gate(z, i32, f, mask=torch.zeros(12, dtype=torch.bool)[::2]),
            lambda: Z.moe_gate(z, i32, f, counts=counts), lambda: Z.moe_gate(z, i32, f, sums=sums, loss=loss),
            lambda: Z.moe_gate(z, i32, f, counts=counts[:8], sums=sums, loss=loss, workspace=ws),
            lambda: Z.moe_gate(z, i32, f, counts=counts, sums=sums[:7], loss=loss, workspace=ws),
            lambda: Z.moe_balance(z, i32[:5], counts, sums, loss, ws),
            lambda: Z.moe_balance(z, f, counts, sums, loss, ws),
            lambda: Z.moe_balance(z, i32, counts, sums, loss.double(), ws),
            lambda: Z.moe_gate_backward(z, i32, z[:, :7], dweights=f),
            lambda: Z.moe_gate_backward(z, i32, z.bfloat16(), dweights=f),
            lambda: Z.moe_gate_backward(z, i32, z, dweights=f[:5]),
            lambda: Z.moe_gate_backward(z, i32, z, counts=counts[:8], dloss=loss),
            lambda: Z.moe_gate_backward(z, i32, z, counts=counts, dloss=loss[:0]),
            lambda: Z.quantize_weights4(bf.float(), 64, q, s), lambda: Z.quantize_weights4(bf, 64, q[:1023], s),
            lambda: Z.quantize_weights4(torch.zeros(0, 6, 100, dtype=torch.bfloat16), 64, q, s),
            lambda: Z.quantize_weights4(bf, 128, q, s), lambda: Z.quantize_weights4(bf, 0, q, s),
            lambda: Z.experts_product4(bf.float(), q, s, 128, out, rows=off, offsets=off),
            lambda: Z.experts_product4(bf, q[:1024], s, 128, out, offsets=off),
            lambda: Z.experts_product4(bf, q, s, 64, out, offsets=off),
            lambda: Z.experts_product4(bf, q, s.half(), 128, out, offsets=off),
            lambda: Z.experts_product4(bf, q, s, 128, out, offsets=off),                 # 5 rows, 6 of x
            lambda: Z.experts_product4(bf, q, s, 128, out, rows=off[:2], offsets=off),
            lambda: Z.experts_product4(bf, q.view(torch.int8), s, 128, out, rows=torch.zeros(5, dtype=torch.int32),
                                       offsets=off)]:
        with pytest.raises(ValueError):
            call()


def test_pack4_lays_out_tiles(moe):
    rng = np.random.default_rng(0)
    for E, N, H in ((1, 1, 1), (2, 17, 129), (3, 40, 300)):
        values = rng.integers(-8, 8, (E, N, H))
        q = moe.pack4(torch.from_numpy(values).to(torch.int8))
        assert q.shape == (E, -(-N // 16) * -(-H // 128) * 1024) and q.dtype == torch.uint8
        back, clean = R.unpack4(q.numpy(), E, N, H)
        assert clean and np.array_equal(back, values)
    with pytest.raises(ValueError):
        moe.pack4(torch.full((1, 2, 3), 8))
    with pytest.raises(ValueError):
        moe.QuantizedExperts4.of(torch.zeros(1, 2, 130, dtype=torch.int8), torch.ones(1, 2, 1), 64)


def test_a_wrong_product_is_seen():
    # the plain product with a mistake planted in it differs by more than the tolerance held on the GPU
    rng = np.random.default_rng(1)
    E, N, H, group, M = 2, 20, 300, 64, 9
    values, scales = rng.integers(-8, 8, (E, N, H)), rng.uniform(0.5, 1.5, (E, 5, N))
    x, index, offsets = rng.standard_normal((M, H)), rng.integers(0, M, M), [0, 4, 9]
    want, size = R.product4(x, index, values, scales, group, offsets)
    tol = H * 2.0 ** -23 * size + 2.0 ** -8 * np.abs(want)

    def seen(v, s):
        return bool((np.abs(R.product4(x, index, v, s, group, offsets)[0] - want) > tol).any())

    swapped = values.copy()
    swapped[:, :, :2] = values[:, :, 1::-1]
    assert seen(swapped, scales)
    assert seen(values & 15, scales)                       # unsigned values
    assert seen(values, np.roll(scales, 1, axis=1))        # a group off
    cut = values.copy()
    cut[:, :, 288:] = 0                                     # the last piece left out
    assert seen(cut, scales)
