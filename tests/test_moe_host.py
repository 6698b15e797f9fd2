"""Refusals of the mixture-of-experts calls: every bad argument is an error before anything
is enqueued.  No call here reaches a GPU."""
import pytest
import torch

P = 1 << 20   # an aligned stand-in for a device address: every call below is refused


@pytest.fixture(scope="module")
def Z():
    from lossless_bf16_exponent_codec_amd import zipccl
    return zipccl


def cases(good, changes):
    for want, change in changes:
        args = dict(good)
        args.update(change)
        yield want, list(args.values()), change


def check(fn, good, changes):
    for want, args, change in cases(good, changes):
        assert fn(*args) == want, change


def test_sort_refusals(Z):
    good = dict(ids=P, id_bytes=8, stride=4, tokens=10, top_k=4, experts=16, offsets=P, rows=P, slots=P, ws=P,
                ws_bytes=Z.MOE_SORT_WORKSPACE_BYTES, status=None, stream=None)
    check(Z.lib().zipccl_moe_sort, good, [
        (Z.ERR_INVALID, dict(ids=None)), (Z.ERR_INVALID, dict(id_bytes=2)), (Z.ERR_INVALID, dict(stride=3)),
        (Z.ERR_INVALID, dict(top_k=0)), (Z.ERR_INVALID, dict(top_k=65, stride=65)), (Z.ERR_INVALID, dict(experts=0)),
        (Z.ERR_INVALID, dict(experts=1025)), (Z.ERR_INVALID, dict(offsets=None)), (Z.ERR_INVALID, dict(rows=None)),
        (Z.ERR_INVALID, dict(slots=None)), (Z.ERR_INVALID, dict(ws=None)),
        (Z.ERR_SIZE, dict(ws_bytes=Z.MOE_SORT_WORKSPACE_BYTES - 1)), (Z.ERR_SIZE, dict(tokens=1 << 29)),
        (Z.ERR_SIZE, dict(tokens=1 << 62)), (Z.ERR_SIZE, dict(stride=1 << 40)),
        (Z.ERR_ALIGN, dict(ids=P + 4)), (Z.ERR_ALIGN, dict(offsets=P + 2)), (Z.ERR_ALIGN, dict(rows=P + 1)),
        (Z.ERR_ALIGN, dict(slots=P + 2)), (Z.ERR_ALIGN, dict(ws=P + 128)), (Z.ERR_ALIGN, dict(status=P + 2))])


ROWS = [("INVALID", dict(slots=None)), ("INVALID", dict(top_k=0)), ("INVALID", dict(top_k=65)),
        ("INVALID", dict(row_len=0)), ("INVALID", dict(dtype=2)), ("INVALID", dict(dtype=-1)),
        ("SIZE", dict(tokens=1 << 31)), ("SIZE", dict(tokens=1 << 30)), ("SIZE", dict(y_rows=1 << 31)),
        ("SIZE", dict(row_len=(1 << 28) + 1)), ("INVALID", dict(y=None)), ("INVALID", dict(y_stride=99)),
        ("SIZE", dict(y_stride=1 << 40)), ("ALIGN", dict(y=P + 1)), ("ALIGN", dict(slots=P + 2)),
        ("ALIGN", dict(status=P + 2)), ("ALIGN", dict(y=P + 2, dtype=1))]


def rows_changes(Z, more):
    return [(getattr(Z, "ERR_" + want), change) for want, change in ROWS + more]


def test_dispatch_refusals(Z):
    good = dict(x=P, x_stride=100, slots=P, tokens=10, top_k=2, row_len=100, dtype=0, y=P, y_rows=20, y_stride=100,
                status=None, stream=None)
    check(Z.lib().zipccl_moe_dispatch, good, rows_changes(Z, [
        ("INVALID", dict(x=None)), ("INVALID", dict(x_stride=99)), ("ALIGN", dict(x=P + 1))]))


def test_combine_refusals(Z):
    good = dict(y=P, y_rows=20, y_stride=100, slots=P, weights=P, tokens=10, top_k=2, row_len=100, dtype=0, out=P,
                out_stride=100, status=None, stream=None)
    more = [("INVALID", dict(out=None)), ("INVALID", dict(out_stride=99)), ("ALIGN", dict(out=P + 1))]
    check(Z.lib().zipccl_moe_combine, good, rows_changes(Z, more + [("ALIGN", dict(weights=P + 2))]))
    del good["weights"]
    check(Z.lib().zipccl_moe_dispatch_backward, good, rows_changes(Z, more))


def test_combine_backward_refusals(Z):
    good = dict(dout=P, dout_stride=100, y=P, y_rows=20, y_stride=100, slots=P, weights=P, tokens=10, top_k=2,
                row_len=100, dtype=0, dy=P, dy_stride=100, dweights=P, status=None, stream=None)
    check(Z.lib().zipccl_moe_combine_backward, good, rows_changes(Z, [
        ("INVALID", dict(dout=None)), ("INVALID", dict(dout_stride=99)), ("ALIGN", dict(dout=P + 1)),
        ("INVALID", dict(dy=None)), ("INVALID", dict(dy_stride=99)), ("ALIGN", dict(dy=P + 1)),
        ("INVALID", dict(weights=None)), ("INVALID", dict(dweights=None)), ("ALIGN", dict(weights=P + 2)),
        ("ALIGN", dict(dweights=P + 2))]))


def test_quantize_refusals(Z):
    good = dict(x=P, x_stride=100, tokens=10, row_len=100, slots=P, top_k=2, q=P, q_rows=20, q_stride=128, scales=P,
                status=None, stream=None)
    E = Z
    check(Z.lib().zipccl_quantize_rows, good, [
        (E.ERR_INVALID, dict(x=None)), (E.ERR_INVALID, dict(x_stride=99)), (E.ERR_INVALID, dict(row_len=0)),
        (E.ERR_INVALID, dict(top_k=0)), (E.ERR_INVALID, dict(q=None)), (E.ERR_INVALID, dict(scales=None)),
        (E.ERR_INVALID, dict(row_len=129, x_stride=129)), (E.ERR_INVALID, dict(slots=None, q_rows=9)),
        (E.ERR_SIZE, dict(slots=None, q_rows=1 << 31)), (E.ERR_SIZE, dict(q_stride=1 << 40)),
        (E.ERR_SIZE, dict(tokens=1 << 30)), (E.ERR_ALIGN, dict(q_stride=136)), (E.ERR_ALIGN, dict(q=P + 8)),
        (E.ERR_ALIGN, dict(x=P + 1)), (E.ERR_ALIGN, dict(scales=P + 2)), (E.ERR_ALIGN, dict(slots=P + 2)),
        (E.ERR_ALIGN, dict(status=P + 2)), (E.ERR_ALIGN, dict(slots=None, status=P + 2))])


def test_product_refusals(Z):
    good = dict(q=P, q_stride=128, scales=P, rows=20, w=P, w_stride=128, w_scales=P, experts=4, outputs=50,
                row_len=100, offsets=P, out=P, out_stride=50, dtype=0, status=None, stream=None)
    check(Z.lib().zipccl_experts_product, good, [
        (Z.ERR_INVALID, dict(q=None)), (Z.ERR_INVALID, dict(scales=None)), (Z.ERR_INVALID, dict(w=None)),
        (Z.ERR_INVALID, dict(w_scales=None)), (Z.ERR_INVALID, dict(out=None)), (Z.ERR_INVALID, dict(offsets=None)),
        (Z.ERR_INVALID, dict(experts=0)), (Z.ERR_INVALID, dict(experts=1025)), (Z.ERR_INVALID, dict(outputs=0)),
        (Z.ERR_INVALID, dict(row_len=0)), (Z.ERR_INVALID, dict(row_len=129)), (Z.ERR_INVALID, dict(dtype=2)),
        (Z.ERR_INVALID, dict(out_stride=49)), (Z.ERR_SIZE, dict(rows=1 << 31)),
        (Z.ERR_SIZE, dict(row_len=131072, q_stride=131072, w_stride=131072)),
        (Z.ERR_SIZE, dict(rows=(1 << 31) - 1, outputs=1 << 20, out_stride=1 << 20)),
        (Z.ERR_SIZE, dict(outputs=1 << 24, out_stride=1 << 24)), (Z.ERR_SIZE, dict(w_stride=1 << 40)),
        (Z.ERR_ALIGN, dict(q_stride=192)), (Z.ERR_ALIGN, dict(w_stride=160)), (Z.ERR_ALIGN, dict(q=P + 8)),
        (Z.ERR_ALIGN, dict(w=P + 4)), (Z.ERR_ALIGN, dict(scales=P + 1)), (Z.ERR_ALIGN, dict(w_scales=P + 2)),
        (Z.ERR_ALIGN, dict(offsets=P + 2)), (Z.ERR_ALIGN, dict(out=P + 1)), (Z.ERR_ALIGN, dict(out=P + 2, dtype=1)),
        (Z.ERR_ALIGN, dict(status=P + 2))])


def test_nothing_to_do_is_no_error(Z):
    L = Z.lib()
    assert L.zipccl_moe_dispatch(None, 100, None, 0, 2, 100, 0, None, 0, 100, None, None) == Z.OK
    assert L.zipccl_moe_combine(None, 0, 100, None, None, 0, 2, 100, 0, None, 100, None, None) == Z.OK
    assert L.zipccl_quantize_rows(None, 100, 0, 100, None, 1, None, 0, 128, None, None, None) == Z.OK
    assert L.zipccl_experts_product(None, 128, None, 0, P, 128, P, 4, 50, 100, P, None, 50, 0, None, None) == Z.OK


def test_binding_checks_shapes_and_types(Z):
    bf, i32 = torch.zeros(4, 10, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    f32, i8 = torch.zeros(8, 10), torch.zeros(8, 128, dtype=torch.int8)
    one = torch.zeros(8)
    for call in [
            lambda: Z.moe_dispatch(bf, i32, f32),                                  # dtypes differ
            lambda: Z.moe_dispatch(bf.half(), i32, bf.half()),                     # no such dtype
            lambda: Z.moe_dispatch(bf, i32.long(), bf),                            # slots are int32
            lambda: Z.moe_dispatch(bf, i32[:3], bf),                               # slots of other tokens
            lambda: Z.moe_dispatch(bf.t(), i32, bf),                               # columns are not rows
            lambda: Z.moe_dispatch(bf[:1].expand(4, 10), i32, bf),                 # one row four times
            lambda: Z.moe_dispatch(bf[0], i32, bf),
            lambda: Z.moe_combine(f32, i32, one[:7], f32[:4]),                     # too few weights
            lambda: Z.moe_combine(f32, i32, one.double(), f32[:4]),
            lambda: Z.moe_combine_backward(f32[:4], f32, i32, one, f32[:7], one),  # dy of other rows
            lambda: Z.moe_sort(i32.float(), 4, i32, i32, i32, i8),
            lambda: Z.moe_sort(i32, 8, torch.zeros(8, dtype=torch.int32), i32, i32, i8),   # too few offsets
            lambda: Z.quantize_rows(f32, i8, one),                                 # BF16 rows only
            lambda: Z.quantize_rows(torch.zeros(8, 200, dtype=torch.bfloat16), i8, one),   # longer than q's rows
            lambda: Z.experts_product(i8, one, i8, one, 10, f32[:, :7]),           # out is rows x outputs
            lambda: Z.experts_product(i8, one, i8, one, 129, torch.zeros(8, 8)),
            lambda: Z.experts_product(i8, one, i8[:, :64], one, 10, torch.zeros(8, 8))]:
        with pytest.raises(ValueError):
            call()
