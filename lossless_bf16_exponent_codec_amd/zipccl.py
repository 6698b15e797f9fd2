"""Python binding of libzipccl (ctypes).  Argument marshalling only: every step of the
codec runs in the library's HIP kernels; torch supplies device memory and streams.

The names mirror the C ABI in include/zipccl.h.  There is no CPU fallback: if the
library is not built, importing this module raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libzipccl.so")

OK, ERR_INVALID, ERR_ALIGN, ERR_SIZE, ERR_HIP, ERR_CORRUPT = range(6)
STATUS_ESC_OVERFLOW, STATUS_CORRUPT, STATUS_BAD_INDEX, STATUS_WAIT_LIMIT = 1, 2, 4, 8
MAX_SEGMENTS, MAX_PEERS = 64, 16
FORMAT_VERSION, MAGIC = 1, 0x3143435A
MAX_EXPERTS, MAX_TOP_K, ROW_PAD, MOE_SORT_WORKSPACE_BYTES = 1024, 64, 128, 1 << 20
MOE_GATE_WORKSPACE_BYTES = 256 * (8 * MAX_EXPERTS + 16)
TILE4_OUTPUTS, TILE4_INPUTS, TILE4_BYTES = 16, 128, 1024
BF16, FP32 = 0, 1


class PlanT(ctypes.Structure):
    _fields_ = [("table", ctypes.c_uint8 * 7), ("reserved", ctypes.c_uint8)]

    @property
    def exponents(self):
        return list(self.table)

    def __repr__(self):
        return f"Plan({list(self.table)})"


class SegmentT(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("n", ctypes.c_uint64), ("plan", PlanT)]


class GatherSegmentT(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("src_rows", ctypes.c_uint64), ("row_len", ctypes.c_uint64),
                ("rows", ctypes.c_void_p), ("nrows", ctypes.c_uint64), ("plan", PlanT)]


class CodecProfileT(ctypes.Structure):
    _fields_ = [("compress_GBps", ctypes.c_double), ("accumulate_GBps", ctypes.c_double),
                ("compressed_fraction", ctypes.c_double)]


class LinkT(ctypes.Structure):
    _fields_ = [("bw_GBps", ctypes.c_double), ("latency_us", ctypes.c_double), ("links", ctypes.c_int)]


class DSegmentT(ctypes.Structure):
    _fields_ = [("dst", ctypes.c_void_p), ("n", ctypes.c_uint64)]


class ZipcclError(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = _lib.zipccl_strerror(status).decode() if _lib is not None else str(status)
        super().__init__(f"{what}: {msg} (status {status})")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run python -m lossless_bf16_exponent_codec_amd.build")
    lib = ctypes.CDLL(LIB_PATH)
    vp, u64, i32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int
    lib.zipccl_strerror.restype = ctypes.c_char_p
    lib.zipccl_strerror.argtypes = [i32]
    lib.zipccl_plan.restype = i32
    lib.zipccl_plan.argtypes = [ctypes.c_double, ctypes.POINTER(ctypes.c_uint8), ctypes.POINTER(PlanT)]
    lib.zipccl_plan_many.restype = i32
    lib.zipccl_plan_many.argtypes = [ctypes.POINTER(ctypes.c_double), i32, ctypes.POINTER(PlanT)]
    lib.zipccl_static_size.restype = u64
    lib.zipccl_static_size.argtypes = [u64]
    lib.zipccl_compressed_size.restype = u64
    lib.zipccl_compressed_size.argtypes = [u64, u64]
    lib.zipccl_workspace_size.restype = u64
    lib.zipccl_workspace_size.argtypes = [u64, i32]
    lib.zipccl_compress.restype = i32
    lib.zipccl_compress.argtypes = [ctypes.POINTER(SegmentT), i32, vp, u64, vp, u64, vp, u64, vp, vp, vp]
    lib.zipccl_compress_noalloc.restype = i32
    lib.zipccl_compress_noalloc.argtypes = [ctypes.POINTER(SegmentT), i32, vp, u64, vp, u64, vp, vp, vp]
    lib.zipccl_compress_chunks.restype = i32
    lib.zipccl_compress_chunks.argtypes = [ctypes.POINTER(SegmentT), i32, i32, ctypes.POINTER(vp),
                                           ctypes.POINTER(u64), ctypes.POINTER(vp), ctypes.POINTER(u64), vp, u64,
                                           vp, vp, vp]
    lib.zipccl_estimate_plans.restype = i32
    lib.zipccl_estimate_plans.argtypes = [ctypes.POINTER(SegmentT), i32, ctypes.c_uint32, vp, vp, u64, vp]
    lib.zipccl_estimate_workspace_size.restype = u64
    lib.zipccl_estimate_workspace_size.argtypes = [i32]
    lib.zipccl_compress_device_plans.restype = i32
    lib.zipccl_compress_device_plans.argtypes = [ctypes.POINTER(SegmentT), i32, vp, vp, u64, vp, u64, vp, u64, vp,
                                                 vp, vp]
    lib.zipccl_compress_gather.restype = i32
    lib.zipccl_compress_gather.argtypes = [ctypes.POINTER(GatherSegmentT), i32, vp, u64, vp, u64, vp, u64, vp, vp,
                                           vp]
    lib.zipccl_decompress.restype = i32
    lib.zipccl_decompress.argtypes = [vp, u64, vp, u64, ctypes.POINTER(DSegmentT), i32, vp, vp]
    lib.zipccl_decompress_shards.restype = i32
    lib.zipccl_decompress_shards.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(u64),
                                             ctypes.POINTER(DSegmentT), i32, ctypes.c_uint32, vp, vp]
    lib.zipccl_decompress_accumulate.restype = i32
    lib.zipccl_decompress_accumulate.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(u64), i32,
                                                 u64, vp, vp, vp, vp]
    lib.zipccl_decompress_accumulate_chunks.restype = i32
    lib.zipccl_decompress_accumulate_chunks.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(u64),
                                                        i32, u64, u64, vp, vp, vp, vp]
    lib.zipccl_profile_scratch_size.restype = u64
    lib.zipccl_profile_scratch_size.argtypes = [u64, i32]
    lib.zipccl_profile_codec.restype = i32
    lib.zipccl_profile_codec.argtypes = [vp, u64, PlanT, i32, vp, u64, vp, ctypes.POINTER(CodecProfileT)]
    lib.zipccl_rs_choose.restype = i32
    lib.zipccl_rs_choose.argtypes = [ctypes.POINTER(CodecProfileT), ctypes.POINTER(LinkT), i32, u64,
                                     ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(ctypes.c_double)]
    lib.zipccl_moe_sort.restype = i32
    lib.zipccl_moe_sort.argtypes = [vp, i32, u64, u64, i32, i32, vp, vp, vp, vp, u64, vp, vp]
    lib.zipccl_moe_dispatch.restype = i32
    lib.zipccl_moe_dispatch.argtypes = [vp, u64, vp, u64, i32, u64, i32, vp, u64, u64, vp, vp]
    lib.zipccl_moe_dispatch_backward.restype = i32
    lib.zipccl_moe_dispatch_backward.argtypes = [vp, u64, u64, vp, u64, i32, u64, i32, vp, u64, vp, vp]
    lib.zipccl_moe_combine.restype = i32
    lib.zipccl_moe_combine.argtypes = [vp, u64, u64, vp, vp, u64, i32, u64, i32, vp, u64, vp, vp]
    lib.zipccl_moe_combine_backward.restype = i32
    lib.zipccl_moe_combine_backward.argtypes = [vp, u64, vp, u64, u64, vp, vp, u64, i32, u64, i32, vp, u64, vp, vp,
                                                vp]
    lib.zipccl_quantize_rows.restype = i32
    lib.zipccl_quantize_rows.argtypes = [vp, u64, u64, u64, vp, i32, vp, u64, u64, vp, vp, vp]
    lib.zipccl_experts_product.restype = i32
    lib.zipccl_experts_product.argtypes = [vp, u64, vp, u64, vp, u64, vp, i32, u64, u64, vp, vp, u64, i32, vp, vp]
    lib.zipccl_moe_gate.restype = i32
    lib.zipccl_moe_gate.argtypes = [vp, i32, u64, u64, i32, vp, i32, i32, vp, vp, vp, vp, vp, vp, u64, vp, vp]
    lib.zipccl_moe_balance.restype = i32
    lib.zipccl_moe_balance.argtypes = [vp, i32, u64, u64, i32, vp, vp, i32, u64, i32, vp, vp, vp, vp, u64, vp, vp]
    lib.zipccl_moe_gate_backward.restype = i32
    lib.zipccl_moe_gate_backward.argtypes = [vp, i32, u64, u64, i32, vp, vp, i32, u64, i32, i32, vp, vp, vp, vp, u64,
                                             vp, vp]
    lib.zipccl_weights4_size.restype = u64
    lib.zipccl_weights4_size.argtypes = [i32, u64, u64]
    lib.zipccl_quantize_weights4.restype = i32
    lib.zipccl_quantize_weights4.argtypes = [vp, u64, i32, u64, u64, u64, vp, vp, i32, vp]
    lib.zipccl_experts_product4.restype = i32
    lib.zipccl_experts_product4.argtypes = [vp, u64, u64, vp, u64, vp, vp, i32, u64, i32, u64, u64, vp, vp, u64, i32,
                                            vp, vp]
    lib.zipccl_pipeline_scratch_size.restype = u64
    lib.zipccl_pipeline_scratch_size.argtypes = [i32, u64]
    lib.zipccl_pipeline_create.restype = i32
    lib.zipccl_pipeline_create.argtypes = [i32, u64, vp, u64, vp, vp, ctypes.POINTER(vp)]
    lib.zipccl_pipeline_reduce.restype = i32
    lib.zipccl_pipeline_reduce.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(PlanT), u64, vp, vp, vp]
    lib.zipccl_pipeline_destroy.restype = None
    lib.zipccl_pipeline_destroy.argtypes = [vp]
    return lib


_lib = _load()


def lib() -> ctypes.CDLL:
    return _lib


def _check(rc: int, what: str):
    if rc != OK:
        raise ZipcclError(rc, what)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


try:   # the handle alone: building a torch.cuda.Stream takes 3 us, as long as a launch
    from torch._C import _cuda_getCurrentRawStream as _raw_stream
    from torch._C import _cuda_getDevice as _current_device
except ImportError:   # a torch that has no such call (one built without GPU support)
    _current_device = torch.cuda.current_device

    def _raw_stream(device: int) -> int:
        return torch.cuda.current_stream(device).cuda_stream


def _stream(stream) -> int | None:
    if stream is None:
        return _raw_stream(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


# ------------------------------------------------------------------------------------
# C ABI mirrors
# ------------------------------------------------------------------------------------
def plan(sigma: float | None = None, table=None) -> PlanT:
    """zipccl_plan: sigma -> 7-exponent window, or a given table (sorted)."""
    out = PlanT()
    if table is not None:
        arr = (ctypes.c_uint8 * 7)(*[int(v) for v in table]) if len(table) == 7 else None
        if arr is None:
            raise ZipcclError(ERR_INVALID, "zipccl_plan")
        _check(_lib.zipccl_plan(0.0, arr, ctypes.byref(out)), "zipccl_plan")
    else:
        _check(_lib.zipccl_plan(float(sigma), None, ctypes.byref(out)), "zipccl_plan")
    return out


def plan_many(sigmas):
    """zipccl_plan_many: one plan per sigma, as a ctypes array of PlanT."""
    n = len(sigmas)
    sig = (ctypes.c_double * max(n, 1))(*[float(x) for x in sigmas])
    out = (PlanT * max(n, 1))()
    _check(_lib.zipccl_plan_many(sig, n, out), "zipccl_plan_many")
    return out


def static_size(n: int) -> int:
    return int(_lib.zipccl_static_size(n))


def compressed_size(n: int, n_esc: int) -> int:
    return int(_lib.zipccl_compressed_size(n, n_esc))


def workspace_size(total_n: int, nseg: int) -> int:
    return int(_lib.zipccl_workspace_size(total_n, nseg))


def compress(segments, static_out, esc_out, workspace, n_esc_out=None, status=None, stream=None,
             esc_cap: int | None = None):
    """zipccl_compress.  segments: list of (bf16 device tensor, PlanT)."""
    nseg = len(segments)
    arr = (SegmentT * max(nseg, 1))()
    for k, (t, p) in enumerate(segments):
        arr[k].src = _ptr(t) if t.numel() else None
        arr[k].n = t.numel()
        arr[k].plan = p
    cap = _nbytes(esc_out) if esc_cap is None else esc_cap
    rc = _lib.zipccl_compress(arr, nseg, _ptr(static_out), _nbytes(static_out), _ptr(esc_out), cap,
                              _ptr(workspace), _nbytes(workspace), _ptr(n_esc_out), _ptr(status), _stream(stream))
    _check(rc, "zipccl_compress")


NOALLOC_MAX_VALUES = 1 << 26


def compress_noalloc(segments, static_out, esc_out, n_esc_out=None, status=None, stream=None,
                     esc_cap: int | None = None):
    """zipccl_compress_noalloc: zipccl_compress with the library's static device workspace."""
    nseg = len(segments)
    arr = (SegmentT * max(nseg, 1))()
    for k, (t, p) in enumerate(segments):
        arr[k].src = _ptr(t) if t.numel() else None
        arr[k].n = t.numel()
        arr[k].plan = p
    cap = _nbytes(esc_out) if esc_cap is None else esc_cap
    rc = _lib.zipccl_compress_noalloc(arr, nseg, _ptr(static_out), _nbytes(static_out), _ptr(esc_out), cap,
                                      _ptr(n_esc_out), _ptr(status), _stream(stream))
    _check(rc, "zipccl_compress_noalloc")


class PreparedCompressChunks:
    """A zipccl_compress_chunks call over fixed buffers, marshalled once.  chunks: a list
    of per-chunk lists of bf16 device tensors (the same number in each); static_outs /
    esc_outs: per-chunk uint8 device tensors.  run(plans) uses plans[i] for segment i of
    every chunk.  esc_caps: per-chunk escape capacities (default: each buffer's size)."""

    def __init__(self, chunks, static_outs, esc_outs, workspace, n_esc_out=None, status=None, stream=None,
                 esc_caps=None):
        self.nchunks, self.nseg = len(chunks), len(chunks[0])
        self._arr = (SegmentT * (self.nchunks * self.nseg))()
        for k, tensors in enumerate(chunks):
            if len(tensors) != self.nseg:
                raise ValueError("every chunk needs the same number of segments")
            for i, t in enumerate(tensors):
                e = self._arr[k * self.nseg + i]
                e.src = _ptr(t) if t.numel() else None
                e.n = t.numel()
        C = self.nchunks
        sp = (ctypes.c_void_p * C)(*[_ptr(t) for t in static_outs])
        sc = (ctypes.c_uint64 * C)(*[_nbytes(t) for t in static_outs])
        ep = (ctypes.c_void_p * C)(*[_ptr(t) for t in esc_outs])
        ec = (ctypes.c_uint64 * C)(*([_nbytes(t) for t in esc_outs] if esc_caps is None else esc_caps))
        self._args = (sp, sc, ep, ec, _ptr(workspace), _nbytes(workspace), _ptr(n_esc_out), _ptr(status),
                      _stream(stream))
        self._keep = (chunks, static_outs, esc_outs, workspace, n_esc_out, status)

    def run(self, plans):
        for k in range(self.nchunks):
            for i in range(self.nseg):
                self._arr[k * self.nseg + i].plan = plans[i]
        _check(_lib.zipccl_compress_chunks(self._arr, self.nseg, self.nchunks, *self._args), "zipccl_compress_chunks")


def _segment_array(tensors):
    arr = (SegmentT * max(len(tensors), 1))()
    for k, t in enumerate(tensors):
        arr[k].src = _ptr(t) if t.numel() else None
        arr[k].n = t.numel()
    return arr


def estimate_workspace_size(nseg: int) -> int:
    return int(_lib.zipccl_estimate_workspace_size(nseg))


def estimate_plans(tensors, plans_dev, workspace, stride: int = 16, stream=None):
    """zipccl_estimate_plans: plans_dev, a uint8 device tensor of 8 * len(tensors) bytes,
    receives one plan per bf16 tensor (PlanT.from_buffer_copy on its bytes reads them);
    workspace, a device tensor of at least estimate_workspace_size(len(tensors)) bytes."""
    _check(_lib.zipccl_estimate_plans(_segment_array(tensors), len(tensors), stride, _ptr(plans_dev),
                                      _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "zipccl_estimate_plans")


def compress_device_plans(tensors, plans_dev, static_out, esc_out, workspace, n_esc_out=None, status=None,
                          stream=None, esc_cap: int | None = None):
    """zipccl_compress_device_plans: tensors coded by the plans in plans_dev (device)."""
    cap = _nbytes(esc_out) if esc_cap is None else esc_cap
    _check(_lib.zipccl_compress_device_plans(_segment_array(tensors), len(tensors), _ptr(plans_dev),
                                             _ptr(static_out), _nbytes(static_out), _ptr(esc_out), cap,
                                             _ptr(workspace), _nbytes(workspace), _ptr(n_esc_out), _ptr(status),
                                             _stream(stream)), "zipccl_compress_device_plans")


def compress_gather(segments, static_out, esc_out, workspace, n_esc_out=None, status=None, stream=None,
                    esc_cap: int | None = None):
    """zipccl_compress_gather.  segments: list of (matrix, rows, plan): matrix a 2-D bf16
    device tensor (row-major, contiguous), rows a 1-D int32 device tensor of row indices."""
    PreparedCompressGather(segments, static_out, esc_out, workspace, n_esc_out, status, stream, esc_cap).run()


class PreparedCompressGather:
    """A zipccl_compress_gather call over fixed buffers, marshalled once; run([plans])
    makes it."""

    def __init__(self, segments, static_out, esc_out, workspace, n_esc_out=None, status=None, stream=None,
                 esc_cap: int | None = None):
        nseg = len(segments)
        self._arr = (GatherSegmentT * max(nseg, 1))()
        for k, (m, rows, p) in enumerate(segments):
            if m.dim() != 2 or not m.is_contiguous() or rows.dtype != torch.int32:
                raise ValueError("compress_gather takes a contiguous 2-D matrix and int32 row indices")
            self._arr[k].src = _ptr(m) if m.numel() else None
            self._arr[k].src_rows = m.shape[0]
            self._arr[k].row_len = m.shape[1]
            self._arr[k].rows = _ptr(rows) if rows.numel() else None
            self._arr[k].nrows = rows.numel()
            self._arr[k].plan = p
        cap = _nbytes(esc_out) if esc_cap is None else esc_cap
        self._args = (self._arr, nseg, _ptr(static_out), _nbytes(static_out), _ptr(esc_out), cap, _ptr(workspace),
                      _nbytes(workspace), _ptr(n_esc_out), _ptr(status), _stream(stream))
        self._keep = (segments, static_out, esc_out, workspace, n_esc_out, status)

    def run(self, plans=None):
        """Makes the call; `plans`, if given, replaces the segments' plans first."""
        if plans is not None:
            for k, p in enumerate(plans):
                self._arr[k].plan = p
        _check(_lib.zipccl_compress_gather(*self._args), "zipccl_compress_gather")


def decompress(static_in, esc_in, dsts, status=None, stream=None, static_bytes=None, esc_bytes=None):
    """zipccl_decompress.  dsts: list of bf16 device tensors (their numel is n)."""
    nseg = len(dsts)
    arr = (DSegmentT * max(nseg, 1))()
    for k, t in enumerate(dsts):
        arr[k].dst = _ptr(t) if t.numel() else None
        arr[k].n = t.numel()
    sb = _nbytes(static_in) if static_bytes is None else static_bytes
    eb = (_nbytes(esc_in) if esc_in is not None else 0) if esc_bytes is None else esc_bytes
    rc = _lib.zipccl_decompress(_ptr(static_in), sb, _ptr(esc_in), eb, arr, nseg, _ptr(status), _stream(stream))
    _check(rc, "zipccl_decompress")


SHARDS_ESC_AT_FIRST = 1


def decompress_shards(static_ins, esc_ins, dsts, status=None, stream=None, esc_bytes=None, flags=0):
    """zipccl_decompress_shards.  static_ins / esc_ins: per-shard device tensors or raw
    device addresses (int; an escape entry may be None); dsts: bf16 device tensors, one
    per shard (their numel is n); esc_bytes: per-shard escape buffer sizes; flags:
    SHARDS_ESC_AT_FIRST when each escape buffer starts at its shard's first escape."""
    PreparedDecompressShards(static_ins, esc_ins, dsts, status, stream, esc_bytes, flags).run()


class PreparedDecompressShards:
    """A zipccl_decompress_shards call over fixed buffers, marshalled once; run() makes it."""

    def __init__(self, static_ins, esc_ins, dsts, status=None, stream=None, esc_bytes=None, flags=0):
        nseg = len(dsts)
        sp = (ctypes.c_void_p * nseg)(*[_ptr(t) for t in static_ins])
        ep = (ctypes.c_void_p * nseg)(*[_ptr(t) for t in esc_ins])
        if esc_bytes is None:
            esc_bytes = [_nbytes(t) if t is not None else 0 for t in esc_ins]
        eb = (ctypes.c_uint64 * nseg)(*[int(v) for v in esc_bytes])
        arr = (DSegmentT * max(nseg, 1))()
        for k, t in enumerate(dsts):
            arr[k].dst = _ptr(t) if t.numel() else None
            arr[k].n = t.numel()
        self._args = (sp, ep, eb, arr, nseg, flags, _ptr(status), _stream(stream))
        self._keep = (static_ins, esc_ins, dsts, status)

    def run(self):
        _check(_lib.zipccl_decompress_shards(*self._args), "zipccl_decompress_shards")


def decompress_accumulate(static_ins, esc_ins, n: int, local, dst, status=None, stream=None, esc_bytes=None):
    """zipccl_decompress_accumulate.  static_ins / esc_ins: per-peer device tensors or
    raw device addresses (int); esc_bytes: per-peer escape buffer sizes."""
    P = len(static_ins)
    sp = (ctypes.c_void_p * P)(*[_ptr(t) for t in static_ins])
    ep = (ctypes.c_void_p * P)(*[_ptr(t) for t in esc_ins])
    if esc_bytes is None:
        esc_bytes = [_nbytes(t) for t in esc_ins]
    eb = (ctypes.c_uint64 * P)(*[int(v) for v in esc_bytes])
    rc = _lib.zipccl_decompress_accumulate(sp, ep, eb, P, n, _ptr(local), _ptr(dst), _ptr(status), _stream(stream))
    _check(rc, "zipccl_decompress_accumulate")


class PreparedCompress:
    """A zipccl_compress call over fixed buffers: the segment table and every other
    argument are marshalled once; run(plans) writes this call's plans into the table and
    makes the call (for loops that compress the same buffers with new plans)."""

    def __init__(self, tensors, static_out, esc_out, workspace, n_esc_out=None, status=None, stream=None,
                 esc_cap=None):
        self.n = len(tensors)
        self._arr = (SegmentT * max(self.n, 1))()
        for k, t in enumerate(tensors):
            self._arr[k].src = _ptr(t) if t.numel() else None
            self._arr[k].n = t.numel()
        cap = _nbytes(esc_out) if esc_cap is None else esc_cap
        self._args = (_ptr(static_out), _nbytes(static_out), _ptr(esc_out), cap, _ptr(workspace),
                      _nbytes(workspace), _ptr(n_esc_out), _ptr(status), _stream(stream))
        self._keep = (tensors, static_out, esc_out, workspace, n_esc_out, status)

    def run(self, plans):
        arr = self._arr
        for k in range(self.n):
            arr[k].plan = plans[k]
        _check(_lib.zipccl_compress(arr, self.n, *self._args), "zipccl_compress")


class PreparedDecompress:
    """A zipccl_decompress call over fixed buffers, marshalled once; run() makes it."""

    def __init__(self, static_in, esc_in, dsts, status=None, stream=None, static_bytes=None, esc_bytes=None):
        self.n = len(dsts)
        self._arr = (DSegmentT * max(self.n, 1))()
        for k, t in enumerate(dsts):
            self._arr[k].dst = _ptr(t) if t.numel() else None
            self._arr[k].n = t.numel()
        sb = _nbytes(static_in) if static_bytes is None else static_bytes
        eb = (_nbytes(esc_in) if esc_in is not None else 0) if esc_bytes is None else esc_bytes
        self._args = (_ptr(static_in), sb, _ptr(esc_in), eb, self._arr, self.n, _ptr(status), _stream(stream))
        self._keep = (static_in, esc_in, dsts, status)

    def run(self):
        _check(_lib.zipccl_decompress(*self._args), "zipccl_decompress")


class PreparedAccumulate:
    """A zipccl_decompress_accumulate call over fixed buffers, marshalled once."""

    def __init__(self, static_ins, esc_ins, n: int, local, dst, status=None, stream=None, esc_bytes=None):
        P = len(static_ins)
        self._sp = (ctypes.c_void_p * P)(*[_ptr(t) for t in static_ins])
        self._ep = (ctypes.c_void_p * P)(*[_ptr(t) for t in esc_ins])
        if esc_bytes is None:
            esc_bytes = [_nbytes(t) for t in esc_ins]
        self._eb = (ctypes.c_uint64 * P)(*[int(v) for v in esc_bytes])
        self._args = (self._sp, self._ep, self._eb, P, n, _ptr(local), _ptr(dst), _ptr(status), _stream(stream))
        self._keep = (static_ins, esc_ins, local, dst, status)

    def run(self):
        _check(_lib.zipccl_decompress_accumulate(*self._args), "zipccl_decompress_accumulate")


def pipeline_scratch_size(npeers: int, chunk: int) -> int:
    return int(_lib.zipccl_pipeline_scratch_size(npeers, chunk))


class PreparedAccumulateChunks:
    """A zipccl_decompress_accumulate_chunks call over fixed buffers, marshalled once.
    static_ins / esc_ins / esc_bytes: per-(chunk, peer) entries, chunk-major (device
    tensors or raw addresses); n values of local and dst in chunks of `chunk`."""

    def __init__(self, static_ins, esc_ins, npeers: int, chunk: int, n: int, local, dst, status=None,
                 stream=None, esc_bytes=None):
        m = len(static_ins)
        sp = (ctypes.c_void_p * m)(*[_ptr(t) for t in static_ins])
        ep = (ctypes.c_void_p * m)(*[_ptr(t) for t in esc_ins])
        if esc_bytes is None:
            esc_bytes = [_nbytes(t) for t in esc_ins]
        eb = (ctypes.c_uint64 * m)(*[int(v) for v in esc_bytes])
        self._args = (sp, ep, eb, npeers, chunk, n, _ptr(local), _ptr(dst), _ptr(status), _stream(stream))
        self._keep = (static_ins, esc_ins, local, dst, status)

    def run(self):
        _check(_lib.zipccl_decompress_accumulate_chunks(*self._args), "zipccl_decompress_accumulate_chunks")


def profile_codec(sample, plan, npeers: int, stream=None) -> CodecProfileT:
    """zipccl_profile_codec on a bf16 device tensor (scratch allocated with torch)."""
    n = sample.numel()
    size = _lib.zipccl_profile_scratch_size(n, npeers)
    scratch = torch.empty(max(size, 1), dtype=torch.uint8, device=sample.device)
    out = CodecProfileT()
    _check(_lib.zipccl_profile_codec(_ptr(sample), n, plan, npeers, _ptr(scratch), size, _stream(stream),
                                     ctypes.byref(out)), "zipccl_profile_codec")
    return out


def rs_choose(profile: CodecProfileT, link: LinkT, ranks: int, nbytes: int):
    """zipccl_rs_choose: (use_codec, native_us, zipped_us)."""
    use = ctypes.c_int32()
    t_n, t_z = ctypes.c_double(), ctypes.c_double()
    _check(_lib.zipccl_rs_choose(ctypes.byref(profile), ctypes.byref(link), ranks, nbytes, ctypes.byref(use),
                                 ctypes.byref(t_n), ctypes.byref(t_z)), "zipccl_rs_choose")
    return bool(use.value), t_n.value, t_z.value


class Pipeline:
    """zipccl_pipeline_*: chunked compress (stream_a) -> decode-accumulate (stream_b)."""

    def __init__(self, npeers: int, chunk: int, stream_a, stream_b, device=None):
        self.npeers, self.chunk = npeers, chunk
        size = pipeline_scratch_size(npeers, chunk)
        self.scratch = torch.zeros(size, dtype=torch.uint8, device=device or "cuda")
        h = ctypes.c_void_p()
        rc = _lib.zipccl_pipeline_create(npeers, chunk, _ptr(self.scratch), size, _stream(stream_a),
                                         _stream(stream_b), ctypes.byref(h))
        _check(rc, "zipccl_pipeline_create")
        self._h = h
        self.stream_a, self.stream_b = stream_a, stream_b

    def reduce(self, peer_src, plans, local, dst, status=None):
        P = self.npeers
        sp = (ctypes.c_void_p * P)(*[_ptr(t) for t in peer_src])
        pl = (PlanT * P)(*plans)
        rc = _lib.zipccl_pipeline_reduce(self._h, sp, pl, local.numel(), _ptr(local), _ptr(dst), _ptr(status))
        _check(rc, "zipccl_pipeline_reduce")

    def close(self):
        # at interpreter exit the module globals may already be gone
        if getattr(self, "_h", None) and _lib is not None:
            _lib.zipccl_pipeline_destroy(self._h)
        self._h = None

    def __del__(self):
        self.close()


# ------------------------------------------------------------------------------------
# mixture-of-experts rows: the tensors of a call are on one GPU, and the call is enqueued there
# ------------------------------------------------------------------------------------
_VALUES = {torch.bfloat16: BF16, torch.float32: FP32}
_IDS = {torch.int32: 4, torch.int64: 8}
_BF16_ONLY = {torch.bfloat16: BF16}
_INT8 = {torch.int8: 1}
_INT32 = {torch.int32: 4}
_BYTES = (torch.bool, torch.uint8)


def _matrix(t, what, kinds=_VALUES):
    """(address, rows, row length, row stride, kind) of a 2-D row-major tensor; kinds: the
    types it may have, and what the library calls them."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} is a 2-D tensor")
    rows, length = shape
    if t.is_contiguous():
        stride = length
    else:
        stride, step = t.stride()
        if rows > 0 and length > 1 and step != 1:
            raise ValueError(f"{what} has contiguous rows")
        if rows > 1 and stride < length:
            raise ValueError(f"{what} has rows that do not overlap")
        stride = max(stride, length)
    kind = kinds.get(t.dtype)
    if kind is None:
        raise ValueError(f"{what} is {t.dtype}")
    return t.data_ptr(), rows, length, stride, kind


def _holds_padding(t, stride, row_len, what, written):
    """Refuses 8-bit rows whose values from row_len up to the next multiple of ROW_PAD, which
    the kernels touch, are not the rows' own.  They are where the view's rows hold them; else
    they lie past the view's columns: inside the tensor's memory, and, where they are written,
    in the 128 bytes that the row's end began (rows that start at a multiple of ROW_PAD)."""
    rows, wide = t.shape
    padded = -(-row_len // ROW_PAD) * ROW_PAD
    if rows == 0 or wide >= padded:
        return
    first = t.storage_offset()
    if first + (rows - 1) * stride + padded > t.untyped_storage().nbytes() or (written and first % ROW_PAD):
        raise ValueError(f"{what}'s rows hold their padding: {padded} values")


def _vector(t, n, dtype, what):
    """Address of a contiguous tensor of at least n values."""
    if t.dtype is dtype and t.is_contiguous() and t.numel() >= n:
        return t.data_ptr()
    raise ValueError(f"{what} is a contiguous {dtype} tensor of at least {n} values")


def _slots(slots, tokens):
    """(address, top_k) of tokens x top_k slots."""
    if slots.dtype is torch.int32 and slots.is_contiguous():
        shape = slots.shape
        if len(shape) == 2 and shape[0] == tokens:
            return slots.data_ptr(), shape[1]
    raise ValueError(f"slots is a contiguous int32 tensor, tokens x top_k, of {tokens} tokens")


def _differ(a, b, what):
    raise ValueError(f"{what} agree: {a} and {b}")


def _enqueue(call, tensors, status, stream, args):
    """The library's call(*args, status, stream) on the GPU that holds the tensors, on that
    GPU's current stream if none is given."""
    device = _current_device()
    for t in tensors:
        if t.get_device() != device:
            device = _one_device(tensors)
            with torch.cuda.device(device):
                return _enqueue_on(device, call, status, stream, args)
    if status is None and stream is None:
        rc = call(*args, None, _raw_stream(device))
        if rc != OK:
            raise ZipcclError(rc, call.__name__)
    else:
        _enqueue_on(device, call, status, stream, args)


def _one_device(tensors) -> int:
    """The GPU that holds every tensor (pinned host memory is any GPU's)."""
    found = {t.get_device() for t in tensors if not (t.device.type == "cpu" and t.is_pinned())}
    if len(found) > 1 or -1 in found:
        raise ValueError("the tensors are on one GPU")
    return found.pop() if found else _current_device()


def _enqueue_on(device, call, status, stream, args):
    if status is not None and not isinstance(status, int):
        if status.nbytes < 4 or (status.element_size() < 4 and not status.is_contiguous()):
            raise ValueError("status is a tensor whose first 4 bytes are its own")
        other = status.get_device()
        if other != device and _one_device([status]) != device:
            _differ(other, device, "the GPUs of status and the other tensors")
        status = status.data_ptr()
    if stream is None:
        stream = _raw_stream(device)
    elif not isinstance(stream, int):
        other = getattr(stream, "device_index", device)
        if other != device:
            _differ(other, device, "the GPUs of the stream and the tensors")
        stream = stream.cuda_stream
    _check(call(*args, status, stream), call.__name__)


def moe_sort(experts, num_experts: int, offsets, rows, slots, workspace, status=None, stream=None):
    """zipccl_moe_sort.  experts: int32 or int64 device tensor, tokens x top_k (a router's
    top-k indices; negative: dropped).  Writes offsets (int32, num_experts + 1), rows
    (int32, tokens * top_k) and slots (int32, tokens x top_k).  workspace:
    MOE_SORT_WORKSPACE_BYTES device bytes."""
    ep, T, K, stride, id_bytes = _matrix(experts, "experts", _IDS)
    if not workspace.is_contiguous():
        raise ValueError("workspace is contiguous")
    n = T * K
    _enqueue(_lib.zipccl_moe_sort, (experts, offsets, rows, slots, workspace), status, stream,
             (ep, id_bytes, stride, T, K, num_experts,
              _vector(offsets, num_experts + 1, torch.int32, "offsets"), _vector(rows, n, torch.int32, "rows"),
              _vector(slots, n, torch.int32, "slots"), workspace.data_ptr(), workspace.nbytes))


def moe_dispatch(x, slots, y, status=None, stream=None):
    """zipccl_moe_dispatch: y[slots[t, k]] = x[t]."""
    xp, T, H, xs, kind = _matrix(x, "x")
    yp, M, yh, ys, y_kind = _matrix(y, "y")
    if H != yh or kind != y_kind:
        _differ((H, x.dtype), (yh, y.dtype), "the rows of x and y")
    sp, K = _slots(slots, T)
    _enqueue(_lib.zipccl_moe_dispatch, (x, slots, y), status, stream,
             (xp, xs, sp, T, K, H, kind, yp, M, ys))


def moe_dispatch_backward(dy, slots, dx, status=None, stream=None):
    """zipccl_moe_dispatch_backward: dx[t] = sum over k of dy[slots[t, k]]."""
    yp, M, H, ys, kind = _matrix(dy, "dy")
    xp, T, xh, xs, x_kind = _matrix(dx, "dx")
    if H != xh or kind != x_kind:
        _differ((H, dy.dtype), (xh, dx.dtype), "the rows of dy and dx")
    sp, K = _slots(slots, T)
    _enqueue(_lib.zipccl_moe_dispatch_backward, (dy, slots, dx), status, stream,
             (yp, M, ys, sp, T, K, H, kind, xp, xs))


def moe_combine(y, slots, weights, out, status=None, stream=None):
    """zipccl_moe_combine: out[t] = sum over k of weights[t, k] * y[slots[t, k]] (weights
    float32, or None for 1)."""
    yp, M, H, ys, kind = _matrix(y, "y")
    op, T, oh, os_, o_kind = _matrix(out, "out")
    if H != oh or kind != o_kind:
        _differ((H, y.dtype), (oh, out.dtype), "the rows of y and out")
    sp, K = _slots(slots, T)
    wp = None if weights is None else _vector(weights, T * K, torch.float32, "weights")
    _enqueue(_lib.zipccl_moe_combine, (y, slots, out) if weights is None else (y, slots, weights, out), status, stream,
             (yp, M, ys, sp, wp, T, K, H, kind, op, os_))


def moe_combine_backward(dout, y, slots, weights, dy, dweights, status=None, stream=None):
    """zipccl_moe_combine_backward: dy[slots[t, k]] = weights[t, k] * dout[t] and
    dweights[t, k] = <dout[t], y[slots[t, k]]>."""
    gp, T, gh, gs, g_kind = _matrix(dout, "dout")
    yp, M, H, ys, kind = _matrix(y, "y")
    dp, dm, dh, ds, d_kind = _matrix(dy, "dy")
    if H != gh or kind != g_kind:
        _differ((H, y.dtype), (gh, dout.dtype), "the rows of y and dout")
    if M != dm or H != dh or kind != d_kind:
        _differ((M, H, y.dtype), (dm, dh, dy.dtype), "y and dy")
    sp, K = _slots(slots, T)
    _enqueue(_lib.zipccl_moe_combine_backward, (dout, y, slots, weights, dy, dweights), status, stream,
             (gp, gs, yp, M, ys, sp, _vector(weights, T * K, torch.float32, "weights"), T, K, H, kind,
              dp, ds, _vector(dweights, T * K, torch.float32, "dweights")))


def quantize_rows(x, q, scales, slots=None, status=None, stream=None):
    """zipccl_quantize_rows: BF16 rows x to int8 rows q (row stride a multiple of ROW_PAD,
    at least as long as x's rows) with float32 scales, to every slot of a token or, without
    slots, row by row.  q is written up to the next multiple of ROW_PAD: rows of fewer columns
    are taken where they start at a multiple of ROW_PAD in a tensor that goes on that far."""
    xp, T, H, xs, _ = _matrix(x, "x", _BF16_ONLY)
    qp, M, wide, qs, _ = _matrix(q, "q", _INT8)
    if wide < H:
        raise ValueError("q's rows hold x's rows")
    if wide % ROW_PAD:
        _holds_padding(q, qs, H, "q", True)
    sp, K = (None, 1) if slots is None else _slots(slots, T)
    _enqueue(_lib.zipccl_quantize_rows, (x, q, scales) if slots is None else (x, q, scales, slots), status, stream,
             (xp, xs, T, H, sp, K, qp, M, qs, _vector(scales, M, torch.float32, "scales")))


def experts_product(q, scales, w, w_scales, row_len: int, out, offsets=None, status=None, stream=None):
    """zipccl_experts_product.  q: int8 rows with scales, sorted by expert; w: int8,
    experts x outputs x stride (or outputs x stride for one), w_scales float32, experts x
    outputs; row_len: values of a row without its padding; out: rows x outputs, bfloat16
    or float32; offsets: int32, experts + 1 (None: one expert)."""
    qp, M, wide, qs, _ = _matrix(q, "q", _INT8)
    op, om, on, os_, kind = _matrix(out, "out")
    shape = w.shape
    if len(shape) not in (2, 3):
        raise ValueError("w is experts x outputs x row stride")
    E, N, ws = shape if len(shape) == 3 else (1, *shape)
    if om != M or on != N:
        _differ((om, on), (M, N), "out, and q's rows x w's outputs")
    if row_len > wide or row_len > ws:
        raise ValueError("row_len is at most the row length of q and w")
    if wide % ROW_PAD:
        _holds_padding(q, qs, row_len, "q", False)
    if offsets is None:
        tensors, starts = (q, scales, w, w_scales, out), None
    else:
        tensors, starts = (q, scales, w, w_scales, offsets, out), _vector(offsets, E + 1, torch.int32, "offsets")
    _enqueue(_lib.zipccl_experts_product, tensors, status, stream,
             (qp, qs, _vector(scales, M, torch.float32, "scales"), M, _vector(w, 0, torch.int8, "w"), ws,
              _vector(w_scales, E * N, torch.float32, "w_scales"), E, N, row_len, starts, op, os_, kind))


def _mask(mask, tokens):
    """Address of one truth value (or byte) per token."""
    if mask is None:
        return None
    if mask.dtype not in _BYTES or not mask.is_contiguous() or mask.shape != (tokens,):
        raise ValueError(f"mask is a contiguous bool or uint8 tensor of {tokens} values")
    return mask.data_ptr()


def _balance(counts, sums, loss, workspace, num_experts):
    """Addresses of the balance outputs, and the workspace's with its size."""
    if not workspace.is_contiguous():
        raise ValueError("workspace is contiguous")
    return (_vector(counts, num_experts + 1, torch.int32, "counts"), _vector(sums, num_experts, torch.float32, "sums"),
            _vector(loss, 1, torch.float32, "loss"), workspace.data_ptr(), workspace.nbytes)


_NO_BALANCE = (None, None, None, None, 0)


def _there(*tensors):
    return tuple(t for t in tensors if t is not None)


def moe_gate(logits, experts, weights, renormalize: bool = True, mask=None, counts=None, sums=None, loss=None,
             workspace=None, status=None, stream=None):
    """zipccl_moe_gate.  logits: bfloat16 or float32, tokens x experts.  Writes experts (int32,
    tokens x top_k) and weights (float32, as many) and, all four given or none, counts (int32,
    experts + 1), sums (float32, experts) and loss (float32, one value), through workspace
    (MOE_GATE_WORKSPACE_BYTES device bytes).  mask: bool or uint8, one per token."""
    zp, T, E, zs, kind = _matrix(logits, "logits")
    ep, et, K, es, _ = _matrix(experts, "experts", _INT32)
    if et != T or (es != K and T > 1):
        raise ValueError(f"experts is a contiguous int32 tensor, tokens x top_k, of {T} tokens")
    tensors = (logits, experts, weights)
    if counts is not None and sums is not None and loss is not None and workspace is not None:
        balance = _balance(counts, sums, loss, workspace, E)
        tensors += (counts, sums, loss, workspace)
    elif counts is None and sums is None and loss is None and workspace is None:
        balance = _NO_BALANCE
    else:
        raise ValueError("counts, sums, loss and workspace are given together")
    if mask is not None:
        tensors += (mask,)
        mask = _mask(mask, T)
    _enqueue(_lib.zipccl_moe_gate, tensors, status, stream,
             (zp, kind, zs, T, E, mask, K, bool(renormalize), ep,
              _vector(weights, T * K, torch.float32, "weights"), *balance))


def moe_balance(logits, experts, counts, sums, loss, workspace, mask=None, status=None, stream=None):
    """zipccl_moe_balance: counts, sums and loss of given choices (int32 or int64, tokens x
    top_k, negative: dropped)."""
    zp, T, E, zs, kind = _matrix(logits, "logits")
    ep, et, K, es, id_bytes = _matrix(experts, "experts", _IDS)
    if et != T:
        _differ(et, T, "the tokens of experts and logits")
    _enqueue(_lib.zipccl_moe_balance, (logits, experts, counts, sums, loss, workspace, *_there(mask)), status, stream,
             (zp, kind, zs, T, E, _mask(mask, T), ep, id_bytes, es, K, *_balance(counts, sums, loss, workspace, E)))


def moe_gate_backward(logits, experts, dlogits, dweights=None, counts=None, dloss=None, renormalize: bool = True,
                      mask=None, status=None, stream=None):
    """zipccl_moe_gate_backward: dlogits (as logits) for dweights (float32, tokens x top_k) and,
    with the forward call's counts, dloss (float32, one value)."""
    zp, T, E, zs, kind = _matrix(logits, "logits")
    dp, dt, de, ds, d_kind = _matrix(dlogits, "dlogits")
    if (dt, de, d_kind) != (T, E, kind):
        _differ((dt, de, dlogits.dtype), (T, E, logits.dtype), "dlogits and logits")
    ep, et, K, es, id_bytes = _matrix(experts, "experts", _IDS)
    if et != T:
        _differ(et, T, "the tokens of experts and logits")
    _enqueue(_lib.zipccl_moe_gate_backward,
             (logits, experts, dlogits, *_there(dweights, counts, dloss, mask)), status, stream,
             (zp, kind, zs, T, E, _mask(mask, T), ep, id_bytes, es, K, bool(renormalize),
              None if dweights is None else _vector(dweights, T * K, torch.float32, "dweights"),
              None if counts is None else _vector(counts, E + 1, torch.int32, "counts"),
              None if dloss is None else _vector(dloss, 1, torch.float32, "dloss"), dp, ds))


def weights4_size(num_experts: int, outputs: int, row_len: int) -> int:
    """zipccl_weights4_size."""
    return _lib.zipccl_weights4_size(num_experts, outputs, row_len)


def _scales4(scales, E, G, N):
    """(address, kind) of experts x groups x outputs scales."""
    kind = _VALUES.get(scales.dtype)
    if kind is None or not scales.is_contiguous() or scales.numel() != E * G * N:
        raise ValueError(f"scales are contiguous, bfloat16 or float32, {E} x {G} x {N}")
    return scales.data_ptr(), kind


def quantize_weights4(w, group: int, q, scales, stream=None):
    """zipccl_quantize_weights4.  w: bfloat16, experts x outputs x inputs (or outputs x inputs);
    q: uint8, weights4_size bytes; scales: bfloat16 or float32, experts x groups x outputs."""
    shape = w.shape
    if len(shape) not in (2, 3):
        raise ValueError("w is experts x outputs x inputs")
    E, N, H = shape if len(shape) == 3 else (1, *shape)
    if E < 1:
        raise ValueError("w has one expert at least")
    if len(shape) == 3 and E > 1 and N > 1 and w.stride(0) != N * w.stride(1):
        raise ValueError("w's experts follow one another")
    wp, _, _, ws, _ = _matrix(w[0] if len(shape) == 3 else w, "w", _BF16_ONLY)
    if len(shape) == 3 and E > 1 and N == 1:
        ws = w.stride(0)
    if group < 1:
        raise ValueError("group is 32, 64 or a multiple of 128")
    sp, kind = _scales4(scales, E, -(-H // group), N)
    _enqueue_plain(_lib.zipccl_quantize_weights4, (w, q, scales), stream,
                   (wp, ws, E, N, H, group, _vector(q, weights4_size(E, N, H), torch.uint8, "q"), sp, kind))


def _enqueue_plain(call, tensors, stream, args):
    """_enqueue of a call that has no status word."""
    device = _one_device(tensors)
    with torch.cuda.device(device):
        if stream is None:
            stream = _raw_stream(device)
        elif not isinstance(stream, int):
            other = getattr(stream, "device_index", device)
            if other != device:
                _differ(other, device, "the GPUs of the stream and the tensors")
            stream = stream.cuda_stream
        _check(call(*args, stream), call.__name__)


def experts_product4(x, q, scales, group: int, out, rows=None, offsets=None, status=None, stream=None):
    """zipccl_experts_product4.  x: bfloat16, tokens x inputs; q and scales (bfloat16 or
    float32): experts' 4-bit weights as quantize_weights4 writes them; out: rows x outputs,
    bfloat16 or float32, sorted by expert; rows: int32, the token of each row (None: row s of
    x); offsets: int32, experts + 1 (None: one expert)."""
    xp, T, H, xs, _ = _matrix(x, "x", _BF16_ONLY)
    op, M, N, os_, kind = _matrix(out, "out")
    if group < 1 or H < 1:
        raise ValueError("group is 32, 64 or a multiple of 128, rows have a value at least")
    E = 1 if offsets is None else offsets.numel() - 1
    sp, s_kind = _scales4(scales, E, -(-H // group), N)
    size = E * -(-N // TILE4_OUTPUTS) * -(-H // TILE4_INPUTS) * TILE4_BYTES
    if q.dtype is not torch.uint8 or not q.is_contiguous() or q.numel() != size:
        raise ValueError(f"q is a contiguous uint8 tensor of {size} bytes")
    if rows is None and M != T:
        _differ(M, T, "the rows of out and x")
    _enqueue(_lib.zipccl_experts_product4, (x, q, scales, out, *_there(rows, offsets)), status, stream,
             (xp, xs, T, None if rows is None else _vector(rows, M, torch.int32, "rows"), M, q.data_ptr(), sp, s_kind,
              group, E, N, H, None if offsets is None else _vector(offsets, E + 1, torch.int32, "offsets"), op, os_,
              kind))


# ------------------------------------------------------------------------------------
# convenience: buffers from torch, one call each way
# ------------------------------------------------------------------------------------
@dataclass
class Compressed:
    static: torch.Tensor        # uint8, segments back to back
    esc: torch.Tensor           # uint8, escape capacity
    n_esc: torch.Tensor         # uint64 as int64, nseg + 1 entries (last = total)
    sizes: list                 # n of each segment
    status: torch.Tensor        # int32 device status word

    def static_sizes(self):
        return [static_size(n) for n in self.sizes]


def _as_bf16(t):
    return t if t.dtype == torch.bfloat16 else t.view(torch.bfloat16)


def compress_tensors(tensors, plans, esc_cap=None, workspace=None, stream=None) -> Compressed:
    """Allocates outputs with torch and compresses the tensors in one launch."""
    dev = tensors[0].device
    sizes = [t.numel() for t in tensors]
    total_static = sum(static_size(n) for n in sizes)
    static = torch.empty(max(total_static, 1), dtype=torch.uint8, device=dev)
    cap = sum(sizes) if esc_cap is None else esc_cap
    esc = torch.empty(max(cap, 1), dtype=torch.uint8, device=dev)
    n_esc = torch.zeros(len(tensors) + 1, dtype=torch.int64, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = torch.empty(workspace_size(sum(sizes), len(tensors)), dtype=torch.uint8, device=dev)
    compress([(_as_bf16(t), p) for t, p in zip(tensors, plans)], static, esc, workspace, n_esc, status,
             stream=stream, esc_cap=cap)
    return Compressed(static, esc, n_esc, sizes, status)


def decompress_tensors(c: Compressed, out=None, stream=None):
    dev = c.static.device
    if out is None:
        out = [torch.empty(n, dtype=torch.bfloat16, device=dev) for n in c.sizes]
    decompress(c.static, c.esc, out, c.status, stream=stream)
    return out
