"""A mixture-of-experts layer's row traffic around the codec, from torch: a router's choices
sorted by expert, tokens dispatched to their experts' rows and combined back with weights
(differentiable), and experts' weights in 8 bits.

Each step is one call of the same name in `zipccl`; this module adds the buffers and the
gradients (of first order).  A status word (int32, on the device) given to a step takes the
bits that its calls set, those of its gradient among them: STATUS_BAD_INDEX for a choice that
was dropped because its expert or its row is out of range.  `examples/moe_exchange.py` runs
the whole path, the compressed exchange between ranks included.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch
from torch.autograd.function import once_differentiable

from . import zipccl as Z

__all__ = ["Routing", "route", "dispatch", "combine", "QuantizedRows", "quantize", "QuantizedExperts"]


@dataclass
class Routing:
    """Choices sorted by expert: rows[offsets[e]:offsets[e + 1]] are the tokens of expert
    e's rows, slots[t, k] the row of token t's k-th choice (-1: dropped).  The tensors are
    one sort's: another sort makes another routing."""
    offsets: torch.Tensor
    rows: torch.Tensor
    slots: torch.Tensor
    kept: int | None = None   # number of rows, once splits() has brought it to the host

    def splits(self) -> list:
        """The offsets on the host (waits for the sort): sizes of buffers and of the
        all-to-all.  The last one is the number of rows."""
        ends = self.offsets.tolist()
        self.kept = ends[-1]
        return ends


def route(experts: torch.Tensor, num_experts: int, status=None) -> Routing:
    """Sorts a router's choices (tokens x top_k expert numbers, negative ones dropped)."""
    dev, i32 = experts.device, torch.int32
    r = Routing(torch.empty(num_experts + 1, dtype=i32, device=dev), torch.empty(experts.numel(), dtype=i32, device=dev),
                torch.empty(experts.shape, dtype=i32, device=dev))
    space = torch.empty(Z.MOE_SORT_WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
    Z.moe_sort(experts, num_experts, r.offsets, r.rows, r.slots, space, status)
    return r


# Bytes of rows from which on those that no choice has are cleared apart.  A dispatch of BF16
# rows of 7168 to 4 rows each, in us, with the count on the host, with all rows cleared, and with
# those past the count: 128 MB 26, 44, 54; 256 MB 49, 83, 81; 512 MB 96, 181, 133; 1.9 GB 428, 738, 511.
CLEAR_APART = 256 << 20


def _cleared(like, nrows, offsets, kept):
    """nrows rows as long as `like`'s, zero from the kept count on, the others not set.

    Where the host has no count, the device's is not waited for: small buffers are cleared
    whole, of large ones the rows past the count are those to which tokens of zeros go."""
    length = like.shape[1]
    if kept is None and nrows * length * like.element_size() < CLEAR_APART:
        return like.new_zeros(nrows, length)
    y = like.new_empty(nrows, length)
    if kept is None:
        places = torch.arange(-(-nrows // Z.MAX_TOP_K) * Z.MAX_TOP_K, dtype=torch.int32, device=like.device)
        places = torch.where((places >= offsets[-1]) & (places < nrows), places, -1).view(-1, Z.MAX_TOP_K)
        Z.moe_dispatch(like.new_zeros(places.shape[0], length), places, y)
    elif kept < nrows:
        y[kept:].zero_()
    return y


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, slots, nrows, offsets, kept, status):
        ctx.save_for_backward(slots)
        ctx.status = status
        y = _cleared(x, nrows, offsets, kept)
        Z.moe_dispatch(x, slots, y, status)
        return y

    @staticmethod
    @once_differentiable   # the kernels write past autograd: a second derivative is an error
    def backward(ctx, dy):
        slots, = ctx.saved_tensors
        dx = dy.new_empty(slots.shape[0], dy.shape[1])
        Z.moe_dispatch_backward(dy.contiguous(), slots, dx, ctx.status)
        return dx, None, None, None, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, slots, weights, status):
        ctx.save_for_backward(y, slots, weights)
        ctx.status = status
        out = y.new_empty(slots.shape[0], y.shape[1])
        Z.moe_combine(y, slots, weights, out, status)
        return out

    @staticmethod
    @once_differentiable   # the kernels write past autograd: a second derivative is an error
    def backward(ctx, dout):
        y, slots, weights = ctx.saved_tensors
        dy, dw = torch.zeros_like(y), torch.empty_like(weights)   # zeros: rows that no choice names
        Z.moe_combine_backward(dout.contiguous(), y, slots, weights, dy, dw, ctx.status)
        return dy, None, dw, None


def dispatch(x: torch.Tensor, routing: Routing, nrows: int, status=None) -> torch.Tensor:
    """Rows by expert of the tokens x; differentiable in x.  nrows: routing.splits()[-1], or
    a fixed number of rows, of which those that no choice has are zero (they cost least to
    clear after splits())."""
    return _Dispatch.apply(x, routing.slots, nrows, routing.offsets, routing.kept, status)


def combine(y: torch.Tensor, routing: Routing, weights: torch.Tensor, status=None) -> torch.Tensor:
    """Tokens from rows by expert: sums with weights (float32, tokens x top_k);
    differentiable in y and weights."""
    shape, choices = weights.shape, routing.slots.shape   # or any shape with the same order
    if shape.numel() != choices.numel() or (len(shape) == 2 and shape != choices and 1 not in shape):
        raise ValueError(f"weights are {tuple(shape)}, choices are {tuple(choices)}")
    return _Combine.apply(y, routing.slots, weights.contiguous(), status)


@dataclass
class QuantizedRows:
    """8-bit rows (padded to a multiple of 128) and their scales."""
    q: torch.Tensor
    scales: torch.Tensor
    row_len: int


def quantize(x: torch.Tensor, slots=None, nrows: int | None = None, status=None) -> QuantizedRows:
    """BF16 rows in 8 bits: row by row, or each token's to its slots among nrows rows (those
    that no choice has, and their products, are not set)."""
    n, wide = x.shape[0] if slots is None else nrows, -(-x.shape[1] // Z.ROW_PAD) * Z.ROW_PAD
    r = QuantizedRows(torch.empty(n, wide, dtype=torch.int8, device=x.device),
                      torch.empty(n, dtype=torch.float32, device=x.device), x.shape[1])
    Z.quantize_rows(x, r.q, r.scales, slots=slots, status=status)
    return r


class QuantizedExperts:
    """Weights of all experts (experts x outputs x inputs, BF16) laid out once in 8 bits
    with a scale per output channel.  Calling it multiplies rows (of `inputs` values) sorted
    by expert."""

    def __init__(self, weights: torch.Tensor):
        self.experts, self.outputs, self.inputs = weights.shape
        rows = quantize(weights.reshape(-1, self.inputs))
        self.q = rows.q.view(self.experts, self.outputs, -1)
        self.scales = rows.scales.view(self.experts, self.outputs)

    def __call__(self, rows: QuantizedRows, routing: Routing, dtype=torch.bfloat16, status=None) -> torch.Tensor:
        if rows.row_len != self.inputs:
            raise ValueError(f"rows of {rows.row_len} values, experts of {self.inputs} inputs")
        if routing.offsets.numel() != self.experts + 1:
            raise ValueError(f"{routing.offsets.numel()} offsets, {self.experts} experts")
        out = torch.empty(rows.q.shape[0], self.outputs, dtype=dtype, device=rows.q.device)
        Z.experts_product(rows.q, rows.scales, self.q, self.scales, self.inputs, out, offsets=routing.offsets,
                          status=status)
        return out
