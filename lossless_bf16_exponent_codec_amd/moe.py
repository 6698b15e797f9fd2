"""A mixture-of-experts layer's router and row traffic around the codec, from torch: choices,
weights and a balance loss from the router's logits, the choices sorted by expert, tokens
dispatched to their experts' rows and combined back with weights (all differentiable), and, for
serving, experts' weights in 8 or 4 bits (no gradient goes through their products).

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

__all__ = ["Gate", "gate", "balance", "Routing", "route", "dispatch", "combine", "QuantizedRows", "quantize",
           "QuantizedExperts", "pack4", "QuantizedExperts4"]


@dataclass
class Gate:
    """A router's choices (int32, tokens x top_k, largest logit first, -1: none) and their
    weights (float32), and, where they were asked for, the balance loss and the counts (int32:
    choices of each expert, then the number of tokens counted)."""
    experts: torch.Tensor
    weights: torch.Tensor
    loss: torch.Tensor | None = None
    counts: torch.Tensor | None = None


def _balance_buffers(num_experts, device):
    return (torch.empty(num_experts + 1, dtype=torch.int32, device=device),
            torch.empty(num_experts, dtype=torch.float32, device=device),
            torch.empty((), dtype=torch.float32, device=device),
            torch.empty(Z.MOE_GATE_WORKSPACE_BYTES, dtype=torch.uint8, device=device))


def _gate_gradient(logits, experts, mask, renormalize, dweights, counts, dloss, status):
    if dweights is None and dloss is None:
        return None
    dlogits = logits.new_empty(logits.shape)
    Z.moe_gate_backward(logits, experts, dlogits, None if dweights is None else dweights.contiguous(),
                        None if dloss is None else counts, dloss, renormalize, mask, status)
    return dlogits


class _Gate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k, renormalize, mask, with_balance, status):
        dev = logits.device
        experts = torch.empty(logits.shape[0], top_k, dtype=torch.int32, device=dev)
        weights = torch.empty(logits.shape[0], top_k, dtype=torch.float32, device=dev)
        counts, sums, loss, space = _balance_buffers(logits.shape[1], dev) if with_balance else (None,) * 4
        Z.moe_gate(logits, experts, weights, renormalize, mask, counts, sums, loss, space, status)
        ctx.save_for_backward(logits, experts, mask, counts)
        ctx.renormalize, ctx.status = renormalize, status
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(experts, *(() if counts is None else (counts,)))
        return experts, weights, loss, counts

    @staticmethod
    @once_differentiable   # the kernels write past autograd: a second derivative is an error
    def backward(ctx, _, dweights, dloss, __):
        logits, experts, mask, counts = ctx.saved_tensors
        return _gate_gradient(logits, experts, mask, ctx.renormalize, dweights, counts, dloss,
                              ctx.status), None, None, None, None, None


class _Balance(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, experts, mask, status):
        counts, sums, loss, space = _balance_buffers(logits.shape[1], logits.device)
        Z.moe_balance(logits, experts, counts, sums, loss, space, mask, status)
        ctx.save_for_backward(logits, experts, mask, counts)
        ctx.status = status
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(counts)
        return loss, counts

    @staticmethod
    @once_differentiable   # the kernels write past autograd: a second derivative is an error
    def backward(ctx, dloss, _):
        logits, experts, mask, counts = ctx.saved_tensors
        return _gate_gradient(logits, experts, mask, True, None, counts, dloss, ctx.status), None, None, None


def gate(logits: torch.Tensor, top_k: int, renormalize: bool = True, mask=None, balance: bool = False,
         status=None) -> Gate:
    """The top_k experts of each token by its logits (tokens x experts, bfloat16 or float32),
    the lowest number first among equals, and their weights: softmax probabilities, or, with
    renormalize, those over their sum.  Logits of minus infinity close an expert; mask (bool,
    one per token) leaves out tokens that are padding.  balance: also the loss that spreads
    tokens over the experts, experts / (top_k n^2) * sum of counts * probabilities over the n
    tokens counted.  Differentiable in the logits through weights and loss."""
    return Gate(*_Gate.apply(logits, top_k, renormalize, mask, balance, status))


def balance(logits: torch.Tensor, experts: torch.Tensor, mask=None, status=None):
    """(loss, counts) as from gate(balance=True), for choices made otherwise (int32 or int64,
    tokens x top_k, negative ones dropped); the loss is differentiable in the logits."""
    return _Balance.apply(logits, experts, mask, status)


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


_SIGNED = {torch.uint8: torch.int8, torch.uint16: torch.int16, torch.uint32: torch.int32, torch.uint64: torch.int64}


def pack4(values: torch.Tensor) -> torch.Tensor:
    """Whole numbers from -8 to 7 (experts x outputs x inputs, any integer type) as 4-bit tiles of
    16 outputs x 128 inputs: one row of bytes per expert."""
    E, N, H = values.shape
    low, signed = -8, _SIGNED.get(values.dtype)
    if signed is not None:      # the upper half of the type's range is below 0 then
        low, values = 0, values.view(signed)
    if bool(((values < low) | (values > 7)).any()):
        raise ValueError("4-bit values are from -8 to 7")
    tiles, slabs = -(-N // Z.TILE4_OUTPUTS), -(-H // Z.TILE4_INPUTS)
    v = torch.zeros(E, tiles * Z.TILE4_OUTPUTS, slabs * Z.TILE4_INPUTS, dtype=torch.uint8, device=values.device)
    v[:, :N, :H] = (values & 15).to(torch.uint8)
    v = v.view(E, tiles, 16, slabs, 4, 4, 4, 2)   # ..., output, slab, dword, quarter, byte, half
    return (v[..., 0] | v[..., 1] << 4).permute(0, 1, 3, 5, 2, 4, 6).reshape(E, -1)


class QuantizedExperts4:
    """Weights of all experts (experts x outputs x inputs, BF16) laid out once in 4 bits with a
    scale for each output and group of inputs.  Calling it multiplies BF16 rows: each row's
    token is looked up in x, or, by_expert, x's rows are sorted by expert already."""

    def __init__(self, weights: torch.Tensor, group: int = 128, scale_dtype=torch.bfloat16):
        self.experts, self.outputs, self.inputs = weights.shape
        self.group = group
        if group < 1:
            raise ValueError("group is 32, 64 or a multiple of 128")
        self.q = torch.empty(self.experts, Z.weights4_size(1, self.outputs, self.inputs), dtype=torch.uint8,
                             device=weights.device)
        self.scales = torch.empty(self.experts, -(-self.inputs // group), self.outputs, dtype=scale_dtype,
                                  device=weights.device)
        Z.quantize_weights4(weights, group, self.q, self.scales)

    @classmethod
    def of(cls, values: torch.Tensor, scales: torch.Tensor, group: int):
        """From 4-bit values (experts x outputs x inputs, -8 to 7) and scales (experts x outputs x
        groups, BF16 or FP32) that exist already."""
        self = cls.__new__(cls)
        self.experts, self.outputs, self.inputs = values.shape
        if group < 1 or scales.shape != (self.experts, self.outputs, -(-self.inputs // group)):
            raise ValueError(f"scales are {tuple(scales.shape)}, values {tuple(values.shape)} in groups of {group}")
        self.group, self.q, self.scales = group, pack4(values), scales.transpose(1, 2).contiguous()
        return self

    def __call__(self, x: torch.Tensor, routing: Routing, nrows: int | None = None, by_expert: bool = False,
                 dtype=torch.bfloat16, status=None) -> torch.Tensor:
        """nrows: rows of the result (default: the kept choices where splits() has counted them,
        else all choices; by_expert: x's rows).  Those that no choice has are not set."""
        if x.shape[1] != self.inputs:
            raise ValueError(f"rows of {x.shape[1]} values, experts of {self.inputs} inputs")
        if routing.offsets.numel() != self.experts + 1:
            raise ValueError(f"{routing.offsets.numel()} offsets, {self.experts} experts")
        if by_expert:
            nrows = x.shape[0]
        elif nrows is None:
            nrows = routing.rows.numel() if routing.kept is None else routing.kept
        out = torch.empty(nrows, self.outputs, dtype=dtype, device=x.device)
        Z.experts_product4(x, self.q, self.scales, self.group, out, rows=None if by_expert else routing.rows,
                           offsets=routing.offsets, status=status)
        return out
