"""The expert layer between a dispatch and its combine, and the norm that
makes the next layer's payload (ctypes over ``include/moe_ep.h``).

``expert_sort`` takes the received rows to expert order, ``expert_matmul``
multiplies them by each expert's int8 weights, ``silu_mul_quantize`` is the
gated activation between two such products, ``expert_unsort`` takes weighted
expert rows back to their slots (the combine's input), and ``add_rms_norm``
adds the residual and writes the norm in an 8-bit format: the MXFP8 or
DeepSeekFp8 payload of a dispatch, or int8 rows for ``expert_matmul``.

Everything runs in the gfx950 kernels of ``libmoe_ep.so`` on the stream of
the call (``stream``, or the current stream of the tensors' device), without
synchronisation; outputs that are not given are allocated on that stream, and
given ones are checked and written in place.  Tensors that live on another
stream must be ordered by the caller.  Calls may be captured into a HIP
graph.  A refused call raises ``MoeEpArgError`` (or ``MoeEpError`` with the
library's code) and launches nothing.  Under grad mode an input that asks for
a gradient is refused where the operator has none for it, and so is a given
output that does.
"""
from __future__ import annotations

import functools
import struct
from typing import NamedTuple, Optional

import torch

from .moe_ep import ERR_INVALID_ARG, MoeEpArgError, _check, _need, lib

BF16_ROWS, FP32_ROWS = 0, 1
MAX_SORT_EXPERTS = 4096  # MOE_EP_MAX_SORT_EXPERTS
_INT_MAX = (1 << 31) - 1
NORM_INT8, NORM_MXFP8, NORM_DEEPSEEK_FP8 = 0, 1, 2

_ROW_TYPES = {torch.bfloat16: BF16_ROWS, torch.float32: FP32_ROWS}
# format -> (code, elements of a scale block (0: the row), code dtype, scale dtype)
_NORMS = {"int8": (NORM_INT8, 0, torch.int8, torch.float32),
          "mxfp8": (NORM_MXFP8, 32, torch.float8_e4m3fn, torch.float8_e8m0fnu),
          "deepseek_fp8": (NORM_DEEPSEEK_FP8, 128, torch.float8_e4m3fn, torch.float32)}

# The argument blocks of include/moe_ep.h in native layout.
_SORT = struct.Struct("@PqPqqPqqPPPPPPqqiiiiiiQ")
_UNSORT = struct.Struct("@PPPqPqqiiiiii")
_UNSORT_GRAD = struct.Struct("@PPqPPqPPqiiiiii")
_MATMUL = struct.Struct("@PPPPPPqiiii")
_SILU = struct.Struct("@PPPPqii")
_NORM = struct.Struct("@PPPPPPqiiif")


def _call(entry, block, dev, *values):
    """The entry point with its packed argument block, on the device's current stream."""
    try:
        packed = block.pack(*values)
    except (struct.error, OverflowError) as e:
        _refuse(f"an argument is out of range: {e}")
    _check(entry(packed, _stream_now(dev.index)))


class SortedRows(NamedTuple):
    """Rows in expert order.  ``rows`` [capacity, row] and ``scales`` (scale
    rows, or fp32 [capacity] of int8 rows, or None); ``position`` int32
    [R, S, k]: the place of each (slot, j) pair, or -1; ``offsets`` int32
    [E + 1]: expert e's rows are offsets[e]..offsets[e + 1] - 1; ``counts``
    int32 [E]: pairs of each expert, those beyond the capacity among them."""
    rows: torch.Tensor
    scales: Optional[torch.Tensor]
    position: torch.Tensor
    offsets: torch.Tensor
    counts: torch.Tensor


class QuantizedRows(NamedTuple):
    """int8 codes [M, N] and one fp32 scale a row [M]."""
    rows: torch.Tensor
    scales: torch.Tensor


class NormedRows(NamedTuple):
    """8-bit rows, their scales, and the new residual."""
    rows: torch.Tensor
    scales: torch.Tensor
    residual: torch.Tensor


def _refuse(msg: str):
    raise MoeEpArgError(ERR_INVALID_ARG, msg)


def _device(t, name):
    """The device of the call, from its first tensor."""
    if not t.is_cuda:
        _refuse(f"{name} must be a GPU tensor")
    return t.device


def _flat(t, name, dev, dtype, shape):
    """A contiguous tensor of this device, type and shape."""
    if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
        return
    if t.device != dev:
        _refuse(f"{name} must be on {dev}, got {t.device}")
    if t.dtype != dtype or t.shape != shape:
        _refuse(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    _refuse(f"{name} must be contiguous")


def _plane(t, name, dev):
    """Rank stride in bytes of a tensor [R, S, X] whose ranks may lie apart
    (a plane of the dispatch's workspace) but whose slots are contiguous."""
    if t.device != dev:
        _refuse(f"{name} must be on {dev}, got {t.device}")
    if t.dim() != 3:
        _refuse(f"{name} must be [ranks, slots, row], got {list(t.shape)}")
    R, S, X = t.shape
    if t.is_contiguous():
        return S * X * t.element_size()
    s0, s1, s2 = t.stride()
    if (X > 1 and s2 != 1) or (S > 1 and s1 != X) or (R > 1 and s0 < S * X):
        _refuse(f"{name}: the slots of a rank must be contiguous, got strides {t.stride()}")
    return s0 * t.element_size() if R > 1 else S * X * t.element_size()


def _row_type(t, name):
    rt = _ROW_TYPES.get(t.dtype)
    if rt is None:
        _refuse(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return rt


_written = torch.autograd.graph.increment_version  # of a given output: autograd then knows what it saved is gone


def _no_grad(*tensors):
    """Without a gradient of its own, an operator refuses to drop one."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                break
        else:
            return
        _refuse("this call has no gradient: detach its tensors or call it under torch.no_grad()")


def _whole(grad):
    """A gradient as autograd hands it over (expanded, a part of a larger buffer) as the kernels read it:
    contiguous, from a 16-byte boundary on."""
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 16 == 0 else grad.clone()


def _empty(shape, strides, dtype, dev):
    """A contiguous tensor; 0.4 us less of a call than ``torch.empty``."""
    return torch.empty_strided(shape, strides, dtype=dtype, device=dev)


_device_now = torch._C._cuda_getDevice
_stream_now = torch._C._cuda_getCurrentRawStream


class _On:
    """The device and stream of a call as the current ones: outputs allocated
    inside belong to that stream, launches go to it."""

    def __init__(self, dev, stream):
        self.contexts = []
        if _device_now() != dev.index:
            self.contexts.append(torch.cuda.device(dev))
        if stream is not None:
            if isinstance(stream, int):
                # torch takes 0 for "some stream of the pool", not for the default stream's handle
                stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
            if stream.device != dev:
                _refuse(f"the stream is on {stream.device}, the tensors on {dev}")
            self.contexts.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)


# ----------------------------------------------------------------------------
# expert sort
# ----------------------------------------------------------------------------

@functools.lru_cache(maxsize=4096)
def expert_sort_workspace_bytes(ranks: int, slots: int, top_k: int, experts_per_rank: int) -> int:
    if (not 1 <= experts_per_rank <= MAX_SORT_EXPERTS or min(ranks, slots, top_k) < 0
            or max(ranks, slots, top_k) > _INT_MAX):
        _refuse(f"bad sort shape: {ranks} ranks, {slots} slots, top_k {top_k}, {experts_per_rank} experts a rank")
    n = lib.moe_ep_expert_sort_workspace_bytes(ranks, slots, top_k, experts_per_rank)
    if n < 0:
        _refuse(lib.moe_ep_last_error().decode())
    return n


def expert_sort(ids, rows, experts_per_rank: int, *, scales=None, capacity: Optional[int] = None,
                quantize: bool = False, active_rank_mask: Optional[int] = None, out=None, out_scales=None,
                stream=None) -> SortedRows:
    """Rows to expert order.  ``ids`` int32 [R, S, k], ``rows`` [R, S, row]
    of any dtype and ``scales`` [R, S, scale row] or None, as a dispatch
    leaves them (R = 1: a batch of tokens); ranks may lie apart.  A pair (slot, j) counts when its
    id is one of its rank's ``experts_per_rank`` experts; counted pairs are
    placed by ascending (id, slot, j), those from place ``capacity`` on (by
    default R*S*k) are dropped; ranks outside ``active_rank_mask`` (the
    dispatch's) hold no pair.  Rows behind the last pair are left as they
    were, in ``out`` or uninitialised.  ``quantize``: bf16 or fp32 rows become
    int8 codes with scales = amax / 127.

    Differentiable in ``rows`` (bf16 or fp32; not with ``quantize``, ``out``
    or ``stream``: autograd orders its work by the current stream); the rows
    behind the last pair are then zeros.  ``scales`` have no gradient."""
    _no_grad(scales, out, out_scales)
    if rows.requires_grad and torch.is_grad_enabled():
        _need(not quantize and out is None and stream is None and rows.dtype in _ROW_TYPES,
              "only a sort of bf16 or fp32 rows into a new tensor, on the current stream, has a gradient")
        r, sc, p, o, c = _SortFunction.apply(rows, ids, experts_per_rank, scales, capacity, out_scales, active_rank_mask)
        return SortedRows(r, sc, p, o, c)
    return _sort(ids, rows, experts_per_rank, scales, capacity, quantize, out, out_scales, stream, active_rank_mask)


def _sort(ids, rows, epr, scales, capacity, quantize, out, out_scales, stream, active_rank_mask, zeros=False):
    dev = _device(rows, "rows")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return _sort(ids, rows, epr, scales, capacity, quantize, out, out_scales, None, active_rank_mask, zeros)
    if ids.dtype != torch.int32:
        _refuse(f"ids must be int32, got {ids.dtype}")
    ids_stride, rows_stride = _plane(ids, "ids", dev), _plane(rows, "rows", dev)
    R, S, k = ids.shape
    if rows.shape[0] != R or rows.shape[1] != S:
        _refuse(f"ids are [{R}, {S}, k], rows {list(rows.shape)}")
    X = rows.shape[2]
    row_type = _row_type(rows, "rows") if quantize else 0
    masked = 0
    if active_rank_mask is not None:
        active_rank_mask = int(active_rank_mask)
        if not 0 <= active_rank_mask < 1 << R:
            _refuse(f"active_rank_mask must be a mask of {R} ranks, got {active_rank_mask:#x}")
        masked = active_rank_mask ^ (1 << R) - 1
    if capacity is None:
        capacity = R * S * k
    elif capacity < 0:
        _refuse("capacity may not be negative")
    scales_stride = scale_bytes = 0
    if scales is not None:
        if quantize:
            _refuse("quantised rows take no scale rows")
        scales_stride = _plane(scales, "scales", dev)
        if scales.shape[:2] != ids.shape[:2]:
            _refuse(f"ids are [{R}, {S}, k], scales {list(scales.shape)}")
        scale_bytes = scales.shape[2] * scales.element_size()
    work = expert_sort_workspace_bytes(R, S, k, epr)
    dtype = torch.int8 if quantize else rows.dtype
    if out is None:
        out = torch.zeros((capacity, X), dtype=dtype, device=dev) if zeros else _empty((capacity, X), (X, 1), dtype, dev)
    else:
        _flat(out, "out", dev, dtype, (capacity, X))
        _written(out)
    if quantize or scales is not None:
        shape, dtype = ((capacity,), torch.float32) if quantize else ((capacity, scales.shape[2]), scales.dtype)
        if out_scales is None:
            out_scales = torch.empty(shape, dtype=dtype, device=dev)
        else:
            _flat(out_scales, "out_scales", dev, dtype, shape)
            _written(out_scales)
    else:
        out_scales = None
    E = R * epr
    position = _empty((R, S, k), (S * k, k, 1), torch.int32, dev)
    offsets = _empty((E + 1,), (1,), torch.int32, dev)
    counts = _empty((E,), (1,), torch.int32, dev)
    # held until the launches are on the stream: no other thread's call may take its memory between them
    space = torch.empty(work, dtype=torch.uint8, device=dev) if work else None
    _call(lib.moe_ep_expert_sort, _SORT, dev,
          ids.data_ptr(), ids_stride, rows.data_ptr(), rows_stride, X * rows.element_size(),
          scales.data_ptr() if scales is not None else 0, scales_stride, scale_bytes,
          out.data_ptr(), out_scales.data_ptr() if out_scales is not None else 0,
          position.data_ptr(), offsets.data_ptr(), counts.data_ptr(), space.data_ptr() if work else 0, work,
          capacity, R, S, k, epr, 1 if quantize else 0, row_type, masked)
    return SortedRows(out, out_scales, position, offsets, counts)


def expert_sort_backward(position, grad_rows, *, out=None, stream=None):
    """Gradient of the sort's rows: [R, S, H], each slot the sum of its
    pairs' rows of ``grad_rows`` [capacity, H] (zeros without a pair)."""
    _no_grad(grad_rows, out)
    return _unsort(position, grad_rows, None, out, False, stream)


class _SortFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, ids, epr, scales, capacity, out_scales, active_rank_mask):
        s = _sort(ids, rows, epr, scales, capacity, False, None, out_scales, None, active_rank_mask, zeros=True)
        ctx.save_for_backward(s.position)
        ctx.mark_non_differentiable(*(t for t in s[1:] if t is not None))
        ctx.set_materialize_grads(False)
        return tuple(s)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, *_):
        if grad is None:
            return (None,) * 7
        return (expert_sort_backward(ctx.saved_tensors[0], _whole(grad)),) + (None,) * 6


# ----------------------------------------------------------------------------
# expert unsort
# ----------------------------------------------------------------------------

def expert_unsort(position, rows, weights=None, *, out=None, keep_empty: bool = False, stream=None):
    """Expert rows back to their slots: out[r, q] = sum over j of
    weights[r, q, j] * rows[position[r, q, j]] in fp32, rounded once.
    ``position`` int32 [R, S, k] of the sort, ``rows`` [M, H] bf16 or fp32,
    ``weights`` fp32 [R, S, k] (ranks may lie apart) or None for 1.  Slots
    without a row become zeros, or with ``keep_empty`` (a given ``out``) are
    left alone: a combine never reads a slot without a token.  It does read
    one whose pairs a capacity dropped, so leave ``keep_empty`` off where the
    sort may drop pairs.

    Differentiable in ``rows`` and ``weights`` (without ``out`` or
    ``stream``)."""
    _no_grad(out)
    if (rows.requires_grad or (weights is not None and weights.requires_grad)) and torch.is_grad_enabled():
        _need(out is None and not keep_empty and stream is None,
              "only an unsort into a new tensor, on the current stream, has a gradient")
        return _UnsortFunction.apply(rows, weights, position)
    return _unsort(position, rows, weights, out, keep_empty, stream)


def _position(position, dev):
    if position.dim() != 3:
        _refuse(f"position must be [ranks, slots, top_k], got {list(position.shape)}")
    _flat(position, "position", dev, torch.int32, position.shape)


def _weights(weights, position, dev):
    if weights is None:
        return 0, 0
    if weights.dtype != torch.float32 or weights.shape != position.shape:
        _refuse(f"weights must be float32 {list(position.shape)}, got {weights.dtype} {list(weights.shape)}")
    return weights.data_ptr(), _plane(weights, "weights", dev)


def _unsort(position, rows, weights, out, keep_empty, stream):
    dev = _device(rows, "rows")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return _unsort(position, rows, weights, out, keep_empty, None)
    rt = _row_type(rows, "rows")
    if rows.dim() != 2:
        _refuse(f"rows must be [num_rows, hidden], got {list(rows.shape)}")
    M, H = rows.shape
    _flat(rows, "rows", dev, rows.dtype, rows.shape)
    _position(position, dev)
    R, S, k = position.shape
    wp, ws = _weights(weights, position, dev)
    if out is None:
        if keep_empty:
            _refuse("keep_empty needs a given out")
        out = _empty((R, S, H), (S * H, H, 1), rows.dtype, dev)
        stride = S * H * rows.element_size()
    else:
        if out.dtype != rows.dtype or out.shape != (R, S, H):
            _refuse(f"out must be {rows.dtype} [{R}, {S}, {H}], got {out.dtype} {list(out.shape)}")
        stride = _plane(out, "out", dev)
        _written(out)
    _call(lib.moe_ep_expert_unsort, _UNSORT, dev,
          position.data_ptr(), rows.data_ptr(), wp, ws, out.data_ptr(), stride, M, R, S, k, H, rt,
          1 if keep_empty else 0)
    return out


def expert_unsort_backward(position, grad_out, rows=None, weights=None, *, grad_rows=None, need_rows: bool = True,
                           need_weights: bool = True, stream=None):
    """Gradients of ``expert_unsort`` for ``grad_out`` [R, S, H]:
    (grad_rows [M, H], grad_weights fp32 [R, S, k]), None for one not needed.
    grad_rows' rows that no pair names are left as they were, in a given
    ``grad_rows``, or zeros.  ``rows``, the unsort's input, is needed for
    grad_weights; without it give ``grad_rows``."""
    _no_grad(grad_out, rows, weights, grad_rows)
    dev = _device(grad_out, "grad_out")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return expert_unsort_backward(position, grad_out, rows, weights, grad_rows=grad_rows, need_rows=need_rows,
                                          need_weights=need_weights)
    rt = _row_type(grad_out, "grad_out")
    stride = _plane(grad_out, "grad_out", dev)
    _position(position, dev)
    R, S, k = position.shape
    if grad_out.shape[:2] != position.shape[:2]:
        _refuse(f"position is [{R}, {S}, k], grad_out {list(grad_out.shape)}")
    H = grad_out.shape[2]
    like = rows if rows is not None else grad_rows
    if like is None or (need_weights and rows is None):
        _refuse("rows are needed for grad_weights; without it give grad_rows")
    if like.dim() != 2:
        _refuse(f"rows and grad_rows must be [num_rows, hidden], got {list(like.shape)}")
    M = like.shape[0]
    if rows is not None:
        _flat(rows, "rows", dev, grad_out.dtype, (M, H))
    if grad_rows is not None:
        _flat(grad_rows, "grad_rows", dev, grad_out.dtype, (M, H))
        _written(grad_rows)
    wp, ws = _weights(weights, position, dev)
    if not need_rows:
        grad_rows = None
    elif grad_rows is None:
        grad_rows = torch.zeros((M, H), dtype=grad_out.dtype, device=dev)
    gw = torch.empty((R, S, k), dtype=torch.float32, device=dev) if need_weights else None
    _call(lib.moe_ep_expert_unsort_backward, _UNSORT_GRAD, dev,
          position.data_ptr(), grad_out.data_ptr(), stride, rows.data_ptr() if rows is not None else 0, wp, ws,
          grad_rows.data_ptr() if grad_rows is not None else 0, gw.data_ptr() if gw is not None else 0,
          M, R, S, k, H, rt, 0)
    return grad_rows, gw


class _UnsortFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, position):
        need_weights = weights is not None and weights.requires_grad
        kept = weights
        if weights is not None and weights.untyped_storage().nbytes() != 4 * weights.numel():
            # a plane of a workspace, which the next dispatch overwrites unseen by autograd
            kept = weights.clone()
        # the rows matter to the weights' gradient only
        ctx.save_for_backward(position, kept, rows if need_weights else None)
        ctx.rows_shape = rows.shape
        return _unsort(position, rows, weights, None, False, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        position, weights, rows = ctx.saved_tensors
        need_rows = ctx.needs_input_grad[0]
        g = None
        if rows is None:
            g = torch.zeros(ctx.rows_shape, dtype=grad.dtype, device=grad.device)
        gr, gw = expert_unsort_backward(position, _whole(grad), rows, weights, grad_rows=g, need_rows=need_rows,
                                        need_weights=ctx.needs_input_grad[1])
        return gr, gw, None


# ----------------------------------------------------------------------------
# products and row-wise operators
# ----------------------------------------------------------------------------

def expert_matmul(x, x_scales, weight, weight_scales, *, offsets=None, out=None, dtype=None, stream=None):
    """Product of int8 rows [M, K] (fp32 scales [M]) with each expert's int8
    weights [E, N, K] (fp32 channel scales [E, N]): rows
    offsets[e]..offsets[e + 1] - 1 meet expert e's, other rows of the result
    [M, N] are left as they were, in ``out`` or uninitialised.  Dense: weight
    [N, K], scales [N], no offsets.  The sum is exact; the result is of
    ``dtype`` (bf16 or fp32), by default ``out``'s, bf16 without ``out``."""
    if out is not None and dtype not in (None, out.dtype):
        _refuse(f"out is {out.dtype}, the result's dtype {dtype}")
    _no_grad(x_scales, weight_scales, out)
    dev = _device(x, "x")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return expert_matmul(x, x_scales, weight, weight_scales, offsets=offsets, out=out, dtype=dtype)
    if x.dim() != 2 or weight.dim() not in (2, 3):
        _refuse(f"x must be [M, K] and weight [E, N, K] or [N, K], got {list(x.shape)} and {list(weight.shape)}")
    M, K = x.shape
    _flat(x, "x", dev, torch.int8, (M, K))
    _flat(x_scales, "x_scales", dev, torch.float32, (M,))
    if weight.dim() == 3:
        E, N = weight.shape[:2]
        if offsets is None:
            _refuse("expert weights [E, N, K] need offsets")
        _flat(weight, "weight", dev, torch.int8, (E, N, K))
        _flat(weight_scales, "weight_scales", dev, torch.float32, (E, N))
        _flat(offsets, "offsets", dev, torch.int32, (E + 1,))
    else:
        E, N = 1, weight.shape[0]
        if offsets is not None:
            _refuse("a dense weight [N, K] takes no offsets")
        _flat(weight, "weight", dev, torch.int8, (N, K))
        _flat(weight_scales, "weight_scales", dev, torch.float32, (N,))
    if out is None:
        out = _empty((M, N), (N, 1), dtype or torch.bfloat16, dev)
    else:
        _flat(out, "out", dev, out.dtype, (M, N))
        _written(out)
    _call(lib.moe_ep_expert_matmul, _MATMUL, dev,
          x.data_ptr(), x_scales.data_ptr(), weight.data_ptr(), weight_scales.data_ptr(),
          offsets.data_ptr() if offsets is not None else 0, out.data_ptr(), M, E, N, K,
          _row_type(out, "out"))
    return out


def silu_mul_quantize(x, *, offsets=None, out=None, out_scales=None, stream=None) -> QuantizedRows:
    """silu(x[:, :I]) * x[:, I:] of bf16 or fp32 rows [M, 2 I] as int8 codes
    [M, I] with scales = amax / 127.  With the sort's ``offsets`` only its
    offsets[-1] rows are computed, the others left as they were."""
    _no_grad(x, out_scales)
    dev = _device(x, "x")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return silu_mul_quantize(x, offsets=offsets, out=out, out_scales=out_scales)
    rt = _row_type(x, "x")
    if x.dim() != 2 or x.shape[1] % 2:
        _refuse(f"x must be [M, 2 I], got {list(x.shape)}")
    M, I = x.shape[0], x.shape[1] // 2
    _flat(x, "x", dev, x.dtype, x.shape)
    last = 0
    if offsets is not None:
        if offsets.dim() != 1 or offsets.numel() < 1:
            _refuse(f"offsets must be [E + 1], got {list(offsets.shape)}")
        _flat(offsets, "offsets", dev, torch.int32, offsets.shape)
        last = offsets.data_ptr() + 4 * (offsets.numel() - 1)
    if out is None:
        out = _empty((M, I), (I, 1), torch.int8, dev)
    else:
        _flat(out, "out", dev, torch.int8, (M, I))
        _written(out)
    if out_scales is None:
        out_scales = _empty((M,), (1,), torch.float32, dev)
    else:
        _flat(out_scales, "out_scales", dev, torch.float32, (M,))
        _written(out_scales)
    _call(lib.moe_ep_silu_mul_quantize, _SILU, dev,
          x.data_ptr(), last, out.data_ptr(), out_scales.data_ptr(), M, I, rt)
    return QuantizedRows(out, out_scales)


def add_rms_norm(x, residual, weight, eps: float = 1e-6, *, format: str = "mxfp8", out=None, out_scales=None,
                 residual_out=None, stream=None) -> NormedRows:
    """s = x + residual (``residual`` None: x), y = s / sqrt(mean(s^2) + eps)
    * weight in fp32, as 8-bit rows: ``format`` "mxfp8" (e4m3 codes, an e8m0
    scale for 32) and "deepseek_fp8" (e4m3, an fp32 scale for 128) are
    dispatch payloads, "int8" (one fp32 scale a row) feeds ``expert_matmul``.
    x, residual [M, H] and weight [H], all bf16 or all fp32.  The returned
    residual is s rounded to x's type, written to ``residual_out`` (which may
    be ``residual`` or ``x``) or a new tensor; without a residual it is x."""
    _no_grad(x, residual, weight, out, out_scales, residual_out)
    if format not in _NORMS:
        _refuse(f"format must be one of {sorted(_NORMS)}, got {format!r}")
    code, block, row_dtype, scale_dtype = _NORMS[format]
    dev = _device(x, "x")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return add_rms_norm(x, residual, weight, eps, format=format, out=out, out_scales=out_scales,
                                residual_out=residual_out)
    rt = _row_type(x, "x")
    if x.dim() != 2:
        _refuse(f"x must be [M, H], got {list(x.shape)}")
    M, H = x.shape
    _flat(x, "x", dev, x.dtype, (M, H))
    _flat(weight, "weight", dev, x.dtype, (H,))
    if residual is not None:
        _flat(residual, "residual", dev, x.dtype, (M, H))
    if not 0 <= eps <= 1e30:
        _refuse(f"eps must be finite and >= 0, got {eps}")
    if block and H % block:
        _refuse(f"{format} needs a hidden size that is a multiple of {block}, got {H}")
    scale_shape = (M, H // block) if block else (M,)
    if out is None:
        out = torch.empty_like(x, dtype=row_dtype)
    else:
        _flat(out, "out", dev, row_dtype, (M, H))
        _written(out)
    if out_scales is None:
        out_scales = _empty(scale_shape, (H // block, 1) if block else (1,), scale_dtype, dev)
    else:
        _flat(out_scales, "out_scales", dev, scale_dtype, scale_shape)
        _written(out_scales)
    if residual_out is not None:
        _flat(residual_out, "residual_out", dev, x.dtype, (M, H))
        _written(residual_out)
    elif residual is not None:
        residual_out = torch.empty_like(x)
    _call(lib.moe_ep_add_rms_norm, _NORM, dev,
          x.data_ptr(), residual.data_ptr() if residual is not None else 0, weight.data_ptr(),
          residual_out.data_ptr() if residual_out is not None else 0, out.data_ptr(), out_scales.data_ptr(),
          M, H, rt, code, eps)
    return NormedRows(out, out_scales, x if residual_out is None else residual_out)
