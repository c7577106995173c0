"""The trainable expert layer (ctypes over ``include/moe_ep.h``): the gated
feed-forward block of experts in bf16 with its gradients, 8-bit checkpoints of
what its backward pass reads, and products with 4-bit weights for serving.

``expert_ffn`` takes the rows of ``experts.expert_sort`` (bf16) and its
``offsets`` and gives the rows that ``experts.expert_unsort`` takes back; with
dense weights and no offsets it is a shared expert.  Streams, allocations,
errors and gradients follow the rules of ``experts``.  In a HIP graph capture
the explicit calls (``expert_ffn_forward``, ``expert_ffn_backward``): torch
ends the process when autograd's backward pass is captured while an eager
graph of the same leaves lives.
"""
from __future__ import annotations

import struct
from typing import NamedTuple, Optional

import torch

from .experts import (_call, _device, _device_now, _empty, _flat, _new, _no_grad, _no_tangent, _On, _refuse, _row_type,
                      _whole, _written)
from .moe_ep import _need, lib

SAVE_NONE, SAVE_HALF, SAVE_MXFP8 = 0, 1, 2
_SAVES = {"bf16": SAVE_HALF, "mxfp8": SAVE_MXFP8}
_BF16, _CODES, _SCALES = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e8m0fnu
_PRE = {SAVE_HALF: (torch.float16, 8), SAVE_MXFP8: (_CODES, 32)}  # the saved product's type, elements of a scale

# The argument blocks of include/moe_ep.h in native layout.
_CHECKPOINT = struct.Struct("@PPPqii")
_PRODUCT = struct.Struct("@PPPPqiiiiii")
_GATED = struct.Struct("@PPPPPPqiiii")
_GATED_GRAD = struct.Struct("@PPPPPPPqiiii")
_WEIGHT_GRAD = struct.Struct("@PPPPqiiii")
_FOUR_BIT = struct.Struct("@PPPPPqiiiiii")


class MxRows(NamedTuple):
    """MXFP8 rows: e4m3 codes [M, H] and e8m0 scales [M, H / 32]."""
    rows: torch.Tensor
    scales: torch.Tensor


class FfnCheckpoint(NamedTuple):
    """What the backward pass of ``expert_ffn`` reads: its input, as it is or
    as MXFP8 codes with scales, and the first product (gate, then up) in fp16
    with an e8m0 scale for eight (17 bits an element), or as MXFP8."""
    x: torch.Tensor
    x_scales: Optional[torch.Tensor]
    pre: torch.Tensor
    pre_scales: torch.Tensor


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _rows2(t, name, dev, dtype):
    """A contiguous tensor [rows, width]."""
    if t.dim() != 2:
        _refuse(f"{name} must be [rows, width], got {list(t.shape)}")
    _flat(t, name, dev, dtype, t.shape)
    return t.shape


def _experts(weight, name, dev, dtype, offsets):
    """(E, first, second axis) of a weight [E, a, b] with offsets or [a, b] without."""
    if weight.dim() == 3:
        if offsets is None:
            _refuse(f"expert weights {name} [E, n, k] need offsets")
        E, a, b = weight.shape
        _flat(offsets, "offsets", dev, torch.int32, (E + 1,))
    elif weight.dim() == 2:
        if offsets is not None:
            _refuse(f"a dense weight {name} [n, k] takes no offsets")
        E, (a, b) = 1, weight.shape
    else:
        _refuse(f"{name} must be [E, n, k] or [n, k], got {list(weight.shape)}")
    _flat(weight, name, dev, dtype, weight.shape)
    return E, a, b


def _out(out, name, dev, dtype, shape):
    """A given output, checked, or a new one."""
    if out is None:
        return _new(shape, dtype, dev)
    _flat(out, name, dev, dtype, shape)
    _written(out)
    return out


def _as(t, dtype):
    """Bytes as what they hold."""
    return t.view(dtype) if t.dtype == torch.uint8 else t


def _save_code(checkpoint, *widths):
    code = _SAVES.get(checkpoint)
    if code is None:
        _refuse(f"checkpoint must be one of {sorted(_SAVES)}, got {checkpoint!r}")
    if code == SAVE_MXFP8 and any(w % 32 for w in widths):
        _refuse(f"an MXFP8 checkpoint needs widths that are multiples of 32, got {list(widths)}")
    return code


# ----------------------------------------------------------------------------
# 8-bit checkpoints
# ----------------------------------------------------------------------------

def checkpoint_rows(x, *, out=None, out_scales=None, stream=None) -> MxRows:
    """Rows [M, H] (bf16 or fp32, H a multiple of 32) as MXFP8: e4m3 codes
    and the smallest power of two a block of 32 that keeps it within 448, as
    in an MXFP8 dispatch.  A block with a NaN or an infinity is NaN."""
    _no_grad(x, out, out_scales)
    dev = _device(x, "x")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return checkpoint_rows(x, out=out, out_scales=out_scales)
    rt = _row_type(x, "x")
    M, H = _rows2(x, "x", dev, x.dtype)
    if H < 32 or H % 32:
        _refuse(f"MXFP8 rows need a width that is a multiple of 32, got {H}")
    out, out_scales = _out(out, "out", dev, _CODES, (M, H)), _out(out_scales, "out_scales", dev, _SCALES, (M, H // 32))
    _call(lib.moe_ep_checkpoint_rows, _CHECKPOINT, dev, x.data_ptr(), out.data_ptr(), out_scales.data_ptr(), M, H, rt)
    return MxRows(out, out_scales)


def restore_rows(rows, scales, *, dtype=None, out=None, stream=None):
    """MXFP8 rows as bf16 or fp32 rows, ``out``'s type or bf16.  fp32 holds
    code * scale exactly, and so does bf16 for scale bytes 3 to 246; for
    smaller ones it rounds to its least step, 2^-133.  ``rows`` and
    ``scales`` are a checkpoint's, or the bytes (uint8) of an MXFP8
    dispatch's payload as the sort leaves them."""
    _no_grad(rows, out)
    if out is not None and dtype not in (None, out.dtype):
        _refuse(f"out is {out.dtype}, the result's dtype {dtype}")
    dev = _device(rows, "rows")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return restore_rows(rows, scales, dtype=dtype, out=out)
    rows, scales = _as(rows, _CODES), _as(scales, _SCALES)
    M, H = _rows2(rows, "rows", dev, _CODES)
    if H < 32 or H % 32:
        _refuse(f"MXFP8 rows need a width that is a multiple of 32, got {H}")
    _flat(scales, "scales", dev, _SCALES, (M, H // 32))
    out = _out(out, "out", dev, out.dtype if out is not None else dtype or _BF16, (M, H))
    _call(lib.moe_ep_restore_rows, _CHECKPOINT, dev, out.data_ptr(), rows.data_ptr(), scales.data_ptr(), M, H,
          _row_type(out, "out"))
    return out


# ----------------------------------------------------------------------------
# products
# ----------------------------------------------------------------------------

def expert_product(x, weight, *, offsets=None, transposed: bool = False, out=None, stream=None):
    """Product of bf16 rows [M, K] with each expert's bf16 weights: [E, N, K]
    (rows times its transpose), or with ``transposed`` [E, K, N].  Rows
    offsets[e]..offsets[e + 1] - 1 meet expert e's, other rows of the result
    are left as they were, in ``out`` or uninitialised.  Dense: a weight of
    two axes, no offsets.  fp32 sums, rounded once."""
    _no_grad(x, weight, out)
    return _product(x, weight, offsets, transposed, out, stream, False)


def _product(x, weight, offsets, transposed, out, stream, zero_rest):
    dev = _device(x, "x")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return _product(x, weight, offsets, transposed, out, None, zero_rest)
    M, K = _rows2(x, "x", dev, _BF16)
    E, N, k = _experts(weight, "weight", dev, _BF16, offsets)
    if transposed:
        N, k = k, N
    if k != K:
        _refuse(f"x is [M, {K}], the weight {list(weight.shape)}")
    out = _out(out, "out", dev, _BF16, (M, N))
    _call(lib.moe_ep_expert_product, _PRODUCT, dev, x.data_ptr(), weight.data_ptr(), _ptr(offsets), out.data_ptr(), M, E,
          N, K, 1 if transposed else 0, 1 if zero_rest else 0, 0)
    return out


def gated_product(x, weight, *, offsets=None, checkpoint: Optional[str] = None, out=None, stream=None):
    """silu(gate) * up of bf16 rows [M, K] with each expert's weights
    [E, 2 I, K], gate channels first, in one kernel: (rows [M, I], pre,
    pre_scales).  ``checkpoint`` also gives the products themselves [M, 2 I]
    for ``gated_product_backward``: "bf16" in fp16 with an e8m0 scale for
    eight (11 significant bits; bf16's eight would cost the gradients half
    their accuracy again), "mxfp8" as e4m3 codes with a scale for 32; else
    pre is None.  Rows as in ``expert_product``."""
    _no_grad(x, weight, out)
    dev = _device(x, "x")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return gated_product(x, weight, offsets=offsets, checkpoint=checkpoint, out=out)
    M, K = _rows2(x, "x", dev, _BF16)
    E, N, k = _experts(weight, "weight", dev, _BF16, offsets)
    if k != K or N % 2:
        _refuse(f"x is [M, {K}], the weight must be [E, 2 I, {K}], got {list(weight.shape)}")
    I = N // 2
    save = SAVE_NONE if checkpoint is None else _save_code(checkpoint, I)
    out = _out(out, "out", dev, _BF16, (M, I))
    pre = scales = None
    if save:
        dtype, block = _PRE[save]
        pre, scales = _empty((M, N), (N, 1), dtype, dev), _empty((M, N // block), (N // block, 1), _SCALES, dev)
    _call(lib.moe_ep_gated_product, _GATED, dev, x.data_ptr(), weight.data_ptr(), _ptr(offsets), out.data_ptr(), _ptr(pre),
          _ptr(scales), M, E, I, K, save)
    return out, pre, scales


def gated_product_backward(grad_out, weight, pre, pre_scales, *, offsets=None, need_rows: bool = True, stream=None):
    """The gradient grad_out [M, N] of the block's second product, weights
    [E, N, I], taken through it and the activation at ``gated_product``'s
    pre: (grad_pre [M, 2 I], the activation rows [M, I] again or None)."""
    if pre is None or pre_scales is None:
        _refuse("pre and pre_scales are what gated_product gives with a checkpoint, and without one it keeps none")
    _no_grad(grad_out, weight, pre)
    dev = _device(grad_out, "grad_out")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return gated_product_backward(grad_out, weight, pre, pre_scales, offsets=offsets, need_rows=need_rows)
    M, N = _rows2(grad_out, "grad_out", dev, _BF16)
    E, n, I = _experts(weight, "weight", dev, _BF16, offsets)
    if n != N:
        _refuse(f"grad_out is [M, {N}], the weight {list(weight.shape)}")
    save = SAVE_HALF if pre.dtype == torch.float16 else SAVE_MXFP8
    dtype, block = _PRE[save]
    if I % block:
        _refuse(f"this checkpoint needs a width that is a multiple of {block}, got {I}")
    _flat(pre, "pre", dev, dtype, (M, 2 * I))
    _flat(pre_scales, "pre_scales", dev, _SCALES, (M, 2 * I // block))
    grad_pre = _empty((M, 2 * I), (2 * I, 1), _BF16, dev)
    rows = _empty((M, I), (I, 1), _BF16, dev) if need_rows else None
    _call(lib.moe_ep_gated_product_backward, _GATED_GRAD, dev, grad_out.data_ptr(), weight.data_ptr(), _ptr(offsets),
          pre.data_ptr(), _ptr(pre_scales), grad_pre.data_ptr(), _ptr(rows), M, E, I, N, save)
    return grad_pre, rows


def product_weight_grad(grad_out, x, *, offsets=None, out=None, stream=None):
    """Gradient of an expert product's weights: [E, N, K], for each expert
    the sum over its rows of grad_out [M, N] times x [M, K], zeros without
    rows; dense [N, K] without offsets."""
    _no_grad(grad_out, x, out)
    dev = _device(grad_out, "grad_out")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return product_weight_grad(grad_out, x, offsets=offsets, out=out)
    M, N = _rows2(grad_out, "grad_out", dev, _BF16)
    m, K = _rows2(x, "x", dev, _BF16)
    if m != M:
        _refuse(f"grad_out has {M} rows, x {m}")
    if offsets is None:
        E, shape = 1, (N, K)
    else:
        if offsets.dim() != 1 or offsets.numel() < 2:
            _refuse(f"offsets must be [E + 1], got {list(offsets.shape)}")
        _flat(offsets, "offsets", dev, torch.int32, offsets.shape)
        E = offsets.numel() - 1
        shape = (E, N, K)
    out = _out(out, "out", dev, _BF16, shape)
    _call(lib.moe_ep_product_weight_grad, _WEIGHT_GRAD, dev, grad_out.data_ptr(), x.data_ptr(), _ptr(offsets),
          out.data_ptr(), M, E, N, K, 0)
    return out


def expert_matmul_mxfp4(x, weight, weight_scales, *, offsets=None, gated: bool = False, out=None, dtype=None, stream=None):
    """Product of bf16 rows [M, K] with each expert's 4-bit weights, made for
    a few rows an expert (serving): ``weight`` uint8 [E, N, K / 2], two e2m1
    codes a byte, the even element in the low half, ``weight_scales`` e8m0
    [E, N, K / 32] (MXFP4).  ``gated``: N = 2 I channels, gate first, and the
    result is silu(gate) * up [M, I].  Rows, dense weights and ``dtype`` (bf16
    or fp32) as in ``experts.expert_matmul``.  Fastest for K a multiple of
    128 and scales that begin on 4 bytes (other calls take 1.4 times as
    long), and for up to 16 rows an expert."""
    if out is not None and dtype not in (None, out.dtype):
        _refuse(f"out is {out.dtype}, the result's dtype {dtype}")
    _no_grad(x, out)
    dev = _device(x, "x")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return expert_matmul_mxfp4(x, weight, weight_scales, offsets=offsets, gated=gated, out=out, dtype=dtype)
    M, K = _rows2(x, "x", dev, _BF16)
    E, N, half = _experts(weight, "weight", dev, torch.uint8, offsets)
    if K % 32 or half * 2 != K:
        _refuse(f"x is [M, {K}] (K a multiple of 32), the weight {list(weight.shape)}")
    if gated and N % 2:
        _refuse(f"a gated weight has 2 I channels, got {N}")
    _flat(weight_scales, "weight_scales", dev, _SCALES, (*weight.shape[:-1], K // 32))
    out = _out(out, "out", dev, out.dtype if out is not None else dtype or _BF16, (M, N // 2 if gated else N))
    _call(lib.moe_ep_four_bit_product, _FOUR_BIT, dev, x.data_ptr(), weight.data_ptr(), weight_scales.data_ptr(),
          _ptr(offsets), out.data_ptr(), M, E, N, K, 1 if gated else 0, _row_type(out, "out"), 0)
    return out


# ----------------------------------------------------------------------------
# the gated feed-forward block
# ----------------------------------------------------------------------------

def expert_ffn(x, w1, w2, *, offsets=None, checkpoint: str = "bf16", out=None, stream=None):
    """The gated feed-forward block of experts: bf16 rows [M, H] through
    ``w1`` [E, 2 I, H] (gate channels first), silu(gate) * up, and ``w2``
    [E, H, I].  Rows offsets[e]..offsets[e + 1] - 1 meet expert e's, other
    rows of the result are left as they were, in ``out`` or uninitialised.
    Dense: w1 [2 I, H], w2 [H, I], no offsets.

    Differentiable in ``x``, ``w1`` and ``w2`` (without ``out`` or
    ``stream``); the rows outside the experts' ranges are then zeros, and
    their gradients too.  ``checkpoint`` says what the backward pass keeps of
    x and of the first product: "bf16", x itself (a copy where x is a part of
    a larger buffer, such as a slice of a batch: the next dispatch would
    overwrite it unseen) and the product in 17 bits an element (fp16, a
    scale for eight), or "mxfp8", both in 8.25 (H and I multiples of 32; the
    gradients are then those at the rounded values).

    Sums are fp32, and what passes from one product to the next is bf16, the
    operand of the matrix cores: the activation and y in the forward pass,
    the gradient of the first product, the activation again and grad_x in
    the backward pass, each rounded once."""
    _no_tangent(x, w1, w2)
    _no_grad(out)
    if torch.is_grad_enabled() and (x.requires_grad or w1.requires_grad or w2.requires_grad):
        _need(out is None and stream is None, "only a block into a new tensor, on the current stream, has a gradient")
        return _FfnFunction.apply(x, w1, w2, offsets, checkpoint)
    dev = _device(x, "x")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return expert_ffn(x, w1, w2, offsets=offsets, checkpoint=checkpoint, out=out)
    _save_code(checkpoint, *_check_ffn(x, w1, w2, offsets))
    return _product(gated_product(x, w1, offsets=offsets)[0], w2, offsets, False, out, None, False)


def _check_ffn(x, w1, w2, offsets):
    """(H, I) of a block whose weights fit each other and the rows."""
    dev = x.device
    _, H = _rows2(x, "x", dev, _BF16)
    E, N, h = _experts(w1, "w1", dev, _BF16, offsets)
    if h != H or N % 2:
        _refuse(f"x is [M, {H}], w1 must be [E, 2 I, {H}], got {list(w1.shape)}")
    if w2.shape != (*w1.shape[:-2], H, N // 2):
        _refuse(f"w2 must be {list((*w1.shape[:-2], H, N // 2))}, got {list(w2.shape)}")
    _flat(w2, "w2", dev, _BF16, w2.shape)
    return H, N // 2


def expert_ffn_forward(x, w1, w2, *, offsets=None, checkpoint: str = "bf16", stream=None):
    """(y, FfnCheckpoint) of ``expert_ffn``, for ``expert_ffn_backward``.
    Rows outside the experts' ranges are zeros in y.  A "bf16" checkpoint
    holds x itself, no copy: leave it as it is until the backward pass."""
    _no_grad(x, w1, w2)
    dev = _device(x, "x")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return expert_ffn_forward(x, w1, w2, offsets=offsets, checkpoint=checkpoint)
    save = _save_code(checkpoint, *_check_ffn(x, w1, w2, offsets))
    rows, pre, pre_scales = gated_product(x, w1, offsets=offsets, checkpoint=checkpoint)
    kept = checkpoint_rows(x) if save == SAVE_MXFP8 else (x, None)
    return _product(rows, w2, offsets, False, None, None, True), FfnCheckpoint(*kept, pre, pre_scales)


def expert_ffn_backward(grad_y, saved: FfnCheckpoint, w1, w2, *, offsets=None, needs=(True, True, True), stream=None):
    """Gradients of ``expert_ffn`` for grad_y [M, H]: (grad_x, grad_w1,
    grad_w2) in bf16, None where ``needs`` says so.  grad_x is zeros outside
    the experts' ranges, a weight's gradient for an expert without rows."""
    _no_grad(grad_y, w1, w2, *saved)
    dev = _device(grad_y, "grad_y")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return expert_ffn_backward(grad_y, saved, w1, w2, offsets=offsets, needs=needs)
    H, _ = _check_ffn(grad_y, w1, w2, offsets)
    M = grad_y.shape[0]
    _flat(saved.x, "the checkpoint's x", dev, _BF16 if saved.x_scales is None else _CODES, (M, H))
    need_x, need_w1, need_w2 = needs
    grad_pre, rows = gated_product_backward(grad_y, w2, saved.pre, saved.pre_scales, offsets=offsets, need_rows=need_w2)
    grad_w2 = product_weight_grad(grad_y, rows, offsets=offsets) if need_w2 else None
    grad_w1 = None
    if need_w1:
        x = saved.x if saved.x_scales is None else restore_rows(saved.x, saved.x_scales)
        grad_w1 = product_weight_grad(grad_pre, x, offsets=offsets)
    grad_x = _product(grad_pre, w1, offsets, True, None, None, True) if need_x else None
    return grad_x, grad_w1, grad_w2


class _FfnFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w1, w2, offsets, checkpoint):
        y, saved = expert_ffn_forward(x, w1, w2, offsets=offsets, checkpoint=checkpoint)
        if saved.x_scales is None and x.untyped_storage().nbytes() != x.numel() * x.element_size():
            # a part of a workspace, which the next dispatch overwrites unseen by autograd
            saved = saved._replace(x=x.clone())
        ctx.save_for_backward(w1, w2, offsets, *saved)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        w1, w2, offsets, *saved = ctx.saved_tensors
        grads = expert_ffn_backward(_whole(grad), FfnCheckpoint(*saved), w1, w2, offsets=offsets,
                                    needs=ctx.needs_input_grad[:3])
        return (*grads, None, None)
