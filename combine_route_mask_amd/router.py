"""The router: the experts of each token and their weights from its logits,
with their gradient (ctypes over ``include/moe_ep.h``).

Its ids and weights are what a dispatch, ``experts.expert_sort`` and
``experts.expert_unsort`` take.  Streams, allocations, errors and gradients
follow the rules of ``experts``.
"""
from __future__ import annotations

import struct
from typing import NamedTuple

import torch

from .experts import (_call, _device, _device_now, _flat, _new, _no_grad, _no_tangent, _On, _refuse, _row_type, _whole,
                      _written)
from .moe_ep import _need, lib

MAX_ROUTED_EXPERTS = 4096  # MOE_EP_MAX_ROUTED_EXPERTS

# The argument blocks of include/moe_ep.h in native layout.
_ROUTE = struct.Struct("@PPPqiiiifi")
_ROUTE_GRAD = struct.Struct("@PPPPqiiiifi")


class Routes(NamedTuple):
    """``ids`` int32 [..., k] and ``weights`` fp32 [..., k] of each token."""
    ids: torch.Tensor
    weights: torch.Tensor


def route_top_k(logits, top_k: int, *, renormalize: bool = True, scale: float = 1.0, ids=None, weights=None,
                stream=None) -> Routes:
    """The ``top_k`` largest of each token's logits [..., E] (bf16 or fp32),
    largest first, equal ones by ascending expert, and scale * softmax over
    the chosen experts (``renormalize``) or over all.  An expert whose logit
    is -infinity or NaN is never chosen: a place without an expert holds the
    id E, which a dispatch routes nowhere and a sort passes over, and the
    weight 0.  A row with a NaN or +infinity has NaN weights.

    Differentiable in ``logits`` (without given outputs or ``stream``); the
    backward pass keeps them, a copy where they are a part of a larger
    buffer, such as a dispatch's workspace."""
    _no_tangent(logits)
    _no_grad(weights)
    if logits.requires_grad and torch.is_grad_enabled():
        _need(ids is None and weights is None and stream is None,
              "only a routing into new tensors, on the current stream, has a gradient")
        return Routes(*_RouteFunction.apply(logits, top_k, renormalize, scale))
    return _route(logits, top_k, renormalize, scale, ids, weights, stream)


def _shape(logits, top_k):
    if logits.dim() < 1:
        _refuse("logits must be [..., experts]")
    E = logits.shape[-1]
    if not 1 <= E <= MAX_ROUTED_EXPERTS:
        _refuse(f"experts must be in [1, {MAX_ROUTED_EXPERTS}], got {E}")
    if not 1 <= top_k <= min(64, E):
        _refuse(f"top_k must be in [1, 64] and at most the {E} experts, got {top_k}")
    return E, logits.numel() // E, (*logits.shape[:-1], top_k)


def _route(logits, top_k, renormalize, scale, ids, weights, stream):
    dev = _device(logits, "logits")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return _route(logits, top_k, renormalize, scale, ids, weights, None)
    rt = _row_type(logits, "logits")
    E, T, shape = _shape(logits, top_k)
    _flat(logits, "logits", dev, logits.dtype, logits.shape)
    if ids is None:
        ids = _new(shape, torch.int32, dev)
    else:
        _flat(ids, "ids", dev, torch.int32, shape)
        _written(ids)
    if weights is None:
        weights = _new(shape, torch.float32, dev)
    else:
        _flat(weights, "weights", dev, torch.float32, shape)
        _written(weights)
    _call(lib.moe_ep_route_top_k, _ROUTE, dev, logits.data_ptr(), ids.data_ptr(), weights.data_ptr(), T, E, top_k,
          1 if renormalize else 0, rt, scale, 0)
    return Routes(ids, weights)


def route_top_k_backward(logits, ids, grad_weights, *, renormalize: bool = True, scale: float = 1.0, out=None,
                         stream=None):
    """Gradient of ``route_top_k``'s weights for the logits [..., E], in
    their type; ``ids`` as the router chose them (an id once a token),
    ``grad_weights`` fp32 [..., k].  With ``renormalize`` only the chosen
    logits are read: a NaN among the others has no part in it.  Without, a
    NaN or +infinity makes its row's gradient NaN."""
    _no_grad(logits, grad_weights, out)
    dev = _device(logits, "logits")
    if stream is not None or dev.index != _device_now():
        with _On(dev, stream):
            return route_top_k_backward(logits, ids, grad_weights, renormalize=renormalize, scale=scale, out=out)
    rt = _row_type(logits, "logits")
    if ids.dim() != logits.dim():
        _refuse(f"ids must be [..., top_k] of logits {list(logits.shape)}, got {list(ids.shape)}")
    k = ids.shape[-1] if ids.dim() else 0
    E, T, shape = _shape(logits, k)
    _flat(logits, "logits", dev, logits.dtype, logits.shape)
    _flat(ids, "ids", dev, torch.int32, shape)
    _flat(grad_weights, "grad_weights", dev, torch.float32, shape)
    if out is None:
        out = _new(logits.shape, logits.dtype, dev)
    else:
        _flat(out, "out", dev, logits.dtype, logits.shape)
        _written(out)
    _call(lib.moe_ep_route_top_k_backward, _ROUTE_GRAD, dev, logits.data_ptr(), ids.data_ptr(), grad_weights.data_ptr(),
          out.data_ptr(), T, E, k, 1 if renormalize else 0, rt, scale, 0)
    return out


class _RouteFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k, renormalize, scale):
        r = _route(logits, top_k, renormalize, scale, None, None, None)
        if logits.untyped_storage().nbytes() != logits.numel() * logits.element_size():
            # a part of a workspace, which the next dispatch overwrites unseen by autograd
            logits = logits.clone()
        ctx.save_for_backward(logits, r.ids)
        ctx.rule = renormalize, scale
        ctx.mark_non_differentiable(r.ids)
        ctx.set_materialize_grads(False)
        return tuple(r)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _, grad):
        if grad is None:
            return (None,) * 4
        logits, ids = ctx.saved_tensors
        renormalize, scale = ctx.rule
        return route_top_k_backward(logits, ids, _whole(grad), renormalize=renormalize, scale=scale), None, None, None
