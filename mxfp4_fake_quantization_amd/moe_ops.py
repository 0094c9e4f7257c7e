"""The mixture-of-experts entry points of the binding (include/mxfp4.h).

As in the package's other calls: torch tensors in and out, outputs given by
the caller, enqueued on torch's current stream, argument checks here and in
the library, no CPU path.

    mxfp4_moe_route(logits, weights, ids, bias=None, score="softmax",
                    num_groups=1, topk_groups=None, renormalize=True, scale=1.0)
    mxfp4_moe_route_bwd(grad_weights, logits, ids, grad_logits, score="softmax",
                        renormalize=True, scale=1.0)
    mxfp4_moe_plan(ids, group_list, rows, workspace=None)
    mxfp4_moe_dispatch(x, rows, y=None, q=None, scales=None, fmt="e4m3", block=32)
    mxfp4_moe_combine(h, rows, y, weights=None, residual=None)
    mxfp4_moe_combine_bwd(grad_y, h, rows, weights=None, grad_h=None,
                          grad_weights=None)

logits, x, h, y and gradients are bfloat16 or float32; weights, biases and
their gradients float32; ids and rows int32 [tokens, k]; group_list int64
[experts].
"""
from __future__ import annotations

import ctypes

import torch

from . import _FP8, FLOOR, _check, _Desc, _dtype, _load, _need, _ptr, _shape2d, _stream

__all__ = ["mxfp4_moe_route", "mxfp4_moe_route_bwd", "mxfp4_moe_plan", "mxfp4_moe_plan_workspace",
           "mxfp4_moe_dispatch", "mxfp4_moe_combine", "mxfp4_moe_combine_bwd"]

_SCORES = {"softmax": 0, "sigmoid": 1}


class _Route(ctypes.Structure):
    """mxfp4_moe_route_t (include/mxfp4.h)."""
    _fields_ = [("dtype", ctypes.c_int32), ("score", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("experts", ctypes.c_int32), ("tokens", ctypes.c_int64), ("k", ctypes.c_int32),
                ("num_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


_typed = False


def _lib():
    global _typed
    lib = _load()
    if not _typed:
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        rp, dp = ctypes.POINTER(_Route), ctypes.POINTER(_Desc)
        lib.mxfp4_moe_route.argtypes = [rp, vp, vp, vp, vp, vp]
        lib.mxfp4_moe_route_bwd.argtypes = [rp, vp, vp, vp, vp, vp]
        lib.mxfp4_moe_plan_workspace.argtypes = [i64, i32]
        lib.mxfp4_moe_plan_workspace.restype = i64
        lib.mxfp4_moe_plan.argtypes = [i64, i32, vp, vp, vp, vp, i64, vp]
        lib.mxfp4_moe_dispatch.argtypes = [dp, i32, vp, vp, i32, i64, vp, vp, vp, vp]
        lib.mxfp4_moe_combine.argtypes = [i32, i64, i64, i32, i64, vp, vp, vp, vp, vp, vp]
        lib.mxfp4_moe_combine_bwd.argtypes = [i32, i64, i64, i32, i64, vp, vp, vp, vp, vp, vp, vp]
        for f in ("mxfp4_moe_route", "mxfp4_moe_route_bwd", "mxfp4_moe_plan", "mxfp4_moe_dispatch",
                  "mxfp4_moe_combine", "mxfp4_moe_combine_bwd"):
            getattr(lib, f).restype = ctypes.c_int32
        _typed = True
    return lib


def _typed_ptr(t, dtype, what):
    if t is not None and t.dtype != dtype:
        raise ValueError(f"{what} is a {dtype} tensor, got {t.dtype}")
    return _ptr(t)


def _matrix(t, what):
    if t is None or t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D tensor")
    return t.shape


def _same_shape(t, shape, what):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")


def _route_desc(logits, k, score, num_groups, topk_groups, renormalize, scale):
    tokens, experts = _matrix(logits, "logits")
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    topk_groups = num_groups if topk_groups is None else topk_groups
    return _Route(_dtype(logits), _SCORES[score], 1 if renormalize else 0, experts, tokens, int(k), int(num_groups),
                  int(topk_groups), float(scale), 0)


def mxfp4_moe_route(logits, weights, ids, bias=None, score="softmax", num_groups=1, topk_groups=None,
                    renormalize=True, scale=1.0):
    """The k experts of every token and their weights: logits [tokens, experts]
    -> weights [tokens, k] float32 and ids [tokens, k] int32, k being ids'
    second dimension; see include/mxfp4.h."""
    tokens, k = _matrix(ids, "ids")
    d = _route_desc(logits, k, score, num_groups, topk_groups, renormalize, scale)
    _same_shape(ids, (d.tokens, k), "ids")
    _same_shape(weights, (d.tokens, k), "weights")
    _same_shape(bias, (d.experts,), "bias")
    st = _lib().mxfp4_moe_route(ctypes.byref(d), _ptr(logits), _typed_ptr(bias, torch.float32, "bias"),
                                _typed_ptr(weights, torch.float32, "weights"), _typed_ptr(ids, torch.int32, "ids"),
                                _stream())
    _check(st, "mxfp4_moe_route")


def mxfp4_moe_route_bwd(grad_weights, logits, ids, grad_logits, score="softmax", renormalize=True, scale=1.0):
    """Gradient of mxfp4_moe_route's weights with respect to the logits (the
    choice is constant; the bias moves the choice only and has none)."""
    tokens, k = _matrix(ids, "ids")
    d = _route_desc(logits, k, score, 1, 1, renormalize, scale)
    _same_shape(ids, (d.tokens, k), "ids")
    _same_shape(grad_weights, (d.tokens, k), "grad_weights")
    _same_shape(grad_logits, logits.shape, "grad_logits")
    st = _lib().mxfp4_moe_route_bwd(ctypes.byref(d), _typed_ptr(grad_weights, torch.float32, "grad_weights"),
                                    _ptr(logits), _typed_ptr(ids, torch.int32, "ids"),
                                    _typed_ptr(grad_logits, logits.dtype, "grad_logits"), _stream())
    _check(st, "mxfp4_moe_route_bwd")


def mxfp4_moe_plan_workspace(slots: int, experts: int) -> int:
    """Bytes of workspace that mxfp4_moe_plan needs (0 for few slots)."""
    n = int(_lib().mxfp4_moe_plan_workspace(int(slots), int(experts)))
    if n < 0:
        raise ValueError(f"mxfp4_moe_plan takes up to 2^31 - 1 slots and 1024 experts, got {slots} and {experts}")
    return n


def mxfp4_moe_plan(ids, group_list, rows, workspace=None):
    """Slots by expert: ids [tokens, k] -> group_list [experts] (the counts the
    grouped calls take) and rows, ids' shape (each slot's row in expert order;
    -1 where ids holds none).  workspace: a uint8 tensor of
    mxfp4_moe_plan_workspace bytes; allocated from torch when None."""
    _same_shape(rows, ids.shape, "rows")
    if group_list is None or group_list.dim() != 1:
        raise ValueError("group_list must be a 1-D tensor with one count per expert")
    slots, experts = ids.numel(), group_list.numel()
    need = mxfp4_moe_plan_workspace(slots, experts)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=ids.device)
    _need(workspace, need, "workspace")
    st = _lib().mxfp4_moe_plan(slots, experts, _typed_ptr(ids, torch.int32, "ids"), _ptr(group_list, "i64"),
                               _typed_ptr(rows, torch.int32, "rows"), _ptr(workspace, "u8") if need else None,
                               need, _stream())
    _check(st, "mxfp4_moe_plan")


def mxfp4_moe_dispatch(x, rows, y=None, q=None, scales=None, fmt="e4m3", block=32):
    """Token rows to their slots' rows: x [tokens, cols] -> y [n, cols] (x's
    type) and / or MXFP8 q [n, cols] with scales [n, ceil(cols / block)]."""
    tokens, cols = _matrix(x, "x")
    k = _matrix(rows, "rows")[1]
    _same_shape(rows, (tokens, k), "rows")
    if fmt not in _FP8:
        raise ValueError(f"fmt must be 'e4m3' or 'e5m2', got {fmt!r}")
    outs = [t.shape[0] for t in (y, q) if t is not None]
    if not outs or outs[0] != outs[-1]:
        raise ValueError("y and / or q with the same number of rows is required")
    n = outs[0]
    _same_shape(y, (n, cols), "y")
    _same_shape(q, (n, cols), "q")
    _same_shape(scales, (n, -(-cols // int(block))), "scales")
    d = _Desc(_dtype(x), int(block), FLOOR, 0, tokens, cols, 6.0, 0)
    st = _lib().mxfp4_moe_dispatch(ctypes.byref(d), _FP8[fmt], _ptr(x), _typed_ptr(rows, torch.int32, "rows"), k, n,
                                   _typed_ptr(y, x.dtype, "y"), _ptr(q, "u8"), _ptr(scales, "u8"), _stream())
    _check(st, "mxfp4_moe_dispatch")


def mxfp4_moe_combine(h, rows, y, weights=None, residual=None):
    """Expert rows back to the tokens: y[t] = residual[t] + sum_j weights[t, j]
    * h[rows[t, j]]; y may be the residual."""
    n, cols = _matrix(h, "h")
    tokens, k = _matrix(rows, "rows")
    _same_shape(y, (tokens, cols), "y")
    _same_shape(weights, (tokens, k), "weights")
    _same_shape(residual, (tokens, cols), "residual")
    if y is None:
        raise ValueError("y is required")
    st = _lib().mxfp4_moe_combine(_dtype(h), tokens, cols, k, n, _ptr(h), _typed_ptr(rows, torch.int32, "rows"),
                                  _typed_ptr(weights, torch.float32, "weights"),
                                  _typed_ptr(residual, h.dtype, "residual"), _typed_ptr(y, h.dtype, "y"), _stream())
    _check(st, "mxfp4_moe_combine")


def mxfp4_moe_combine_bwd(grad_y, h, rows, weights=None, grad_h=None, grad_weights=None):
    """Gradients of mxfp4_moe_combine: grad_h [n, cols] and / or grad_weights
    [tokens, k] (which needs h)."""
    tokens, cols = _matrix(grad_y, "grad_y")
    k = _matrix(rows, "rows")[1]
    _same_shape(rows, (tokens, k), "rows")
    if grad_weights is not None and h is None:
        raise ValueError("grad_weights needs h")
    sized = [t for t in (h, grad_h) if t is not None]
    if grad_h is None and grad_weights is None:
        raise ValueError("grad_h and / or grad_weights is required")
    n = sized[0].shape[0]
    for t, what in ((h, "h"), (grad_h, "grad_h")):
        _same_shape(t, (n, cols), what)
    _same_shape(weights, (tokens, k), "weights")
    _same_shape(grad_weights, (tokens, k), "grad_weights")
    st = _lib().mxfp4_moe_combine_bwd(_dtype(grad_y), tokens, cols, k, n, _ptr(grad_y),
                                      _typed_ptr(h, grad_y.dtype, "h"), _typed_ptr(rows, torch.int32, "rows"),
                                      _typed_ptr(weights, torch.float32, "weights"),
                                      _typed_ptr(grad_h, grad_y.dtype, "grad_h"),
                                      _typed_ptr(grad_weights, torch.float32, "grad_weights"), _stream())
    _check(st, "mxfp4_moe_combine_bwd")
