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
    mxfp4_grouped_matmul_act(a, a_scales, b, b_scales, c, group_list=None,
                             act="none", bias=None, residual=None, z=None)
    mxfp4_act_bwd(grad_c, z, grad_z, act="none", grad_bias=None, group_list=None)

logits, x, h, y and gradients are bfloat16 or float32; weights, biases and
their gradients float32; ids and rows int32 [tokens, k]; group_list int64
[experts].
"""
from __future__ import annotations

import ctypes

import torch

from . import (_FP8, FLOOR, _check, _Desc, _dtype, _group_list, _load, _MxOperand, _need, _operand, _ptr, _stream)

__all__ = ["mxfp4_moe_route", "mxfp4_moe_route_bwd", "mxfp4_moe_plan", "mxfp4_moe_plan_workspace",
           "mxfp4_moe_dispatch", "mxfp4_moe_combine", "mxfp4_moe_combine_bwd", "ACTIVATIONS",
           "mxfp4_grouped_matmul_act", "mxfp4_act_bwd"]

# the last two are gated: act(gate) * up
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "swiglu": 6, "geglu": 7}
_SCORES = {"softmax": 0, "sigmoid": 1}


class _Route(ctypes.Structure):
    """mxfp4_moe_route_t (include/mxfp4.h)."""
    _fields_ = [("dtype", ctypes.c_int32), ("score", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("experts", ctypes.c_int32), ("tokens", ctypes.c_int64), ("k", ctypes.c_int32),
                ("num_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class _Epilogue(ctypes.Structure):
    """mxfp4_epilogue_t (include/mxfp4.h)."""
    _fields_ = [("act", ctypes.c_int32), ("reserved", ctypes.c_int32), ("bias", ctypes.c_void_p),
                ("bias_stride", ctypes.c_int64), ("residual", ctypes.c_void_p), ("ld_residual", ctypes.c_int64),
                ("z", ctypes.c_void_p), ("ld_z", ctypes.c_int64)]


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
        op = ctypes.POINTER(_MxOperand)
        lib.mxfp4_grouped_matmul_act.argtypes = [i64, i64, i64, op, op, vp, i32, i32, ctypes.POINTER(_Epilogue), i32, vp,
                                                 i64, vp]
        lib.mxfp4_act_bwd_workspace.argtypes = [i32, i64, i64, i32]
        lib.mxfp4_act_bwd_workspace.restype = i64
        lib.mxfp4_act_bwd.argtypes = [i32, i32, i64, i64, vp, vp, vp, vp, vp, i32, i32, vp, i64, vp]
        for f in ("mxfp4_grouped_matmul_act", "mxfp4_act_bwd", "mxfp4_moe_route", "mxfp4_moe_route_bwd", "mxfp4_moe_plan", "mxfp4_moe_dispatch",
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


def _act(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def mxfp4_grouped_matmul_act(a, a_scales, b, b_scales, c, group_list=None, act="none", bias=None, residual=None, z=None,
                             K=None, group_list_type=1, a_fmt="e4m3", b_fmt="e2m1", a_block=32, b_block=32):
    """Grouped MX product with its epilogue, c = act(A B_g^T + bias_g) + residual.

    a [M, lda] fp8 codes + a_scales; b [N, ldb] or [G, N, ldb] codes + scales of
    the same rank; c bf16 / f32 [M, N], for the gated "swiglu" and "geglu" [M, N
    / 2] with b's first N / 2 rows the gate; bias float32 [N] or [G, N]; residual
    c's shape and type (c itself may be given); z [M, N] of c's type receives
    the products before the activation.  K defaults to a's row length."""
    code = _act(act)
    if c is None or c.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("c must be a bfloat16 or float32 tensor")
    M = _matrix(a, "a")[0]
    n_list = 0 if group_list is None else (group_list.numel() if isinstance(group_list, torch.Tensor)
                                           else len(group_list))
    if a_scales is None or a_scales.dim() != 2 or a_scales.shape[0] < M:
        raise ValueError(f"a_scales must have M={M} rows")
    if b is None or b_scales is None or b.dim() < 2 or b_scales.dim() < 2 or b_scales.shape[-2] != b.shape[-2]:
        raise ValueError("b_scales must have as many rows as b")
    groups = max(n_list, 1)
    if b.dim() == 3 and (b.shape[0] < groups or b_scales.shape[0] < groups):
        raise ValueError(f"b and b_scales must hold one matrix per group ({groups})")
    nb = b.shape[-2]
    if code & 4 and nb % 2:
        raise ValueError(f"a gated activation needs an even number of rows of b, got {nb}")
    N = nb // 2 if code & 4 else nb
    _same_shape(c, (M, N), "c")
    _same_shape(residual, (M, N), "residual")
    _same_shape(z, (M, nb), "z")
    if bias is not None and tuple(bias.shape) not in ((nb,), (groups, nb)):
        raise ValueError(f"bias must be [{nb}] or [{groups}, {nb}], got {list(bias.shape)}")
    if K is None:
        K = a.shape[1]
    oa = _operand(a, a_scales, a_fmt, a_block)
    ob = _operand(b, b_scales, b_fmt, b_block)
    gl = _group_list(group_list, M, group_list_type)
    ep = _Epilogue(code, 0, _value(_typed_ptr(bias, torch.float32, "bias")),
                   nb if bias is not None and bias.dim() == 2 else 0,
                   _value(_typed_ptr(residual, c.dtype, "residual")), N, _value(_typed_ptr(z, c.dtype, "z")), nb)
    st = _lib().mxfp4_grouped_matmul_act(M, N, int(K), ctypes.byref(oa), ctypes.byref(ob), _ptr(gl, "i64"),
                                         0 if gl is None else gl.numel(), int(group_list_type), ctypes.byref(ep),
                                         1 if c.dtype == torch.float32 else 0, _ptr(c), N, _stream())
    _check(st, "mxfp4_grouped_matmul_act")


def _value(p):
    return None if p is None else p.value


def mxfp4_act_bwd(grad_c, z, grad_z, act="none", grad_bias=None, group_list=None, group_list_type=1, workspace=None):
    """Backward of the epilogue: grad_z (z's shape) from grad_c and z, and
    grad_bias float32 [columns of z] or [G, columns of z].  workspace: a uint8
    tensor of mxfp4_act_bwd_workspace bytes for grad_bias; allocated from torch
    when None."""
    code = _act(act)
    rows, cols = _matrix(grad_c, "grad_c")
    zc = cols * (2 if code & 4 else 1)
    _same_shape(z, (rows, zc), "z")
    _same_shape(grad_z, (rows, zc), "grad_z")
    if z is None or grad_z is None:
        raise ValueError("z and grad_z are required")
    gl = _group_list(group_list, rows, group_list_type)
    groups = 0 if gl is None else gl.numel()
    need = 0
    if grad_bias is not None:
        if tuple(grad_bias.shape) not in ((max(groups, 1), zc),) + (((zc,),) if groups <= 1 else ()):
            raise ValueError(f"grad_bias must be [{groups or 1}, {zc}], got {list(grad_bias.shape)}")
        need = int(_lib().mxfp4_act_bwd_workspace(code, rows, cols, groups))
        if workspace is None:
            workspace = torch.empty(max(need, 4), dtype=torch.uint8, device=grad_c.device)
        _need(workspace, need, "workspace")
    st = _lib().mxfp4_act_bwd(_dtype(grad_c), code, rows, cols, _ptr(grad_c), _typed_ptr(z, grad_c.dtype, "z"),
                              _typed_ptr(grad_z, grad_c.dtype, "grad_z"),
                              _typed_ptr(grad_bias, torch.float32, "grad_bias"), _ptr(gl, "i64"), groups,
                              int(group_list_type), _ptr(workspace, "u8") if need else None, need, _stream())
    _check(st, "mxfp4_act_bwd")
