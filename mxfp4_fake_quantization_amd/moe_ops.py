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
import struct

import torch

from . import (_FP8, FLOOR, MX_FORMATS, _check, _Desc, _dtype, _group_list, _load, _MxOperand, _need, _ptr, _stream)

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


# The same structs as bytes: filling a ctypes structure and pointing at it takes
# about three times as long, which a small call's time shows.
_ROUTE = struct.Struct("@iiiiqiiifi4x")
_EPILOGUE = struct.Struct("@iiPqPqPq")
_DESC = struct.Struct("@iiiiqqfi")
_OPERAND = struct.Struct("@PPiiqqqq")
assert [f.size for f in (_ROUTE, _EPILOGUE, _DESC, _OPERAND)] == [
    ctypes.sizeof(c) for c in (_Route, _Epilogue, _Desc, _MxOperand)]

_typed = False


def _lib():
    global _typed
    lib = _load()
    if not _typed:
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        rp = dp = op = vp  # a struct's bytes, or ctypes.byref of one
        lib.mxfp4_moe_route.argtypes = [rp, vp, vp, vp, vp, vp]
        lib.mxfp4_moe_route_bwd.argtypes = [rp, vp, vp, vp, vp, vp]
        lib.mxfp4_moe_plan_workspace.argtypes = [i64, i32]
        lib.mxfp4_moe_plan_workspace.restype = i64
        lib.mxfp4_moe_plan.argtypes = [i64, i32, vp, vp, vp, vp, i64, vp]
        lib.mxfp4_moe_dispatch.argtypes = [dp, i32, vp, vp, i32, i64, vp, vp, vp, vp]
        lib.mxfp4_moe_combine.argtypes = [i32, i64, i64, i32, i64, vp, vp, vp, vp, vp, vp]
        lib.mxfp4_moe_combine_bwd.argtypes = [i32, i64, i64, i32, i64, vp, vp, vp, vp, vp, vp, vp]
        lib.mxfp4_grouped_matmul_act.argtypes = [i64, i64, i64, op, op, vp, i32, i32, vp, i32, vp,
                                                 i64, vp]
        lib.mxfp4_act_bwd_workspace.argtypes = [i32, i64, i64, i32]
        lib.mxfp4_act_bwd_workspace.restype = i64
        lib.mxfp4_act_bwd.argtypes = [i32, i32, i64, i64, vp, vp, vp, vp, vp, i32, i32, vp, i64, vp]
        for f in ("mxfp4_grouped_matmul_act", "mxfp4_act_bwd", "mxfp4_moe_route", "mxfp4_moe_route_bwd", "mxfp4_moe_plan", "mxfp4_moe_dispatch",
                  "mxfp4_moe_combine", "mxfp4_moe_combine_bwd"):
            getattr(lib, f).restype = ctypes.c_int32
        _typed = True
    return lib


def _matrix(t, what):
    if t is None or t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D tensor")
    return t.shape


def _arg(t, shape, dtype, what):
    """Address of a tensor of this shape and type (None stays None)."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{what} is a {dtype} tensor, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _own(t, dtype, what):
    """Address of a tensor of this type, of any shape (None stays None)."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise ValueError(f"{what} is a {dtype} tensor, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _on_gpu(*tensors):
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must live on the GPU (no CPU path)")


def _groups(group_list):
    if group_list is None:
        return 0
    return group_list.numel() if isinstance(group_list, torch.Tensor) else len(group_list)


def _list(gl):
    return _own(gl, _I64, "group_list")


def _given(t, what):
    if t is None:
        raise ValueError(f"{what} is required")
    return t


_F32, _I32, _I64, _U8 = torch.float32, torch.int32, torch.int64, torch.uint8


def _route_desc(logits, shape, k, score, num_groups, topk_groups, renormalize, scale):
    tokens, experts = shape
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    topk_groups = num_groups if topk_groups is None else topk_groups
    return _ROUTE.pack(_dtype(logits), _SCORES[score], 1 if renormalize else 0, experts, tokens, k, num_groups,
                       topk_groups, scale, 0)


def mxfp4_moe_route(logits, weights, ids, bias=None, score="softmax", num_groups=1, topk_groups=None,
                    renormalize=True, scale=1.0):
    """The k experts of every token and their weights: logits [tokens, experts]
    -> weights [tokens, k] float32 and ids [tokens, k] int32, k being ids'
    second dimension; see include/mxfp4.h."""
    k = _matrix(ids, "ids")[1]
    shape = tokens, experts = _matrix(logits, "logits")
    d = _route_desc(logits, shape, k, score, num_groups, topk_groups, renormalize, scale)
    args = (d, _own(logits, logits.dtype, "logits"), _arg(bias, (experts,), _F32, "bias"),
            _arg(_given(weights, "weights"), (tokens, k), _F32, "weights"), _arg(ids, (tokens, k), _I32, "ids"))
    _on_gpu(logits, weights, ids, bias)
    _check(_lib().mxfp4_moe_route(*args, _stream()), "mxfp4_moe_route")


def mxfp4_moe_route_bwd(grad_weights, logits, ids, grad_logits, score="softmax", renormalize=True, scale=1.0):
    """Gradient of mxfp4_moe_route's weights with respect to the logits (the
    choice is constant; the bias moves the choice only and has none)."""
    k = _matrix(ids, "ids")[1]
    shape = _matrix(logits, "logits")
    chosen = (shape[0], k)
    d = _route_desc(logits, shape, k, score, 1, 1, renormalize, scale)
    args = (d, _arg(_given(grad_weights, "grad_weights"), chosen, _F32, "grad_weights"),
            _own(logits, logits.dtype, "logits"), _arg(ids, chosen, _I32, "ids"),
            _arg(_given(grad_logits, "grad_logits"), shape, logits.dtype, "grad_logits"))
    _on_gpu(grad_weights, logits, ids, grad_logits)
    _check(_lib().mxfp4_moe_route_bwd(*args, _stream()), "mxfp4_moe_route_bwd")


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
    if group_list is None or group_list.dim() != 1:
        raise ValueError("group_list must be a 1-D tensor with one count per expert")
    shape, slots, experts = ids.shape, ids.numel(), group_list.numel()
    if _given(rows, "rows").shape != shape:
        raise ValueError(f"rows must be {list(shape)}, got {list(rows.shape)}")
    need = mxfp4_moe_plan_workspace(slots, experts)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=_U8, device=ids.device)
    _need(workspace, need, "workspace")
    args = (slots, experts, _own(ids, _I32, "ids"), _own(group_list, _I64, "group_list"), _own(rows, _I32, "rows"),
            _ptr(workspace, "u8") if need else None, need)
    _on_gpu(ids, group_list, rows)
    _check(_lib().mxfp4_moe_plan(*args, _stream()), "mxfp4_moe_plan")


def mxfp4_moe_dispatch(x, rows, y=None, q=None, scales=None, fmt="e4m3", block=32):
    """Token rows to their slots' rows: x [tokens, cols] -> y [n, cols] (x's
    type) and / or MXFP8 q [n, cols] with scales [n, ceil(cols / block)]."""
    shape = tokens, cols = _matrix(x, "x")
    k = _matrix(rows, "rows")[1]
    if fmt not in _FP8:
        raise ValueError(f"fmt must be 'e4m3' or 'e5m2', got {fmt!r}")
    outs = [t.shape[0] for t in (y, q) if t is not None]
    if not outs or outs[0] != outs[-1]:
        raise ValueError("y and / or q with the same number of rows is required")
    n = outs[0]
    block = int(block)
    args = (_DESC.pack(_dtype(x), block, FLOOR, 0, tokens, cols, 6.0, 0), _FP8[fmt], _own(x, x.dtype, "x"),
            _arg(rows, (tokens, k), _I32, "rows"), k, n,
            _arg(y, (n, cols), x.dtype, "y"), _arg(q, (n, cols), _U8, "q"),
            _arg(scales, (n, -(-cols // block)), _U8, "scales"))
    _on_gpu(x, rows, y, q, scales)
    _check(_lib().mxfp4_moe_dispatch(*args, _stream()), "mxfp4_moe_dispatch")


def mxfp4_moe_combine(h, rows, y, weights=None, residual=None):
    """Expert rows back to the tokens: y[t] = residual[t] + sum_j weights[t, j]
    * h[rows[t, j]]; y may be the residual."""
    n, cols = _matrix(h, "h")
    tokens, k = _matrix(rows, "rows")
    dt, out = h.dtype, (tokens, cols)
    args = (_dtype(h), tokens, cols, k, n, _own(h, dt, "h"), _own(rows, _I32, "rows"),
            _arg(weights, (tokens, k), _F32, "weights"), _arg(residual, out, dt, "residual"),
            _arg(_given(y, "y"), out, dt, "y"))
    _on_gpu(h, rows, y, weights, residual)
    _check(_lib().mxfp4_moe_combine(*args, _stream()), "mxfp4_moe_combine")


def mxfp4_moe_combine_bwd(grad_y, h, rows, weights=None, grad_h=None, grad_weights=None):
    """Gradients of mxfp4_moe_combine: grad_h [n, cols] and / or grad_weights
    [tokens, k] (which needs h)."""
    shape = tokens, cols = _matrix(grad_y, "grad_y")
    k = _matrix(rows, "rows")[1]
    if grad_weights is not None and h is None:
        raise ValueError("grad_weights needs h")
    if grad_h is None and grad_weights is None:
        raise ValueError("grad_h and / or grad_weights is required")
    n = (grad_h if h is None else h).shape[0]
    dt, chosen = grad_y.dtype, (tokens, k)
    args = (_dtype(grad_y), tokens, cols, k, n, _arg(grad_y, shape, dt, "grad_y"), _arg(h, (n, cols), dt, "h"),
            _arg(rows, chosen, _I32, "rows"), _arg(weights, chosen, _F32, "weights"),
            _arg(grad_h, (n, cols), dt, "grad_h"), _arg(grad_weights, chosen, _F32, "grad_weights"))
    _on_gpu(grad_y, h, rows, weights, grad_h, grad_weights)
    _check(_lib().mxfp4_moe_combine_bwd(*args, _stream()), "mxfp4_moe_combine_bwd")


def _mx(data, scales, shape, sshape, fmt, block):
    """mxfp4_mx_operand_t of codes [rows, ld] or [G, rows, ld] and their scales."""
    if fmt not in MX_FORMATS:
        raise ValueError(f"fmt must be one of {sorted(MX_FORMATS)}, got {fmt!r}")
    three = len(shape) == 3
    if len(sshape) != len(shape):
        raise ValueError("operand data and scales must have the same rank")
    ld, lds = shape[-1], sshape[-1]
    return _OPERAND.pack(_own(data, _U8, "operand data"), _own(scales, _U8, "operand scales"), MX_FORMATS[fmt], block,
                         ld, lds, shape[1] * ld if three else 0, sshape[1] * lds if three else 0)


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
    dt = None if c is None else c.dtype
    if dt is not torch.bfloat16 and dt is not _F32:
        raise ValueError("c must be a bfloat16 or float32 tensor")
    ashape = _matrix(a, "a")
    M = ashape[0]
    n_list = _groups(group_list)
    asshape = None if a_scales is None else a_scales.shape
    if asshape is None or len(asshape) != 2 or asshape[0] < M:
        raise ValueError(f"a_scales must have M={M} rows")
    bshape, bsshape = (None if t is None else t.shape for t in (b, b_scales))
    if bshape is None or bsshape is None or len(bshape) < 2 or len(bsshape) < 2 or bsshape[-2] != bshape[-2]:
        raise ValueError("b_scales must have as many rows as b")
    groups = max(n_list, 1)
    if len(bshape) == 3 and (bshape[0] < groups or bsshape[0] < groups):
        raise ValueError(f"b and b_scales must hold one matrix per group ({groups})")
    nb = bshape[-2]
    if code & 4 and nb % 2:
        raise ValueError(f"a gated activation needs an even number of rows of b, got {nb}")
    N = nb // 2 if code & 4 else nb
    per_group = False
    if bias is not None:
        per_group = bias.dim() == 2
        if bias.shape != ((groups, nb) if per_group else (nb,)):
            raise ValueError(f"bias must be [{nb}] or [{groups}, {nb}], got {list(bias.shape)}")
    K = ashape[1] if K is None else int(K)
    oa = _mx(a, a_scales, ashape, asshape, a_fmt, a_block)
    ob = _mx(b, b_scales, bshape, bsshape, b_fmt, b_block)
    out = (M, N)
    ep = _EPILOGUE.pack(code, 0, _own(bias, _F32, "bias") or 0, nb if per_group else 0,
                        _arg(residual, out, dt, "residual") or 0, N, _arg(z, (M, nb), dt, "z") or 0, nb)
    cp = _arg(c, out, dt, "c")
    _on_gpu(a, a_scales, b, b_scales, c, bias, residual, z)
    gl = _group_list(group_list, M, group_list_type)
    _check(_lib().mxfp4_grouped_matmul_act(M, N, K, oa, ob, _list(gl), n_list, int(group_list_type), ep,
                                           1 if dt is _F32 else 0, cp, N, _stream()), "mxfp4_grouped_matmul_act")


def mxfp4_act_bwd(grad_c, z, grad_z, act="none", grad_bias=None, group_list=None, group_list_type=1, workspace=None):
    """Backward of the epilogue: grad_z (z's shape) from grad_c and z, and
    grad_bias float32 [columns of z] or [G, columns of z].  workspace: a uint8
    tensor of mxfp4_act_bwd_workspace bytes for grad_bias; allocated from torch
    when None."""
    code = _act(act)
    shape = rows, cols = _matrix(grad_c, "grad_c")
    dt, zc = grad_c.dtype, cols * (2 if code & 4 else 1)
    groups, need = _groups(group_list), 0
    if grad_bias is not None:
        if tuple(grad_bias.shape) not in ((max(groups, 1), zc),) + (((zc,),) if groups <= 1 else ()):
            raise ValueError(f"grad_bias must be [{groups or 1}, {zc}], got {list(grad_bias.shape)}")
        need = int(_lib().mxfp4_act_bwd_workspace(code, rows, cols, groups))
        if workspace is None:
            workspace = torch.empty(max(need, 4), dtype=torch.uint8, device=grad_c.device)
        _need(workspace, need, "workspace")
    args = (_dtype(grad_c), code, rows, cols, _arg(grad_c, shape, dt, "grad_c"),
            _arg(_given(z, "z"), (rows, zc), dt, "z"), _arg(_given(grad_z, "grad_z"), (rows, zc), dt, "grad_z"),
            None if grad_bias is None else _arg(grad_bias, grad_bias.shape, _F32, "grad_bias"))
    _on_gpu(grad_c, z, grad_z, grad_bias)
    gl = _group_list(group_list, rows, group_list_type)
    st = _lib().mxfp4_act_bwd(*args, _list(gl), groups, int(group_list_type), _ptr(workspace, "u8") if need else None,
                              need, _stream())
    _check(st, "mxfp4_act_bwd")
