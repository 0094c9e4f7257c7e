"""The low-rank adapters' and the gradient norm's entry points of the binding
(include/mxfp4.h).

As in the package's other calls: torch tensors in and out, outputs given by
the caller, enqueued on torch's current stream, argument checks here and in
the library, no CPU path.

    mxfp4_adapter_fwd(x, a, b, y, ids=None, scale=None, base=None, u=None)
    mxfp4_adapter_bwd(grad_y, a, b, x=None, u=None, ids=None, scale=None,
                      grad_x=None, grad_a=None, grad_b=None, base=None)
    mxfp4_grad_norm(grads, norm, norm_type=2.0)
    mxfp4_grad_clip(grads, max_norm, norm, outs=None, norm_type=2.0,
                    compute_norm=True)

x, y, base, grad_y and grad_x are 2-D with contiguous elements in a row and any
distance between rows (columns of a wider matrix, for instance); a [adapters,
rank, in] and b [adapters, out, rank] are contiguous, as are gradients to be
clipped.  All of one call's tensors are bfloat16 or all float32 (the gradients of
one norm may mix them); scale, u and norm float32; ids int32 [tokens].
"""
from __future__ import annotations

import math
import struct

import torch

from . import _check, _load, _need, _ptr, _stream
from .moe_ops import _arg, _given, _own

__all__ = ["mxfp4_adapter_fwd", "mxfp4_adapter_workspace", "mxfp4_adapter_bwd", "mxfp4_adapter_bwd_workspace",
           "mxfp4_grad_norm", "mxfp4_grad_norm_workspace", "mxfp4_grad_clip"]

_ADAPTER = struct.Struct("@iiiiqqq")   # mxfp4_adapter_t
_ITEM = struct.Struct("@PPqii")        # mxfp4_grad_item_t
_F32, _I32, _BF16 = torch.float32, torch.int32, torch.bfloat16
_CODES = {_F32: 0, _BF16: 1}
_NORMS = {math.inf: 0, 1.0: 1, 2.0: 2}

_typed = False


def _lib():
    global _typed
    lib = _load()
    if not _typed:
        import ctypes
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        dp = vp  # a struct's bytes
        lib.mxfp4_adapter_workspace.argtypes = [dp]
        lib.mxfp4_adapter_fwd.argtypes = [dp, vp, i64, vp, vp, vp, vp, vp, i64, vp, i64, vp, vp, i64, vp]
        lib.mxfp4_adapter_bwd_workspace.argtypes = [dp, i32, i32]
        lib.mxfp4_adapter_bwd.argtypes = [dp, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, i64, vp, i64, vp, vp, vp, i64,
                                          vp]
        lib.mxfp4_grad_norm_workspace.argtypes = [i32, i64]
        lib.mxfp4_grad_norm.argtypes = [i32, i32, vp, vp, vp, i64, vp]
        lib.mxfp4_grad_clip.argtypes = [i32, i32, vp, ctypes.c_float, i32, vp, vp, i64, vp]
        for f in ("mxfp4_adapter_workspace", "mxfp4_adapter_bwd_workspace", "mxfp4_grad_norm_workspace"):
            getattr(lib, f).restype = i64
        for f in ("mxfp4_adapter_fwd", "mxfp4_adapter_bwd", "mxfp4_grad_norm", "mxfp4_grad_clip"):
            getattr(lib, f).restype = i32
        _typed = True
    return lib


def _here(*tensors):
    """All on the current GPU, whose stream the call takes."""
    at = -1
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d < 0:
                raise ValueError("tensors must live on the GPU (no CPU path)")
            if d != at:
                if at >= 0 or d != torch.cuda.current_device():
                    raise ValueError("tensors must live on the current GPU")
                at = d


def _rows(t, shape, dtype, what):
    """Address of a 2-D tensor of this shape and type, and elements between its
    rows (None: 0, 0)."""
    if t is None:
        return None, 0
    if t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{what} is a {dtype} tensor, got {t.dtype}")
    rows, cols = shape
    ld, one = t.stride()
    if cols > 1 and one != 1:
        raise ValueError(f"the elements of a row of {what} must be contiguous")
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError(f"the rows of {what} must not overlap")
    return t.data_ptr(), ld


def _adapter(tokens, a, b, dtype):
    """mxfp4_adapter_t of a [adapters, rank, in] and b [adapters, out, rank]."""
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a and b must be 3-D: [adapters, rank, in] and [adapters, out, rank]")
    n, rank, n_in = a.shape
    nb, n_out, rb = b.shape
    if nb != n or rb != rank:
        raise ValueError(f"b must be [{n}, out, {rank}], got {list(b.shape)}")
    if dtype not in _CODES:
        raise ValueError(f"element dtype must be bfloat16 or float32, got {dtype}")
    return _ADAPTER.pack(_CODES[dtype], rank, n, 0, tokens, n_in, n_out), n, rank, n_in, n_out


def _matrix(t, what):
    if t is None or t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D tensor")
    return t.shape[0]


def _space(workspace, need, device, name):
    if need < 0:
        raise ValueError(f"{name}: {_load().mxfp4_last_error().decode()}")
    if need and workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if need:
        _need(workspace, need, "workspace")
    return workspace


def mxfp4_adapter_workspace(tokens: int, a, b) -> int:
    """Bytes of workspace that mxfp4_adapter_fwd needs."""
    n = int(_lib().mxfp4_adapter_workspace(_adapter(int(tokens), a, b, a.dtype)[0]))
    if n < 0:
        raise ValueError(f"mxfp4_adapter_workspace: {_load().mxfp4_last_error().decode()}")
    return n


def mxfp4_adapter_fwd(x, a, b, y, ids=None, scale=None, base=None, u=None, workspace=None):
    """Low-rank adapters beside a shared projection: y[t] = base[t] + scale[i]
    * (x[t] a[i]^T) b[i]^T with i = ids[t] (adapter 0 for all without ids; an id
    outside [0, adapters): no adapter).  base may be y itself, or None (0); u
    [tokens, rank] float32, when given, receives x[t] a[i]^T for the backward
    pass.  workspace: a uint8 tensor of mxfp4_adapter_workspace bytes; allocated
    from torch when None."""
    tokens, dt = _matrix(x, "x"), x.dtype
    d, n, rank, n_in, n_out = _adapter(tokens, a, b, dt)
    px, ldx = _rows(x, (tokens, n_in), dt, "x")
    py, ldy = _rows(_given(y, "y"), (tokens, n_out), dt, "y")
    pb, ldb = _rows(base, (tokens, n_out), dt, "base")
    args = (_own(a, dt, "a"), _own(b, dt, "b"), _arg(scale, (n,), _F32, "scale"), _arg(ids, (tokens,), _I32, "ids"))
    pu = _arg(u, (tokens, rank), _F32, "u")
    _here(x, a, b, y, ids, scale, base, u, workspace)
    lib = _lib()
    need = int(lib.mxfp4_adapter_workspace(d))
    workspace = _space(workspace, need, x.device, "mxfp4_adapter_fwd")
    _check(lib.mxfp4_adapter_fwd(d, px, ldx, *args, pb, ldb, py, ldy, pu, _ptr(workspace, "u8") if need else None, need,
                                 _stream()), "mxfp4_adapter_fwd")


def mxfp4_adapter_bwd_workspace(tokens: int, a, b, grad_a: bool = True, grad_b: bool = True) -> int:
    """Bytes of workspace that mxfp4_adapter_bwd needs for the gradients wanted."""
    n = int(_lib().mxfp4_adapter_bwd_workspace(_adapter(int(tokens), a, b, a.dtype)[0], bool(grad_a), bool(grad_b)))
    if n < 0:
        raise ValueError(f"mxfp4_adapter_bwd_workspace: {_load().mxfp4_last_error().decode()}")
    return n


def mxfp4_adapter_bwd(grad_y, a, b, x=None, u=None, ids=None, scale=None, grad_x=None, grad_a=None, grad_b=None,
                      base=None, workspace=None):
    """Gradients of mxfp4_adapter_fwd, each written where a tensor is given:
    grad_x (base, the gradient by way of the shared projection, is added; it may
    be grad_x itself), grad_a (needs x) and grad_b (needs u as the forward pass
    wrote it).  workspace: a uint8 tensor of mxfp4_adapter_bwd_workspace bytes;
    allocated from torch when None."""
    tokens, dt = _matrix(grad_y, "grad_y"), grad_y.dtype
    d, n, rank, n_in, n_out = _adapter(tokens, a, b, dt)
    if grad_x is None and grad_a is None and grad_b is None:
        raise ValueError("grad_x, grad_a or grad_b is required")
    if grad_a is not None and x is None:
        raise ValueError("grad_a needs x")
    if grad_b is not None and u is None:
        raise ValueError("grad_b needs u")
    if base is not None and grad_x is None:
        raise ValueError("base is added to grad_x, which is not given")
    pg, ldg = _rows(grad_y, (tokens, n_out), dt, "grad_y")
    px, ldx = _rows(x, (tokens, n_in), dt, "x")
    pgx, ldgx = _rows(grad_x, (tokens, n_in), dt, "grad_x")
    pb, ldb = _rows(base, (tokens, n_in), dt, "base")
    args = (_own(a, dt, "a"), _own(b, dt, "b"), _arg(scale, (n,), _F32, "scale"), _arg(ids, (tokens,), _I32, "ids"),
            _arg(u, (tokens, rank), _F32, "u"))
    pga, pgb = _arg(grad_a, a.shape, dt, "grad_a"), _arg(grad_b, b.shape, dt, "grad_b")
    _here(grad_y, a, b, x, u, ids, scale, grad_x, grad_a, grad_b, base, workspace)
    lib = _lib()
    need = int(lib.mxfp4_adapter_bwd_workspace(d, grad_a is not None, grad_b is not None))
    workspace = _space(workspace, need, grad_y.device, "mxfp4_adapter_bwd")
    _check(lib.mxfp4_adapter_bwd(d, pg, ldg, px, ldx, *args, pb, ldb, pgx, ldgx, pga, pgb,
                                 _ptr(workspace, "u8") if need else None, need, _stream()), "mxfp4_adapter_bwd")


# ---- the gradient norm ----------------------------------------------------------

_pack = None


def _listed(tensors):
    """A list that the caller holds until the kernels are under way: a generator's tensors
    would be freed once their addresses are taken, and the workspace allocated over them."""
    if isinstance(tensors, torch.Tensor):
        raise TypeError("grads and outs are lists of tensors")
    return tensors if tensors is None or isinstance(tensors, (list, tuple)) else list(tensors)


def _items(grads, outs, write):
    """mxfp4_grad_item_t of every tensor, checked, and the number of elements."""
    global _pack
    if _pack is None:
        try:
            from ._tensor_list import pack
        except ImportError as e:
            raise RuntimeError("_tensor_list is not built; build it with "
                               "`python -m mxfp4_fake_quantization_amd.build`") from e
        _pack = pack
    gpu = torch.cuda.is_initialized() or torch.cuda.is_available()  # (the second one asks the driver)
    return _pack(grads, outs, torch.cuda.current_device() if gpu else -1, write)


def _norm_type(p) -> int:
    code = _NORMS.get(float(p))
    if code is None:
        raise ValueError(f"norm_type must be 1, 2 or inf, got {p!r}")
    return code


def _norm_out(norm):
    if norm is None or norm.numel() != 1:
        raise ValueError("norm must hold one element")
    return _own(norm, _F32, "norm")


def mxfp4_grad_norm_workspace(tensors: int, elements: int) -> int:
    """Bytes of workspace that mxfp4_grad_norm and mxfp4_grad_clip need."""
    n = int(_lib().mxfp4_grad_norm_workspace(int(tensors), int(elements)))
    if n < 0:
        raise ValueError("the numbers of tensors and elements must be >= 0")
    return n


def mxfp4_grad_norm(grads, norm, norm_type=2.0, workspace=None):
    """norm (one float32 element) = the 1-, 2- or inf-norm over all elements of a
    list of gradients, summed in 64 bits.  workspace: a uint8 tensor of
    mxfp4_grad_norm_workspace bytes; allocated from torch when None."""
    order, pn, grads = _norm_type(norm_type), _norm_out(norm), _listed(grads)
    items, elements = _items(grads, None, False)
    _here(norm, workspace)
    lib, n = _lib(), len(items) // _ITEM.size
    need = int(lib.mxfp4_grad_norm_workspace(n, elements))
    workspace = _space(workspace, need, norm.device, "mxfp4_grad_norm")
    _check(lib.mxfp4_grad_norm(order, n, items, pn, _ptr(workspace, "u8") if need else None, need, _stream()),
           "mxfp4_grad_norm")


def mxfp4_grad_clip(grads, max_norm, norm, outs=None, norm_type=2.0, compute_norm=True, workspace=None):
    """Every gradient times min(1, max_norm / (norm + 1e-6)), in place or into
    ``outs``.  norm (one float32 element) receives the norm of ``grads``; without
    ``compute_norm`` it is read instead (a norm over several processes).  What is
    written may overlap nothing else: a tensor given twice is refused."""
    order, pn, grads, outs = _norm_type(norm_type), _norm_out(norm), _listed(grads), _listed(outs)
    items, elements = _items(grads, outs, True)
    _here(norm, workspace)
    lib, n = _lib(), len(items) // _ITEM.size
    need = int(lib.mxfp4_grad_norm_workspace(n, elements)) if compute_norm else 0
    workspace = _space(workspace, need, norm.device, "mxfp4_grad_clip")
    _check(lib.mxfp4_grad_clip(order, n, items, float(max_norm), 1 if compute_norm else 0, pn,
                               _ptr(workspace, "u8") if need else None, need, _stream()), "mxfp4_grad_clip")
