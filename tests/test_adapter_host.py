"""Refusals of the low-rank adapters' and the gradient norm's calls, on the CPU:
the binding's own (shapes, types, missing arguments) and the C ABI's (every call
fails validation or has nothing to do, so nothing is launched)."""
import ctypes
import math
import os

import pytest
import torch

import mxfp4_fake_quantization_amd as M
from mxfp4_fake_quantization_amd import adapter_ops

OK, EINVAL, EUNSUP = 0, 1, 2
F32, BF16 = 0, 1
A = [0x10000 * (i + 1) for i in range(14)]  # aligned addresses that are never read
f32, bf16, i32, u8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


def t(*shape, dtype=bf16):
    return torch.empty(shape, dtype=dtype)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.library_path()):
        pytest.fail("libmxfp4.so is not built (python -m mxfp4_fake_quantization_amd.build)")
    return adapter_ops._lib()


def refused(match, f, *a, **k):
    with pytest.raises(ValueError, match=match):
        f(*a, **k)


def test_binding_forward():
    x, a, b, y = t(4, 64), t(3, 8, 64), t(3, 96, 8), t(4, 96)
    f = M.mxfp4_adapter_fwd
    refused("2-D", f, t(64), a, b, y)
    refused("3-D", f, x, t(8, 64), b, y)
    refused("3-D", f, x, a, t(96, 8), y)
    refused("b must be", f, x, a, t(2, 96, 8), y)
    refused("b must be", f, x, a, t(3, 96, 7), y)
    refused("x must be", f, t(4, 63), a, b, y)
    refused("y must be", f, x, a, b, t(4, 95))
    refused("y must be", f, x, a, b, t(5, 96))
    refused("y is required", f, x, a, b, None)
    refused("base must be", f, x, a, b, y, base=t(4, 95))
    refused("base is a", f, x, a, b, y, base=t(4, 96, dtype=f32))
    refused("a is a", f, x, t(3, 8, 64, dtype=f32), b, y)
    refused("b is a", f, x, a, t(3, 96, 8, dtype=f32), y)
    refused("dtype", f, t(4, 64, dtype=torch.float16), a, b, y)
    refused("scale", f, x, a, b, y, scale=t(2, dtype=f32))
    refused("scale is", f, x, a, b, y, scale=t(3))
    refused("ids must", f, x, a, b, y, ids=t(5, dtype=i32))
    refused("ids is", f, x, a, b, y, ids=t(4, dtype=torch.int64))
    refused("u must", f, x, a, b, y, u=t(4, 7, dtype=f32))
    refused("u is", f, x, a, b, y, u=t(4, 8))
    refused("contiguous", f, x, t(3, 64, 8).transpose(1, 2), b, y)
    refused("elements of a row of x", f, t(64, 4).t(), a, b, y)
    refused("rows of y must not overlap", f, x, a, b, t(1, 96).expand(4, 96))
    refused("GPU", f, x, a, b, y)


def test_binding_backward():
    gy, a, b = t(4, 96), t(3, 8, 64), t(3, 96, 8)
    x, u = t(4, 64), t(4, 8, dtype=f32)
    f = M.mxfp4_adapter_bwd
    refused("is required", f, gy, a, b)
    refused("grad_a needs x", f, gy, a, b, u=u, grad_a=a)
    refused("grad_b needs u", f, gy, a, b, x=x, grad_b=b)
    refused("base is added", f, gy, a, b, x=x, grad_a=a, base=x)
    refused("grad_y must be", f, t(4, 95), a, b, grad_x=x)
    refused("grad_x must be", f, gy, a, b, grad_x=t(4, 63))
    refused("grad_a must be", f, gy, a, b, x=x, grad_a=t(3, 8, 63))
    refused("grad_b must be", f, gy, a, b, u=u, grad_b=t(3, 8, 96))
    refused("grad_a is a", f, gy, a, b, x=x, grad_a=t(3, 8, 64, dtype=f32))
    refused("x must be", f, gy, a, b, x=t(5, 64), grad_a=a)
    refused("u must be", f, gy, a, b, u=t(4, 9, dtype=f32), grad_b=b)
    refused("GPU", f, gy, a, b, grad_x=x)


def test_binding_norm():
    n, g = t(1, dtype=f32), [t(4), t(3, 3, dtype=f32)]
    refused("norm_type", M.mxfp4_grad_norm, g, n, norm_type=3)
    refused("norm_type", M.mxfp4_grad_norm, g, n, norm_type=0)
    refused("one element", M.mxfp4_grad_norm, g, t(2, dtype=f32))
    refused("norm is", M.mxfp4_grad_norm, g, t(1))
    refused("bfloat16 or float32", M.mxfp4_grad_norm, [t(4, dtype=torch.float16)], n)
    refused("contiguous", M.mxfp4_grad_norm, [t(4, 6).t()], n)
    refused("GPU", M.mxfp4_grad_norm, g, n)
    with pytest.raises(TypeError, match="list"):
        M.mxfp4_grad_norm(g[0], n)
    refused("outs must", M.mxfp4_grad_clip, g, 1.0, n, outs=[g[0]])
    refused("outs must", M.mxfp4_grad_clip, g, 1.0, n, outs=[t(5), g[1]])
    refused("outs must", M.mxfp4_grad_clip, g, 1.0, n, outs=[t(4, dtype=f32), g[1]])
    refused("GPU", M.mxfp4_grad_clip, g, 1.0, n)
    assert M.mxfp4_grad_norm_workspace(3, 10_000_000) > 0
    refused("must be", M.mxfp4_grad_norm_workspace, -1, 5)


def desc(dtype=BF16, rank=8, adapters=3, reserved=0, tokens=4, n_in=64, n_out=96):
    return adapter_ops._ADAPTER.pack(dtype, rank, adapters, reserved, tokens, n_in, n_out)


def fwd(lib, d, x=A[0], ldx=64, a=A[1], b=A[2], scale=None, ids=None, base=None, ldb=0, y=A[3], ldy=96, u=None, ws=A[4],
        nbytes=1 << 40):
    return lib.mxfp4_adapter_fwd(d, x, ldx, a, b, scale, ids, base, ldb, y, ldy, u, ws, nbytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), EUNSUP), (dict(rank=0), EUNSUP), (dict(rank=129), EUNSUP), (dict(adapters=0), EINVAL),
    (dict(reserved=1), EINVAL), (dict(tokens=-1), EINVAL), (dict(tokens=1 << 27), EUNSUP), (dict(n_in=0), EINVAL),
    (dict(n_out=0), EINVAL), (dict(n_in=1 << 25), EUNSUP), (dict(tokens=1 << 25, n_out=1 << 12), EUNSUP)])
def test_abi_descriptors(lib, bad, status):
    d = desc(**bad)
    assert fwd(lib, d) == status
    assert M.mxfp4_last_error()
    assert lib.mxfp4_adapter_workspace(d) == -1 and lib.mxfp4_adapter_bwd_workspace(d, 1, 1) == -1
    assert bwd(lib, d, gx=A[3]) == status
    assert fwd(lib, None) == EINVAL


def test_abi_forward(lib):
    assert fwd(lib, desc(tokens=0), x=None, a=None, b=None, y=None, ws=None, nbytes=0) == OK
    for k in ("x", "a", "b", "y"):
        assert fwd(lib, desc(), **{k: None}) == EINVAL, k
    many = desc(tokens=4000)                                      # few rows need no workspace
    assert fwd(lib, many, ws=None) == EINVAL
    assert fwd(lib, desc(), x=A[0] + 1) == EINVAL
    assert fwd(lib, desc(dtype=F32), x=A[0] + 2) == EINVAL
    assert fwd(lib, many, ws=A[4] + 8) == EINVAL
    assert fwd(lib, desc(), ldx=63) == EINVAL
    assert fwd(lib, desc(), ldy=95) == EINVAL
    assert fwd(lib, desc(), base=A[5], ldb=95) == EINVAL
    assert fwd(lib, desc(), base=A[3], ldb=100) == EINVAL         # over y, with other rows
    assert fwd(lib, desc(), ids=A[5] + 2) == EINVAL
    assert fwd(lib, desc(), u=A[5] + 2) == EINVAL
    assert fwd(lib, desc(), scale=A[5] + 2) == EINVAL
    need = lib.mxfp4_adapter_workspace(many)
    assert need >= 4 * 4000 * 8
    assert fwd(lib, many, nbytes=need - 1) == EINVAL
    for k in ("x", "a", "b"):                                     # y over an input
        assert fwd(lib, desc(), **{k: A[3]}) == EINVAL, k
    assert fwd(lib, desc(), u=A[4]) == EINVAL                     # u over the workspace


def bwd(lib, d, gy=A[0], ldg=96, x=A[1], ldx=64, a=A[2], b=A[3 + 4], scale=None, ids=None, u=A[5], base=None, ldb=0, gx=None,
        ldgx=64, ga=None, gb=None, ws=A[6], nbytes=1 << 50):
    return lib.mxfp4_adapter_bwd(d, gy, ldg, x, ldx, a, b, scale, ids, u, base, ldb, gx, ldgx, ga, gb, ws, nbytes, None)


def test_abi_backward(lib):
    gx, ga, gb = A[8], A[9], A[10]
    assert bwd(lib, desc()) == EINVAL                             # no output
    assert bwd(lib, desc(tokens=0), gy=None, x=None, a=None, b=None, u=None, ws=None, nbytes=0) == OK
    assert bwd(lib, desc(tokens=0), gx=gx, ws=None, nbytes=0) == OK
    full = dict(gx=gx, ga=ga, gb=gb)
    for k in ("gy", "x", "a", "b", "u", "ws"):
        assert bwd(lib, desc(), **full, **{k: None}) == EINVAL, k
    assert bwd(lib, desc(), **full, ldg=95) == EINVAL
    assert bwd(lib, desc(), **full, ldx=63) == EINVAL
    assert bwd(lib, desc(), **full, ldgx=63) == EINVAL
    assert bwd(lib, desc(), **full, base=A[11], ldb=63) == EINVAL
    assert bwd(lib, desc(), **full, base=gx, ldb=65) == EINVAL
    assert bwd(lib, desc(), gx=gx, ga=gx, gb=gb) == EINVAL        # outputs over one another
    assert bwd(lib, desc(), gx=A[0]) == EINVAL                    # over an input
    assert bwd(lib, desc(), ga=A[6]) == EINVAL                    # over the workspace
    assert bwd(lib, desc(adapters=1025), **full) == EUNSUP
    assert lib.mxfp4_adapter_bwd_workspace(desc(adapters=1025), 1, 1) == -1
    big = dict(adapters=1024, rank=128, n_in=1 << 14)             # the summed gradients fill 2^32 threads
    assert lib.mxfp4_adapter_bwd_workspace(desc(**big, n_out=1 << 14), 1, 1) == -1
    assert lib.mxfp4_adapter_bwd_workspace(desc(**big, n_out=1 << 13), 1, 1) > 0
    need = lib.mxfp4_adapter_bwd_workspace(desc(), 1, 1)
    assert lib.mxfp4_adapter_bwd_workspace(desc(), 0, 0) < need
    assert bwd(lib, desc(), **full, nbytes=need - 1) == EINVAL


def test_abi_norm(lib):
    item = adapter_ops._ITEM.pack

    def norm(items, p=2, n=None, out=A[1], ws=A[2], nbytes=1 << 40):
        return lib.mxfp4_grad_norm(p, len(items) if n is None else n, b"".join(items) or None, out, ws, nbytes, None)

    def clip(items, max_norm=1.0, compute=1, p=2, out=A[1], ws=A[2], nbytes=1 << 40):
        return lib.mxfp4_grad_clip(p, len(items), b"".join(items) or None, max_norm, compute, out, ws, nbytes, None)

    good = item(A[0], A[3], 100, BF16, 0)
    assert norm([good], p=3) == EUNSUP
    assert norm([good], out=None) == EINVAL
    assert norm([good], ws=None) == EINVAL
    assert norm([good], nbytes=0) == EINVAL
    assert norm([], n=1) == EINVAL
    assert norm([good], n=-1) == EINVAL
    assert norm([item(0, 0, 100, BF16, 0)]) == EINVAL
    assert norm([item(A[0] + 1, 0, 100, BF16, 0)]) == EINVAL
    assert norm([item(A[0] + 2, 0, 100, F32, 0)]) == EINVAL
    assert norm([item(A[0], 0, -1, F32, 0)]) == EINVAL
    assert norm([item(A[0], 0, 1 << 61, F32, 0)]) == EINVAL
    assert norm([item(A[0], 0, 100, 2, 0)]) == EUNSUP
    assert norm([item(A[0], 0, 100, F32, 1)]) == EINVAL
    assert clip([item(A[0], 0, 100, BF16, 0)]) == EINVAL          # no output
    assert clip([good], max_norm=-1.0) == EINVAL
    assert clip([good], max_norm=math.nan) == EINVAL
    assert clip([good], compute=2) == EINVAL
    assert clip([good], ws=None) == EINVAL
    assert clip([], compute=0, ws=None, nbytes=0) == OK           # nothing to do
    # what is written overlaps nothing: the same tensor twice, a part of it, another's output or gradient, the norm
    for other in (item(A[0], A[0], 100, BF16, 0), item(A[0] + 198, A[0] + 198, 100, BF16, 0),
                  item(A[4], A[0] + 100, 7, F32, 0), item(A[0] + 4, A[4], 7, BF16, 0),
                  item(A[1] - 4, A[1] - 4, 2, F32, 0), item(A[4], A[4] + 2, 5, BF16, 0), item(A[2], A[2], 4, F32, 0)):
        for pair in ([item(A[0], A[0], 100, BF16, 0), other], [other, item(A[0], A[0], 100, BF16, 0)]):
            assert clip(pair) == EINVAL
            assert b"overlaps" in lib.mxfp4_last_error()
    assert lib.mxfp4_grad_norm_workspace(-1, 5) == -1 and lib.mxfp4_grad_norm_workspace(1, -5) == -1


def test_scale_wants_no_gradient():
    from mxfp4_fake_quantization_amd.adapters import adapter_add
    x, base, a, b = torch.zeros(2, 8), torch.zeros(2, 6), torch.zeros(1, 3, 8), torch.zeros(1, 6, 3)
    with pytest.raises(ValueError, match="no gradient"):
        adapter_add(x, base, a, b, scale=torch.ones(1, requires_grad=True))


def test_abi_structs():
    """The packed structs have the sizes of the C ones."""
    assert adapter_ops._ADAPTER.size == 40 and adapter_ops._ITEM.size == 32

    class Item(ctypes.Structure):
        _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("count", ctypes.c_int64),
                    ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]

    assert ctypes.sizeof(Item) == 32
