"""Refusals of the mixture-of-experts calls, on the CPU: the binding's own
(shapes, types, missing outputs) and the C ABI's (every call fails validation
or has nothing to do, so nothing is launched)."""
import ctypes
import os

import pytest
import torch

import mxfp4_fake_quantization_amd as M
from mxfp4_fake_quantization_amd.moe_ops import _Route

OK, EINVAL, EUNSUP = 0, 1, 2
F32, BF16 = 0, 1
P = ctypes.c_void_p
A = [0x10000 * (i + 1) for i in range(12)]  # aligned addresses that are never read


def t(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype)


i32, u8, i64, bf16 = torch.int32, torch.uint8, torch.int64, torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.library_path()):
        pytest.fail("libmxfp4.so is not built (python -m mxfp4_fake_quantization_amd.build)")
    from mxfp4_fake_quantization_amd import moe_ops
    return moe_ops._lib()


def refused(match, f, *a, **k):
    with pytest.raises(ValueError, match=match):
        f(*a, **k)


def test_binding_route():
    l, w, ids = t(4, 8), t(4, 2), t(4, 2, dtype=i32)
    refused("weights", M.mxfp4_moe_route, l, t(4, 3), ids)
    refused("ids", M.mxfp4_moe_route, l, w, t(5, 2, dtype=i32))
    refused("2-D", M.mxfp4_moe_route, t(8), w, ids)
    refused("score", M.mxfp4_moe_route, l, w, ids, score="tanh")
    refused("bias", M.mxfp4_moe_route, l, w, ids, bias=t(7))
    refused("dtype", M.mxfp4_moe_route, t(4, 8, dtype=torch.float16), w, ids)
    refused("GPU", M.mxfp4_moe_route, l, w, ids)
    refused("grad_logits", M.mxfp4_moe_route_bwd, w, l, ids, t(4, 7))
    refused("grad_weights", M.mxfp4_moe_route_bwd, t(4, 1), l, ids, t(4, 8))


def test_binding_rows():
    x, rows = t(4, 64, dtype=bf16), t(4, 2, dtype=i32)
    refused("rows", M.mxfp4_moe_plan, rows, t(8, dtype=i64), t(4, 3, dtype=i32))
    refused("group_list", M.mxfp4_moe_plan, rows, t(2, 8, dtype=i64), rows)
    refused("1024 experts", M.mxfp4_moe_plan, rows, t(1025, dtype=i64), rows)
    refused("workspace", M.mxfp4_moe_plan, t(10000, 2, dtype=i32), t(8, dtype=i64), t(10000, 2, dtype=i32),
            workspace=t(16, dtype=u8))
    refused("required", M.mxfp4_moe_dispatch, x, rows)
    refused("same number of rows", M.mxfp4_moe_dispatch, x, rows, y=t(8, 64, dtype=bf16), q=t(7, 64, dtype=u8))
    refused("q must be", M.mxfp4_moe_dispatch, x, rows, q=t(8, 63, dtype=u8), scales=t(8, 2, dtype=u8))
    refused("scales", M.mxfp4_moe_dispatch, x, rows, q=t(8, 64, dtype=u8), scales=t(8, 3, dtype=u8))
    refused("rows", M.mxfp4_moe_dispatch, x, t(5, 2, dtype=i32), y=t(8, 64, dtype=bf16))
    refused("fmt", M.mxfp4_moe_dispatch, x, rows, y=t(8, 64, dtype=bf16), fmt="e2m1")
    h = t(8, 64, dtype=bf16)
    refused("y must be", M.mxfp4_moe_combine, h, rows, t(4, 63, dtype=bf16))
    refused("weights", M.mxfp4_moe_combine, h, rows, x, weights=t(4, 3))
    refused("residual", M.mxfp4_moe_combine, h, rows, x, residual=t(3, 64, dtype=bf16))
    refused("y is required", M.mxfp4_moe_combine, h, rows, None)
    refused("required", M.mxfp4_moe_combine_bwd, x, h, rows)
    refused("needs h", M.mxfp4_moe_combine_bwd, x, None, rows, grad_weights=t(4, 2))
    refused("grad_h", M.mxfp4_moe_combine_bwd, x, h, rows, grad_h=t(7, 64, dtype=bf16))


def route(dtype=F32, score=0, renorm=1, experts=8, tokens=4, k=2, groups=1, topk=1, scale=1.0, reserved=0):
    return _Route(dtype, score, renorm, experts, tokens, k, groups, topk, scale, reserved)


def test_abi_route(lib):
    def call(d, l=A[0], b=None, w=A[1], i=A[2]):
        return lib.mxfp4_moe_route(ctypes.byref(d) if d else None, P(l), P(b), P(w), P(i), None)
    assert call(None) == EINVAL
    assert call(route(dtype=5)) == EUNSUP
    assert call(route(score=2)) == EINVAL
    assert call(route(renorm=2)) == EINVAL
    assert call(route(tokens=-1)) == EINVAL
    assert call(route(experts=0)) == EUNSUP
    assert call(route(experts=1025)) == EUNSUP
    assert call(route(k=0)) == EUNSUP
    assert call(route(k=9)) == EUNSUP                       # more than the experts
    assert call(route(experts=128, k=65)) == EUNSUP
    assert call(route(groups=3)) == EINVAL                  # does not divide 8
    assert call(route(groups=0)) == EINVAL
    assert call(route(experts=1024, groups=128)) == EINVAL
    assert call(route(groups=2, topk=3)) == EINVAL
    assert call(route(groups=2, topk=0)) == EINVAL
    assert call(route(groups=4, topk=1, k=3)) == EINVAL     # the kept groups hold 2 experts
    assert b"fewer" in lib.mxfp4_last_error()
    assert call(route(reserved=1)) == EINVAL
    assert call(route(tokens=1 << 61)) == EINVAL
    assert call(route(), l=None) == EINVAL
    assert call(route(), l=A[0] + 2) == EINVAL              # half an fp32 element
    assert call(route(), w=A[1] + 2) == EINVAL
    assert call(route(), i=A[0]) == EINVAL                  # ids over the logits
    assert call(route(tokens=0), l=None, w=None, i=None) == OK
    d = route()
    bwd = lambda g=A[0], l=A[1], i=A[2], o=A[3]: lib.mxfp4_moe_route_bwd(ctypes.byref(d), P(g), P(l), P(i), P(o), None)  # noqa: E731
    assert bwd(g=None) == EINVAL and bwd(l=None) == EINVAL and bwd(i=None) == EINVAL and bwd(o=None) == EINVAL
    assert bwd(o=A[1]) == EINVAL


def test_abi_plan(lib):
    def call(slots=10, experts=4, ids=A[0], g=A[1], r=A[2], ws=None, n=0):
        return lib.mxfp4_moe_plan(slots, experts, P(ids), P(g), P(r), P(ws), n, None)
    assert call(slots=-1) == EINVAL
    assert call(slots=1 << 31) == EUNSUP
    assert call(experts=0) == EUNSUP and call(experts=1025) == EUNSUP
    assert call(ids=None) == EINVAL and call(g=None) == EINVAL and call(r=None) == EINVAL
    assert call(g=A[1] + 4) == EINVAL and call(r=A[2] + 2) == EINVAL
    assert call(r=A[0]) == EINVAL
    need = lib.mxfp4_moe_plan_workspace(100000, 4)
    assert need > 0 and lib.mxfp4_moe_plan_workspace(10, 4) == 0
    assert lib.mxfp4_moe_plan_workspace(-1, 4) == -1 and lib.mxfp4_moe_plan_workspace(5, 2000) == -1
    assert call(slots=100000) == EINVAL
    assert call(slots=100000, ws=A[3], n=need - 1) == EINVAL
    assert call(slots=100000, ws=A[0], n=need) == EINVAL    # over ids


def desc(dtype=BF16, block=32, rows=4, cols=64):
    return M._Desc(dtype, block, 0, 0, rows, cols, 6.0, 0)


def test_abi_dispatch_and_combine(lib):
    def disp(d, fmt=0, x=A[0], r=A[1], k=2, n=8, y=None, q=A[2], s=A[3]):
        return lib.mxfp4_moe_dispatch(ctypes.byref(d) if d else None, fmt, P(x), P(r), k, n, P(y), P(q), P(s), None)
    assert disp(None) == EINVAL
    assert disp(desc(block=64)) == EUNSUP and disp(desc(dtype=3)) == EUNSUP
    assert disp(desc(), fmt=4) == EINVAL
    assert disp(desc(), k=0) == EUNSUP and disp(desc(), k=65) == EUNSUP
    assert disp(desc(), n=-1) == EINVAL and disp(desc(), n=1 << 31) == EUNSUP
    assert disp(desc(), q=None, s=None) == EINVAL
    assert disp(desc(), s=None) == EINVAL and disp(desc(), q=None, y=A[4]) == EINVAL
    assert disp(desc(), x=None) == EINVAL and disp(desc(), r=None) == EINVAL
    assert disp(desc(), x=A[0] + 1) == EINVAL and disp(desc(), y=A[4] + 1) == EINVAL
    assert disp(desc(), q=A[0]) == EINVAL
    assert disp(desc(rows=0), x=None, r=None) == OK and disp(desc(), n=0) == OK

    def comb(dtype=BF16, tokens=4, cols=64, k=2, n=8, h=A[0], r=A[1], w=A[2], res=None, y=A[3]):
        return lib.mxfp4_moe_combine(dtype, tokens, cols, k, n, P(h), P(r), P(w), P(res), P(y), None)
    assert comb(dtype=7) == EUNSUP
    assert comb(tokens=-1) == EINVAL and comb(cols=-1) == EINVAL and comb(k=70) == EUNSUP
    assert comb(tokens=1 << 60, cols=64) == EINVAL
    assert comb(h=None) == EINVAL and comb(r=None) == EINVAL and comb(y=None) == EINVAL
    assert comb(w=A[2] + 1) == EINVAL and comb(res=A[4] + 1) == EINVAL
    assert comb(y=A[0]) == EINVAL
    assert comb(tokens=0, h=None, r=None, y=None) == OK

    def bwd(gy=A[0], h=A[1], r=A[2], w=A[3], gh=A[4], gw=A[5], dtype=BF16, tokens=4, cols=64):
        return lib.mxfp4_moe_combine_bwd(dtype, tokens, cols, 2, 8, P(gy), P(h), P(r), P(w), P(gh), P(gw), None)
    assert bwd(gh=None, gw=None) == EINVAL
    assert bwd(gy=None) == EINVAL and bwd(h=None) == EINVAL and bwd(r=None) == EINVAL
    assert bwd(gh=A[0]) == EINVAL and bwd(gh=A[1]) == EINVAL and bwd(gw=A[3]) == EINVAL
    assert bwd(tokens=0) == OK and bwd(cols=0, gw=None) == OK
