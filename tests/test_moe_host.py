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


# ---- the product with its epilogue, and its backward ------------------------------

def test_binding_product():
    a, asc = t(64, 128, dtype=u8), t(64, 4, dtype=u8)
    b, bsc = t(2, 48, 64, dtype=u8), t(2, 48, 4, dtype=u8)            # 2 experts, 48 rows, K = 128 (fp4)
    c, gl = t(64, 48, dtype=bf16), [30, 34]
    f = M.mxfp4_grouped_matmul_act
    refused("act", f, a, asc, b, bsc, c, group_list=gl, act="tanh")
    refused("c must be", f, a, asc, b, bsc, t(64, 24, dtype=bf16), group_list=gl)
    refused("c must be", f, a, asc, b, bsc, c, group_list=gl, act="swiglu")        # gated: half as many columns
    refused("bfloat16 or float32", f, a, asc, b, bsc, t(64, 48, dtype=torch.float16), group_list=gl)
    refused("even number", f, a, asc, t(2, 47, 64, dtype=u8), t(2, 47, 4, dtype=u8), c, group_list=gl, act="geglu")
    refused("bias", f, a, asc, b, bsc, c, group_list=gl, bias=t(47))
    refused("bias", f, a, asc, b, bsc, c, group_list=gl, bias=t(3, 48))
    refused("residual", f, a, asc, b, bsc, c, group_list=gl, residual=t(64, 47, dtype=bf16))
    refused("residual", f, a, asc, b, bsc, c, group_list=gl, residual=t(64, 48))   # another type
    refused("z must be", f, a, asc, b, bsc, t(64, 24, dtype=bf16), group_list=gl, act="swiglu", z=t(64, 24, dtype=bf16))
    refused("one matrix per group", f, a, asc, b, bsc, c, group_list=[10, 20, 34])
    refused("a_scales", f, a, t(63, 4, dtype=u8), b, bsc, c, group_list=gl)
    refused("b_scales", f, a, asc, b, t(2, 47, 4, dtype=u8), c, group_list=gl)
    refused("same rank", f, a, asc, b, t(48, 4, dtype=u8), c)
    refused("fmt", f, a, asc, b, bsc, c, a_fmt="e3m2")
    z, dc = t(9, 32), t(9, 16)
    g = M.mxfp4_act_bwd
    refused("z must be", g, dc, t(9, 16), z, act="swiglu")
    refused("grad_z", g, dc, z, t(9, 16), act="swiglu")
    refused("grad_bias", g, dc, z, z, act="swiglu", grad_bias=t(2, 32))
    refused("workspace", g, dc, z, z, act="swiglu", grad_bias=t(1, 32), workspace=t(8, dtype=u8))
    refused("act", g, dc, z, z, act="none2")


def operand(data, scales, fmt, block=32, ld=128, lds=4, gs=0, gss=0):
    return M._MxOperand(data, scales, fmt, block, ld, lds, gs, gss)


def test_abi_product(lib):
    from mxfp4_fake_quantization_amd.moe_ops import _Epilogue

    def ep(act=0, reserved=0, bias=None, bs=0, res=None, ldr=48, z=None, ldz=48):
        return _Epilogue(act, reserved, bias, bs, res, ldr, z, ldz)

    def call(m=64, n=48, k=128, a=None, b=None, gl=None, ng=1, lt=1, e=None, out=0, c=A[4], ldc=48):
        a = a or operand(A[0], A[1], 0)
        b = b or operand(A[2], A[3], 4, ld=64)
        e = ep() if e is None else e
        return lib.mxfp4_grouped_matmul_act(m, n, k, ctypes.byref(a), ctypes.byref(b), P(gl), ng, lt,
                                            ctypes.byref(e) if e else None, out, P(c), ldc, None)
    assert call(m=-1) == EINVAL and call(k=40) == EINVAL and call(k=0) == EUNSUP
    assert call(e=False) == EINVAL
    for act in (-1, 4, 5, 8):
        assert call(e=ep(act)) == EUNSUP
    assert call(e=ep(reserved=1)) == EINVAL
    assert call(out=2) == EUNSUP
    assert call(gl=A[5], ng=0) == EINVAL and call(gl=A[5], lt=2) == EINVAL and call(gl=A[5] + 4) == EINVAL
    assert call(a=operand(A[0], A[1], 4)) == EUNSUP                         # A is fp8
    assert call(b=operand(A[2], A[3], 1)) == EUNSUP                         # B is E2M1 or E4M3
    assert call(a=operand(A[0], A[1], 0, block=64)) == EUNSUP
    assert call(a=operand(A[0], A[1], 0, ld=112)) == EINVAL and call(a=operand(A[0], A[1], 0, lds=3)) == EINVAL
    assert call(b=operand(A[2] + 8, A[3], 4, ld=64)) == EINVAL
    assert call(c=None) == EINVAL and call(c=A[4] + 1) == EINVAL and call(ldc=47) == EINVAL
    assert call(e=ep(bias=A[6] + 2)) == EINVAL and call(e=ep(bias=A[6], bs=-1)) == EINVAL
    assert call(e=ep(res=A[6], ldr=47)) == EINVAL and call(e=ep(res=A[4], ldr=56)) == EINVAL
    assert call(e=ep(z=A[6], ldz=47)) == EINVAL and call(e=ep(6, z=A[6], ldz=95)) == EINVAL
    assert call(e=ep(z=A[4])) == EINVAL and call(c=A[0]) == EINVAL          # outputs over inputs
    assert call(n=1 << 20, ldc=1 << 20, e=ep(6), b=operand(A[2], A[3], 4, ld=1 << 13)) == EUNSUP   # 2^33 bytes of gate
    assert call(m=0) == OK and call(n=0) == OK


def test_abi_act_bwd(lib):
    def call(dt=F32, act=2, rows=9, cols=16, dc=A[0], z=A[1], dz=A[2], db=None, gl=None, ng=0, lt=1, ws=None, n=0):
        return lib.mxfp4_act_bwd(dt, act, rows, cols, P(dc), P(z), P(dz), P(db), P(gl), ng, lt, P(ws), n, None)
    assert call(dt=4) == EUNSUP and call(act=5) == EUNSUP and call(rows=-1) == EINVAL
    assert call(rows=1 << 40, cols=1 << 40) == EINVAL
    assert call(dc=None) == EINVAL and call(z=None) == EINVAL and call(dz=None) == EINVAL
    assert call(dz=A[2] + 2) == EINVAL
    assert call(gl=A[3], ng=0) == EINVAL and call(gl=A[3], ng=2, lt=3) == EINVAL
    need = lib.mxfp4_act_bwd_workspace(2, 9, 16, 0)
    assert need > 0 and lib.mxfp4_act_bwd_workspace(5, 9, 16, 0) == -1 and lib.mxfp4_act_bwd_workspace(2, -1, 16, 0) == -1
    assert call(db=A[4]) == EINVAL and call(db=A[4], ws=A[5], n=need - 1) == EINVAL
    assert call(db=A[0], ws=A[5], n=need) == EINVAL                          # the sums over grad_c
    assert call(act=6, dz=A[0]) == EINVAL and call(act=6, dz=A[1]) == EINVAL  # gated: not in place
    assert call(rows=0, dc=None, z=None, dz=None) == OK and call(cols=0, dc=None) == OK


def test_layer_refusals():
    from mxfp4_fake_quantization_amd import moe
    with pytest.raises(ValueError, match="act"):
        moe.MoESpec(act="tanh")
    x, l, w1, w2 = t(4, 64, dtype=bf16), t(4, 3), t(3, 64, 64, dtype=bf16), t(3, 64, 32, dtype=bf16)
    s = moe.MoESpec()
    refused("bfloat16", moe._check_shapes, t(4, 64), l, w1, w2, s)
    refused("multiples of 32", moe._check_shapes, x, l, t(3, 62, 64, dtype=bf16), w2, s)
    refused("w2 must be", moe._check_shapes, x, l, w1, t(3, 64, 64, dtype=bf16), s)
    refused("logits", moe._check_shapes, x, t(4, 2), w1, w2, s)
    moe._check_shapes(x, l, w1, w2, s)
