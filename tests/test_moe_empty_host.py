"""Calls without any work to do, on the CPU: an empty torch tensor has a NULL
address, so the C ABI has to accept NULL wherever an array has no elements, and
still refuse it where there are some."""
import ctypes
import os

import pytest

import mxfp4_fake_quantization_amd as M

OK, EINVAL, EUNSUP = 0, 1, 2
BF16 = 1
P = ctypes.c_void_p
A = [0x10000 * (i + 1) for i in range(12)]  # aligned addresses that are never read


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.library_path()):
        pytest.fail("libmxfp4.so is not built (python -m mxfp4_fake_quantization_amd.build)")
    from mxfp4_fake_quantization_amd import moe_ops
    return moe_ops._lib()


def desc(rows, cols, block=32):
    return M._Desc(BF16, block, 0, 0, rows, cols, 6.0, 0)


@pytest.mark.parametrize("rows,cols,out_rows", [(0, 64, 0), (4, 0, 8), (4, 64, 0), (0, 0, 0)])
def test_dispatch_of_nothing(lib, rows, cols, out_rows):
    d = desc(rows, cols)
    assert lib.mxfp4_moe_dispatch(ctypes.byref(d), 0, None, None, 2, out_rows, None, None, None, None) == OK
    # the other arguments are still checked
    assert lib.mxfp4_moe_dispatch(ctypes.byref(d), 0, None, None, 0, out_rows, None, None, None, None) == EUNSUP
    assert lib.mxfp4_moe_dispatch(ctypes.byref(d), 4, None, None, 2, out_rows, None, P(A[2]), P(A[3]), None) == EINVAL


def test_dispatch_of_something_needs_its_outputs(lib):
    d = desc(4, 64)
    for q, s in ((None, None), (A[2], None), (None, A[3])):
        assert lib.mxfp4_moe_dispatch(ctypes.byref(d), 0, P(A[0]), P(A[1]), 2, 8, None, P(q), P(s), None) == EINVAL


@pytest.mark.parametrize("tokens,cols,in_rows", [(0, 64, 0), (0, 64, 8), (4, 64, 0), (4, 0, 8)])
def test_combine_backward_of_nothing(lib, tokens, cols, in_rows):
    f = lib.mxfp4_moe_combine_bwd
    assert f(BF16, tokens, cols, 2, in_rows, None, None, None, None, None, None, None) == OK
    assert f(BF16, tokens, cols, 70, in_rows, None, None, None, None, None, None, None) == EUNSUP


def test_combine_backward_of_something_needs_an_output(lib):
    f = lib.mxfp4_moe_combine_bwd
    assert f(BF16, 4, 64, 2, 8, P(A[0]), P(A[1]), P(A[2]), None, None, None, None) == EINVAL


# ---- the older calls that the layer makes around them ---------------------------

def test_mxfp8_of_nothing(lib):
    for rows, cols in ((0, 64), (4, 0)):
        d = desc(rows, cols)
        assert lib.mxfp8_quant(ctypes.byref(d), 0, None, None, None, None) == OK
        assert lib.mxfp8_quant(ctypes.byref(d), 5, None, None, None, None) == EINVAL
        d = desc(rows, cols)
        assert lib.mxfp8_quant_kmajor(ctypes.byref(d), 0, None, P(A[0]), 3, 1, 4, None, None, None) == OK
        assert lib.mxfp8_quant_kmajor(ctypes.byref(d), 0, None, P(A[0]), 0, 1, 4, None, None, None) == EINVAL
    d = desc(4, 64)
    assert lib.mxfp8_quant(ctypes.byref(d), 0, None, None, None, None) == EINVAL
    assert lib.mxfp8_quant_kmajor(ctypes.byref(d), 0, None, None, 0, 1, 1, None, None, None) == EINVAL


def test_product_of_no_rows(lib):
    """No rows of A (an empty batch): nothing to do, whatever the operands' addresses."""
    def mm(group_type, m, n, k, kb, data, ld, gl):
        a = M._MxOperand(data, data and data + 4096, 0, 32, ld, 4, 0, 0)
        b = M._MxOperand(A[2], A[3], 4, 32, 64, 4, 0, 0)
        return lib.mxfp4_grouped_matmul(group_type, m, n, k, ctypes.byref(a), ctypes.byref(b), P(gl), 3, 1, kb, 0, None,
                                        n, None)
    assert mm(M.GROUP_ROWS, 0, 48, 128, 0, None, 128, A[5]) == OK
    assert mm(M.GROUP_ROWS, 5, 48, 128, 0, None, 128, A[5]) == EINVAL   # a is NULL
    assert mm(M.GROUP_ROWS, 5, 0, 128, 0, None, 128, A[5]) == OK
    assert mm(M.GROUP_K, 48, 48, 0, 0, None, 0, A[5]) == EINVAL          # no tokens: c, which gets zeros, is NULL
    assert b"c is NULL" in lib.mxfp4_last_error()
    assert mm(M.GROUP_K, 48, 48, 0, 1, None, 32, A[5]) == EINVAL
    assert b"a is NULL" in lib.mxfp4_last_error()
