"""The largest calls of the adapters, on the CPU: a launch of the second product has below 2^32
threads, 256 for a tile of 32 rows by 256 columns at least."""
import os

import pytest

import mxfp4_fake_quantization_amd as M
from mxfp4_fake_quantization_amd import adapter_ops


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("side", ["n_in", "n_out"])
def test_the_tiles_bound(dtype, side):
    if not os.path.exists(M.library_path()):
        pytest.fail("libmxfp4.so is not built (python -m mxfp4_fake_quantization_amd.build)")
    lib = adapter_ops._lib()

    def workspace(tokens, features):
        n = {"n_in": 32, "n_out": 32, side: features}
        return lib.mxfp4_adapter_workspace(adapter_ops._ADAPTER.pack(dtype, 8, 2, 0, tokens, n["n_in"], n["n_out"]))

    for rows in (20, 25):                                   # 2^rows tokens, 2^(rows - 5) tiles of them
        most = ((1 << 24) - 1 >> rows - 5) * 256            # columns
        assert workspace(1 << rows, most) > 0
        assert workspace(1 << rows, most + 1) == -1
        assert workspace((1 << rows) - 1, most) > 0
