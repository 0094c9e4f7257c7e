"""Host-side check of the compiled gfx950 kernels (no GPU): the kernels of the
adapters and of the gradient norm keep everything in registers, but for the forms
of the adapters' second product that are named here."""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mxfp4_fake_quantization_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"
FILES = ("adapter_fwd_kernels", "adapter_bwd_kernels", "grad_norm_kernels")
# (fp32, fragments of the ranks) -> the most scratch accesses of a kernel: bf16 of rank 17 to 32 (three
# waves a SIMD leave 168 registers, two are spilled), fp32 of rank 65 to 128 (faster so than with one
# wave a SIMD).
SPILLING = {(False, 1): 4, (True, 8): 156}


def compile_asm(name, tmp):
    out = os.path.join(tmp, name + ".s")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                    "-packed-fp32-ops", "--cuda-device-only", "-S", os.path.join(CSRC, name + ".hip"),
                    "-I", CSRC, "-o", out], check=True, capture_output=True)
    with open(out) as f:
        return f.read()


def test_every_kernel_is_free_of_scratch_or_named(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    with cf.ThreadPoolExecutor(max_workers=len(FILES)) as ex:
        texts = list(ex.map(lambda n: compile_asm(n, str(tmp_path)), FILES))
    counts, cur = {}, None
    for line in "\n".join(texts).split("\n"):
        m = re.match(r"^(_Z\S+):", line)
        if m:
            cur = m.group(1)
            counts.setdefault(cur, 0)
        elif cur and "scratch_" in line:
            counts[cur] += 1
    assert sum("adapter_expand_kernel" in k for k in counts) > 30 and any("grad_clip_kernel" in k for k in counts)
    for k, n in counts.items():
        m = re.search(r"adapter_expand_kernelILi([01])ELi([0-9]+)E", k)
        most = SPILLING.get((m.group(1) == "0", int(m.group(2))), 0) if m else 0
        assert n <= most, (k, n)
