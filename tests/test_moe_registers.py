"""Host-side check of the compiled gfx950 kernels (no GPU): the kernels of the
mixture-of-experts operators keep everything in registers.  Scratch would add
HBM traffic that their bytes do not count, in the main loop of the product at
every step."""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mxfp4_fake_quantization_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"
# source -> kernels that must not touch scratch at all.  The tiled product:
# E2M1 weights, and fp8 ones with dword-aligned scale rows (S4); the few-rows
# form: 16 rows a workgroup.
FILES = {
    "moe_route_kernels": r"route_",
    "moe_rows_kernels": r"(plan|dispatch|combine)_",
    "act_bwd_kernels": r"(act_bwd|bias_sum)_kernel",
    "mxgemm_act_kernels": r"mxgemm_act_kernelILi[01]ELi(4E|0ELb1)",
    "mxgemm_gated_kernels": r"mxgemm_act_kernelILi[01]ELi(4E|0ELb1)",
    "mxgemm_rows_kernels": r"mxgemm_rows_(split_)?kernelILi[01]ELi4ELb1ELi1E",
}


def compile_asm(name, tmp):
    out = os.path.join(tmp, name + ".s")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                    "-packed-fp32-ops", "--cuda-device-only", "-S", os.path.join(CSRC, name + ".hip"),
                    "-I", CSRC, "-o", out], check=True, capture_output=True)
    with open(out) as f:
        return f.read()


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    tmp = str(tmp_path_factory.mktemp("asm"))
    with cf.ThreadPoolExecutor(max_workers=len(FILES)) as ex:
        return dict(zip(FILES, ex.map(lambda n: compile_asm(n, tmp), FILES)))


@pytest.mark.parametrize("name", sorted(FILES))
def test_no_scratch(asm, name):
    counts, cur = {}, None
    for line in asm[name].split("\n"):
        m = re.match(r"^(_Z\S+):", line)
        if m:
            cur = m.group(1)
            counts[cur] = 0
        elif cur and "scratch_" in line:
            counts[cur] += 1
    mine = {k: v for k, v in counts.items() if re.search(FILES[name], k)}
    assert mine, f"no kernels matched in {name}"
    assert not any(mine.values()), {k: v for k, v in mine.items() if v}


# The few-rows forms whose two register sets do not fit the registers that their
# waves a SIMD leave: (K shared by the waves, weights, 16-row tiles) -> the most
# scratch accesses of a kernel, nearly all in its main loop.  All others have none.
SPILLING = {("whole", "e4m3", 1): 31, ("split", "e4m3", 1): 38, ("split", "e4m3", 4): 85, ("split", "e2m1", 4): 6}


def test_every_kernel_is_free_of_scratch_or_named(asm):
    counts, cur = {}, None
    for name, text in asm.items():
        for line in text.split("\n"):
            m = re.match(r"^(_Z\S+):", line)
            if m:
                cur = m.group(1)
                counts[cur] = 0
            elif cur and "scratch_" in line:
                counts[cur] += 1
    few = {}
    for k, n in counts.items():
        m = re.search(r"mxgemm_rows_(split_)?kernelILi[01]ELi([04])ELb[01]ELi([124])E", k)
        if m:
            form = ("split" if m.group(1) else "whole", "e4m3" if m.group(2) == "0" else "e2m1", int(m.group(3)))
            few[form] = max(few.get(form, 0), n)
        else:
            assert n == 0, (k, n)
    assert len(few) == 12, few                                   # every form was seen
    for form, n in few.items():
        assert n <= SPILLING.get(form, 0), (form, n)
