"""Register and scratch budget of the many-tensor kernels (CPU: hipcc
cross-compiles for gfx950, with the library's own flags): no spilled registers,
no scratch memory, none of the packed fp32 instructions that the build turns
off, and the update's code small enough that a launch which mixes types does
not wait for instructions."""

import os
import re
import shutil
import subprocess

import pytest

from matrix_aware_optimizer_step_amd import build as B


def assembly(tmp_path, source):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    out = tmp_path / "out.s"
    cmd = [hipcc, *[f for f in B.COMMON if f != "-fPIC"], *B.EXTRA.get(source, []), "-x", "hip", "--cuda-device-only",
           "-S", os.path.join(B.CSRC, source), "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
    assert res.returncode == 0, res.stderr[-3000:]
    return out.read_text()


@pytest.mark.parametrize("source,kernels,code", [("adamw_multi.hip", 1, 64 << 10), ("grad_norm.hip", 3, 16 << 10)])
def test_kernels_use_no_scratch(tmp_path, source, kernels, code):
    text = assembly(tmp_path, source)
    found = 0
    for block in re.split(r"\n\s+- \.", text):
        vals = {k: int(v) for k, v in re.findall(r"\.(private_segment_fixed_size|vgpr_spill_count|sgpr_spill_count|"
                                                   r"vgpr_count):\s+(\d+)", block)}
        if "vgpr_count" not in vals:
            continue
        found += 1
        assert vals["private_segment_fixed_size"] == vals["vgpr_spill_count"] == vals["sgpr_spill_count"] == 0, vals
        assert vals["vgpr_count"] <= 128, vals
    assert found == kernels
    assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", text)
    assert all(int(n) <= code for n in re.findall(r"codeLenInByte = (\d+)", text))
