"""Register and scratch budget of the expert kernels (CPU: hipcc cross-compiles
for gfx950 with the library's own flags): no spilled vector registers, no
scratch memory (but for some scalar masks where more than 256 experts are chosen
by score), none of the packed fp32 instructions that the build turns off, and
the products on the matrix instructions they are meant to use."""

import re

import pytest

from tests.test_multi_resources import assembly


@pytest.mark.parametrize("source,kernels,most,scratch", [
    ("block_codes.hip", 20, 128, 0), ("route.hip", 23, 256, 128), ("expert_sum.hip", 4, 64, 0),
    ("block_gemm.hip", 30, 256, 0)])
def test_kernels_use_no_scratch(tmp_path, source, kernels, most, scratch):
    text = assembly(tmp_path, source)
    found = 0
    for block in re.split(r"\n\s+- \.", text):
        vals = {k: int(v) for k, v in re.findall(r"\.(private_segment_fixed_size|vgpr_spill_count|vgpr_count):\s+(\d+)",
                                                   block)}
        if "vgpr_count" not in vals:
            continue
        found += 1
        assert vals["vgpr_spill_count"] == 0 and vals["private_segment_fixed_size"] <= scratch, vals
        assert vals["vgpr_count"] <= most, vals
    assert found == kernels
    assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", text)
    if source == "block_gemm.hip":
        assert "v_mfma_f32_16x16x128_f8f6f4" in text and "v_mfma_f32_16x16x32_bf16" in text
