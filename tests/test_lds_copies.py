"""Copies from global memory straight into LDS read their LDS address from m0
(CPU: hipcc cross-compiles for gfx950 with the library's own flags).  The
instruction set asks for one wait state between a write of m0 and such a copy:
an instruction of any kind in between."""

import re

import pytest

from tests.test_multi_resources import assembly


def unsafe(text):
    """(copies, those whose preceding instruction writes m0)"""
    copies, bad, before = 0, [], ""
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        if not line or line.startswith(".") or line.endswith(":"):
            continue
        if re.match(r"(global|buffer|scratch)_load_lds_|buffer_load_\w+ .*\blds\b", line):
            copies += 1
            if re.match(r"\w+ m0\b", before):
                bad.append((before, line))
        before = line
    return copies, bad


@pytest.mark.parametrize("source", ["ns_gemm.hip", "block_gemm.hip"])
def test_a_wait_state_lies_between_m0_and_the_copy(tmp_path, source):
    copies, bad = unsafe(assembly(tmp_path, source))
    assert copies > 20 and not bad, (copies, len(bad), bad[:3])


def test_the_check_sees_a_missing_wait_state():
    ok = "s_mov_b32 m0, s4\n;;#ASMSTART\ns_nop 0\nglobal_load_lds_dwordx4 v0, s[0:1]\n;;#ASMEND\n"
    assert unsafe(ok) == (1, [])
    assert len(unsafe(ok.replace("s_nop 0\n", ""))[1]) == 1
