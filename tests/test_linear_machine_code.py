"""The product library's gfx950 machine code (compiled here; no GPU needed): its
loads into LDS set m0 in inline assembly, which cannot tell the compiler so
(m0 is reserved and may not stand in a list of clobbers). That is sound while
the compiler itself keeps nothing there."""

from __future__ import annotations

import re

from hyper_connection_residual_mhc_amd import _build


def test_only_the_inline_assembly_uses_m0(tmp_path):
    asm = _build.device_asm(tmp_path / "linear.s", src=_build.LINEAR_SRC).read_text()
    inside, sets, loads, others = False, 0, 0, []
    for line in asm.splitlines():
        code = line.split(";", 1)[0]
        if ";;#ASMSTART" in line or ";;#ASMEND" in line:
            inside = ";;#ASMSTART" in line
        elif inside:
            sets += bool(re.match(r"\s*s_mov_b32 m0, ", code))
            loads += bool(re.search(r"\blds\s*$", code))
        elif re.search(r"\bm0\b", code) or re.search(r"\blds\s*$", code):
            others.append(line.strip())
    assert sets == loads > 0
    assert not others, others[:5]
