"""The built libraries' own gfx950 code, as it is in the .so files of this tree.

Every library is held to the one full list of scalar memory writes that
test_build_guards.py keeps, whichever shorter ones other guards look for.

The product libraries' loads into LDS are inline assembly, so the compiler does not
keep the distance that a load needs from a vector instruction that writes one of its
scalar registers: five wait states (an instruction is one, s_nop N is N + 1). Such an
instruction may be the compiler's own readlane of a register that it had spilled, and
a load that comes too soon reads what was there before: another address.
"""

from __future__ import annotations

import re
import shutil
import subprocess
from pathlib import Path

import pytest

from hyper_connection_residual_mhc_amd import _build

guards = pytest.importorskip("test_build_guards")

PRODUCTS = {"linear": _build.LINEAR_LIB_PATH, "gated": _build.GATED_LIB_PATH, "cross_entropy": _build.CROSS_ENTROPY_LIB_PATH}
STATES = 5


@pytest.fixture(scope="module")
def objdump() -> str:
    beside = Path(_build.hipcc()).resolve().parent.parent / "llvm" / "bin" / "llvm-objdump"
    path = str(beside) if beside.exists() else shutil.which("llvm-objdump")
    if path is None:
        pytest.skip("no llvm-objdump beside hipcc")
    return path


def listing(objdump: str, lib: Path, to: Path) -> str:
    """The library's device code, an instruction to a line behind white space, with labels where jumps go."""
    shutil.copy(lib, to)
    subprocess.run([objdump, "--offloading", lib.name], cwd=to, check=True, capture_output=True)
    code, = to.glob("*gfx950*")
    return subprocess.run([objdump, "-d", "--no-show-raw-insn", "--symbolize-operands", str(code)], check=True,
                          capture_output=True, text=True).stdout


@pytest.mark.parametrize("lib", [lib for lib, _ in _build.LIBRARIES.values()], ids=lambda p: p.stem)
def test_no_scalar_memory_writes(built_library, objdump, lib, tmp_path):
    asm = listing(objdump, lib, tmp_path)
    assert "\n\ts_endpgm" in asm and asm.count("\n\ts_load_dword") > 1
    guards.test_no_scalar_memory_writes(asm)


def scalars(text: str) -> set[int]:
    """Numbers of the scalar registers that an operand names."""
    got = set()
    for m in re.finditer(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        got |= set(range(int(m[1]), int(m[2]) + 1)) if m[1] else {int(m[3])}
    return got


def kernels(asm: str) -> dict[str, dict[str, tuple[list[str], list[str]]]]:
    """{kernel: {block: (its instructions, the blocks that may follow)}}; a kernel's first block is ""."""
    found: dict = {}
    blocks = name = None
    for line in asm.splitlines():
        label = re.match(r"[0-9a-f]+ <([^>]+)>:", line)
        code = line.split("//", 1)[0].strip()
        if label and re.fullmatch(r"L\d+", label[1]):
            if name is not None:
                blocks[name][1].append(label[1])
            name = label[1]
            blocks[name] = ([], [])
        elif label:
            blocks = found[label[1]] = {"": ([], [])}
            name = ""
        elif blocks is not None and line.startswith("\t") and code:
            if name is None:                               # behind a jump that is always taken: no one comes here
                name = f"dead {len(blocks)}"
                blocks[name] = ([], [])
            blocks[name][0].append(code)
            jump = re.match(r"s_(c?)branch\S*\s+(\S+)", code)
            if jump:
                blocks[name][1].append(jump[2])
                after = f"after {len(blocks)}"
                if jump[1]:
                    blocks[name][1].append(after)
                    blocks[after] = ([], [])
                name = after if jump[1] else None
            elif code.startswith("s_endpgm"):
                name = None
    return found


def early_loads(blocks) -> list[str]:
    """Loads into LDS that come too soon behind a vector instruction's write to one of their scalar registers, on some
    way through the kernel."""
    bad = set()

    def through(code, written):
        for c in code:
            if c.startswith("buffer_load") and c.endswith(" lds") and set(written) & scalars(c):
                bad.add(c)
            passed = int(c.split()[1], 0) + 1 if c.startswith("s_nop") else 1
            written = {r: n - passed for r, n in written.items() if n > passed}
            operands = c.split(" ", 1)[1].split(",") if " " in c else []
            if c.startswith("v_") and operands:
                # the result, and a carry or a flag beside it
                for r in scalars(operands[0]) | (scalars(operands[1]) if re.match(r"v_\w+_co_|v_div_scale|v_mad_[ui]64", c) else set()):
                    written[r] = STATES
            elif c.startswith("s_") and operands:
                for r in scalars(operands[0]):
                    written.pop(r, None)
        return written

    states: dict = {name: None for name in blocks}
    states[""] = {}
    todo = [""]
    while todo:
        name = todo.pop()
        code, follow = blocks[name]
        written = through(code, dict(states[name]))
        for f in follow:
            old = states[f]
            merged = written if old is None else {r: max(written.get(r, 0), old.get(r, 0)) for r in set(written) | set(old)}
            if merged != old:
                states[f] = merged
                todo.append(f)
    return sorted(bad)


@pytest.mark.parametrize("name", sorted(PRODUCTS))
def test_loads_into_lds_read_what_was_written(built_library, objdump, name, tmp_path):
    loads = 0
    for kernel, blocks in kernels(listing(objdump, PRODUCTS[name], tmp_path)).items():
        assert not early_loads(blocks), kernel
        loads += sum(c.endswith(" lds") for code, _ in blocks.values() for c in code)
    assert loads > 100


def test_the_scan_sees_the_pattern():
    def scan(*lines):
        return early_loads(kernels("0000 <k>:\n" + "\n".join(lines) + "\n\ts_endpgm\n")["k"])

    write, load = "\tv_readlane_b32 s20, v9, 1", "\tbuffer_load_dwordx4 v1, s[20:23], s0 offen lds"
    other = "\tv_add_u32_e32 v2, v3, v4"
    assert scan(write, load) and scan(write, *[other] * 4, load) and scan(write, "\ts_nop 3", load)
    assert not scan(write, *[other] * 5, load) and not scan(write, "\ts_nop 4", load)
    assert scan("\tv_readfirstlane_b32 s0, v9", load) and not scan("\tv_readfirstlane_b32 s1, v9", load)
    assert not scan(write, "\ts_mov_b32 s20, s4", load)
    # over jumps: into a block, and round a loop
    assert scan(write, "\ts_cbranch_scc1 L0", *[other] * 6, "0010 <L0>:", load)
    assert scan("0010 <L0>:", load, *[other] * 6, write, "\ts_cbranch_scc1 L0")
    assert not scan("\ts_branch L0", write, "0010 <L0>:", load)
