"""Checks of the gated and cross entropy libraries' own gfx950 machine code and
exported names, and of what the product libraries' inline assembly relies on
(compiled here; no GPU needed): no packed fp32 arithmetic, no scalar memory
writes, fp32 denormals kept, no spills to scratch, no store of more than 8 bytes
followed at once by an overwrite of its data, m0 left to the loads into LDS, the
waits that a matrix instruction in inline assembly needs, a fast-math build
refused, and headers, bindings and exports that agree."""

from __future__ import annotations

import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from hyper_connection_residual_mhc_amd import _build, _lib
from test_build_guards import (STORE_WIDE, instructions, kernel_blocks, store_data_regs,
                               written_vgprs)

LIBRARIES = {
    "gated": (_build.GATED_SRC, _build.GATED_HEADER, _build.GATED_LIB_PATH, _lib.GATED_SIGNATURES, "mhc_gated_"),
    "cross_entropy": (_build.CROSS_ENTROPY_SRC, _build.CROSS_ENTROPY_HEADER, _build.CROSS_ENTROPY_LIB_PATH,
                      _lib.CROSS_ENTROPY_SIGNATURES, "mhc_cross_entropy_"),
}


SOURCES = {"linear": _build.LINEAR_SRC, **{name: entry[0] for name, entry in LIBRARIES.items()}}


@pytest.fixture(scope="module")
def all_asm(tmp_path_factory) -> dict[str, str]:
    to = tmp_path_factory.mktemp("asm")
    with ThreadPoolExecutor(len(SOURCES)) as pool:  # each is a compiler's minute
        made = pool.map(lambda name: _build.device_asm(to / f"{name}.s", src=SOURCES[name]).read_text(), SOURCES)
        return dict(zip(SOURCES, made))


@pytest.fixture(params=sorted(SOURCES))
def asm(request, all_asm) -> str:
    return all_asm[request.param]


def test_machine_code(asm):
    assert not re.search(r"^\s*v_pk_(add|mul|fma)_f32", asm, flags=re.M)
    assert not re.search(r"^\s*(s_store|s_buffer_store|s_scratch_store|s_atomic|s_buffer_atomic|s_dcache_wb)", asm, flags=re.M)
    modes = re.findall(r"\.amdhsa_float_denorm_mode_32\s+(\d+)", asm)
    assert modes and set(modes) == {"3"}
    spills = re.findall(r"\.vgpr_spill_count:\s+(\d+)", asm)
    assert spills and set(spills) == {"0"}
    assert "scratch_store" not in asm and "scratch_load" not in asm


def test_no_immediate_overwrite_of_wide_store_data(asm):
    checked = 0
    for name, body in kernel_blocks(asm).items():
        ins = instructions(body)
        for a, b in zip(ins, ins[1:]):
            if STORE_WIDE.match(a):
                checked += 1
                assert not store_data_regs(a) & written_vgprs(b), f"{name}: '{a.strip()}' then '{b.strip()}'"
    assert checked > 0


def lines_of(body: str):
    """(instruction, whether it is inline assembly's) of a kernel."""
    return [line for code, _ in blocks_of(body).values() for line in code]


def test_only_the_inline_assembly_uses_m0(asm):
    """Every load into LDS has its place set before it, with something between, and nothing else touches m0."""
    loads = 0
    for name, body in kernel_blocks(asm).items():
        since = None
        for code, inside in lines_of(body):
            uses = bool(re.search(r"\bm0\b", code)) or code.endswith(" lds")
            assert inside or not uses, f"{name}: {code}"
            if re.match(r"s_mov_b32 m0, ", code):
                assert since is None, f"{name}: a place is set twice"
                since = 0
            elif code.endswith(" lds"):
                assert since is not None and since >= 1, f"{name}: {code}"
                since, loads = None, loads + 1
            elif since is not None:
                since += 1
    assert loads > 0


def registers(text: str, file: str) -> set[int]:
    """Numbers of the `file` registers (v or a) that an operand names."""
    got = set()
    for m in re.finditer(rf"\b{file}\[(\d+):(\d+)\]|\b{file}(\d+)\b", text):
        got |= set(range(int(m[1]), int(m[2]) + 1)) if m[1] else {int(m[3])}
    return got


WAIT = 32      # cycles from a matrix instruction in inline assembly to another access to its result
DISTANCE = 3   # instructions from a vector instruction to a matrix instruction that reads what it wrote


def blocks_of(body: str):
    """The kernel's basic blocks: {name: ([(instruction, in inline assembly)], [names of those that follow])}."""
    blocks, name, inside, count = {}, "", False, 0
    blocks[name] = ([], [])
    for line in body.splitlines():
        if ";;#ASMSTART" in line or ";;#ASMEND" in line:
            inside = ";;#ASMSTART" in line
            continue
        code = line.split(";", 1)[0].strip()
        label = re.match(r"(\.L\w+):", code)
        if label:
            blocks[name][1].append(label[1])
            name = label[1]
            blocks[name] = ([], [])
        elif code and not code.startswith(".") and not code.endswith(":"):
            blocks[name][0].append((code, inside))
            jump = re.match(r"s_(c?)branch\S*\s+(\S+)", code)
            if jump or code.startswith("s_endpgm"):
                if jump:
                    blocks[name][1].append(jump[2])
                count += 1
                after = f"after jump {count}"
                if jump and jump[1]:
                    blocks[name][1].append(after)
                name = after
                blocks[name] = ([], [])
    return blocks


def mfma_hazards(body: str) -> tuple[int, list[str]]:
    """How many matrix instructions are inline assembly's, and what reaches one of them, or its result, too soon on
    some way through the kernel: the compiler does not see them, so it keeps none of the distances that it would keep
    from its own. A vector instruction that writes an operand stands DISTANCE instructions ahead; an instruction that
    reads a result or writes it otherwise stands WAIT cycles behind, an instruction other than s_nop counted as one."""
    blocks = blocks_of(body)
    ours = {c for code, _ in blocks.values() for c, inside in code if inside and c.startswith("v_mfma")}
    parts = {c: [o.strip() for o in c.split(" ", 1)[1].split(", ")] for c in ours}
    results = set().union(set(), *(registers(p[0], "a") for p in parts.values()))
    reads = {c: {(f, r) for f in "va" for r in registers(" ".join(p[1:]), f)} for c, p in parts.items()}
    bad = set()

    def through(code, left, written):
        """State behind a block: cycles that a result still takes, and {register: instructions that it still takes}."""
        for c, inside in code:
            if inside and c.startswith("v_mfma"):
                if reads[c] & set(written):
                    bad.add(f"an operand of {c} is written just before it")
                left = WAIT
            elif left and registers(c, "a") & results:
                bad.add(f"{c} with {left} cycles to go")
            passed = int(c.split()[1]) + 1 if c.startswith("s_nop") else 1
            left = max(0, left - passed)
            written = {r: n - passed for r, n in written.items() if n > passed}
            if c.startswith("v_") and not (inside and c.startswith("v_mfma")):
                to = c.split(" ", 1)[1].split(",")[0] if " " in c else ""
                written |= {(f, r): DISTANCE for f in "va" for r in registers(to, f)}
        return left, written

    states = {name: None for name in blocks}
    states[""] = (0, {})
    todo = [""]
    while todo:
        name = todo.pop()
        code, follow = blocks[name]
        left, written = through(code, *states[name])
        for f in follow:
            old = states[f]
            merged = (left, written) if old is None else (
                max(left, old[0]), {r: max(written.get(r, 0), old[1].get(r, 0)) for r in set(written) | set(old[1])})
            if merged != old:
                states[f] = merged
                todo.append(f)
    return sum(1 for code, _ in blocks.values() for c, inside in code if inside and c.startswith("v_mfma")), sorted(bad)


def test_matrix_instructions_in_assembly_are_waited_for(asm):
    found = 0
    for name, body in kernel_blocks(asm).items():
        count, bad = mfma_hazards(body)
        assert not bad, f"{name}: {bad[:5]}"
        assert (count > 0) == ("linear_wide_kernel" in name), name
        found += count
    assert found > 0


def test_only_the_tiles_are_waited_for_in_a_pass(asm):
    """A load that an epilogue leaves on its way is waited for in every pass of the next tile, and the tile's own with it."""
    for name, body in kernel_blocks(asm).items():
        if "linear_wide_kernel" in name:
            for code, _ in blocks_of(body).values():
                if any(c.startswith("v_mfma") for c, _ in code):
                    assert not [c for c, inside in code if "vmcnt" in c and not inside], name


def test_hazard_scan_detects_the_pattern():
    mfma = ";;#ASMSTART\n\tv_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[8:11], a[0:3]\n;;#ASMEND\n"
    wait = ";;#ASMSTART\n\ts_nop 15\n\ts_nop 15\n;;#ASMEND\n"
    read = "\tv_accvgpr_read_b32 v1, a2\n"
    nops = "\ts_nop 0\n\ts_nop 0\n\ts_nop 0\n"
    end = "\ts_endpgm\n"
    assert mfma_hazards(mfma + wait + read + end) == (1, [])
    assert mfma_hazards(mfma + read)[1] and mfma_hazards(mfma + "\ts_nop 15\n" + read)[1]
    assert mfma_hazards("\tv_mov_b32_e32 v9, v1\n" + mfma + wait)[1]
    assert mfma_hazards("\tv_accvgpr_write_b32 a1, v1\n\ts_nop 0\n" + mfma + wait)[1]
    assert not mfma_hazards("\tv_mov_b32_e32 v9, v1\n" + nops + mfma + wait)[1]
    assert mfma_hazards(mfma + read + mfma + wait)[1]
    # through jumps: out of a loop past its wait, and back into it
    loop = ".LBB0_1:\n" + mfma + "\ts_cbranch_scc1 .LBB0_1\n"
    assert not mfma_hazards(loop + wait + read + end)[1]
    assert mfma_hazards(loop + "\ts_branch .LBB0_3\n.LBB0_2:\n" + wait + end + ".LBB0_3:\n" + read + end)[1]
    assert not mfma_hazards(loop + "\ts_branch .LBB0_3\n.LBB0_2:\n" + read + end + ".LBB0_3:\n" + wait + end)[1]
    assert mfma_hazards(nops + ".LBB0_1:\n" + mfma + nops + "\tv_mov_b32_e32 v5, v1\n\ts_cbranch_scc1 .LBB0_1\n" + wait + end)[1]


@pytest.mark.parametrize("name", sorted(LIBRARIES))
def test_header_binding_and_exports_agree(built_library, name):
    src, header, lib, signatures, prefix = LIBRARIES[name]
    text = re.sub(r"/\*.*?\*/", "", header.read_text(), flags=re.S)
    declared = set(re.findall(r"\b(mhc_\w+)\s*\(", text))
    assert declared == set(signatures) and all(n.startswith(prefix) for n in declared)
    out = subprocess.run(["nm", "-D", "--defined-only", str(lib)], capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r"\bT (mhc_\w+)$", out, flags=re.M))
    assert exported == declared
    # as many arguments as the header has
    for fn, args in re.findall(r"\b(mhc_\w+)\s*\(([^)]*)\)", text):
        count = 0 if args.strip() in ("", "void") else args.count(",") + 1
        assert len(signatures[fn][1]) == count, fn


@pytest.mark.parametrize("name", sorted(LIBRARIES))
def test_headers_are_plain_c(tmp_path, name):
    header = LIBRARIES[name][1]
    source = tmp_path / "use.c"
    source.write_text(f'#include "{header.name}"\nint main(void) {{ return 0; }}\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", str(_build.INCLUDE_DIR), "-c", str(source),
                    "-o", str(tmp_path / "use.o")], check=True)


@pytest.mark.parametrize("name", sorted(LIBRARIES))
def test_fast_math_build_is_refused(tmp_path, name):
    src = LIBRARIES[name][0]
    proc = subprocess.run([_build.hipcc(), *_build.COMMON_FLAGS, "-ffast-math", "--cuda-device-only", "-fsyntax-only",
                           str(src)], capture_output=True, text=True)
    assert proc.returncode != 0 and "must not be built with fast-math" in proc.stdout + proc.stderr
    assert "#pragma clang fp contract(off)" in src.read_text()


def test_constants_match_the_headers(built_library):
    for name, values in (("gated", ("MHC_GATED_ABI_VERSION",)),
                         ("cross_entropy", ("MHC_CROSS_ENTROPY_ABI_VERSION", "MHC_REDUCTION_NONE", "MHC_REDUCTION_SUM",
                                            "MHC_REDUCTION_MEAN"))):
        text = LIBRARIES[name][1].read_text()
        for v in values:
            assert re.search(rf"^#define {v} {getattr(_lib, v)}\b", text, flags=re.M), v
    assert "#define MHC_GATED_MAX_BWD_N (1LL << 20)" in LIBRARIES["gated"][1].read_text()
    assert _lib.MHC_GATED_MAX_BWD_N == 1 << 20
    text = LIBRARIES["cross_entropy"][1].read_text()
    assert "#define MHC_CROSS_ENTROPY_MAX_V (1LL << 21)" in text and _lib.MHC_CROSS_ENTROPY_MAX_V == 1 << 21
    assert "#define MHC_CROSS_ENTROPY_CHUNK_BYTES (1LL << 30)" in text and _lib.MHC_CROSS_ENTROPY_CHUNK_BYTES == 1 << 30
    assert re.search(rf"^#define MHC_LINEAR_SHORT {_lib.MHC_LINEAR_SHORT}\b", _build.LINEAR_HEADER.read_text(), flags=re.M)
