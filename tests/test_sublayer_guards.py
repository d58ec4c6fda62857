"""Checks of the norm, product and write-back libraries' own gfx950 machine code
and exported names (compiled here; no GPU needed): no packed fp32 arithmetic,
no scalar memory writes, fp32 denormals kept, no spills to scratch, no store of
more than 8 bytes followed at once by an overwrite of its data, a fast-math
build refused, and headers, bindings and exports that agree."""

from __future__ import annotations

import re
import subprocess

import pytest

from hyper_connection_residual_mhc_amd import _build, _lib
from test_build_guards import (STORE_WIDE, instructions, kernel_blocks, store_data_regs,
                               written_vgprs)

LIBRARIES = {
    "norm": (_build.NORM_SRC, _build.NORM_HEADER, _build.NORM_LIB_PATH, _lib.NORM_SIGNATURES, "mhc_rms_norm_"),
    "linear": (_build.LINEAR_SRC, _build.LINEAR_HEADER, _build.LINEAR_LIB_PATH, _lib.LINEAR_SIGNATURES, "mhc_linear_"),
    "post": (_build.POST_SRC, _build.POST_HEADER, _build.POST_LIB_PATH, _lib.POST_SIGNATURES, "mhc_post_"),
}


@pytest.fixture(scope="module", params=sorted(LIBRARIES))
def asm(request, tmp_path_factory) -> str:
    out = tmp_path_factory.mktemp("asm") / f"{request.param}.s"
    return _build.device_asm(out, src=LIBRARIES[request.param][0]).read_text()


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


@pytest.mark.parametrize("name", sorted(LIBRARIES))
def test_header_binding_and_exports_agree(built_library, name):
    src, header, lib, signatures, prefix = LIBRARIES[name]
    text = re.sub(r"/\*.*?\*/", "", header.read_text(), flags=re.S)
    declared = set(re.findall(r"\b(mhc_\w+)\s*\(", text))
    assert declared == set(signatures) and all(n.startswith(prefix) for n in declared)
    out = subprocess.run(["nm", "-D", "--defined-only", str(lib)], capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r"\bT (mhc_\w+)$", out, flags=re.M))
    assert exported == declared


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
    for name, values in (("norm", ("MHC_NORM_ABI_VERSION", "MHC_NORM_F32", "MHC_NORM_BF16", "MHC_NORM_F16", "MHC_NORM_SAME",
                                   "MHC_NORM_E4M3_ROW", "MHC_NORM_E4M3_MX")),
                         ("linear", ("MHC_LINEAR_ABI_VERSION", "MHC_LINEAR_BF16", "MHC_LINEAR_F16", "MHC_LINEAR_E4M3_ROW",
                                     "MHC_LINEAR_E4M3_MX", "MHC_ACT_NONE", "MHC_ACT_RELU", "MHC_ACT_SILU", "MHC_ACT_GELU",
                                     "MHC_LINEAR_ROWS", "MHC_LINEAR_NARROW", "MHC_LINEAR_SMALL", "MHC_LINEAR_MEDIUM",
                                     "MHC_LINEAR_LARGE")),
                         ("post", ("MHC_POST_ABI_VERSION",))):
        text = LIBRARIES[name][1].read_text()
        for v in values:
            assert re.search(rf"^#define {v} {getattr(_lib, v)}\b", text, flags=re.M), v
    assert "#define MHC_LINEAR_MAX_K (1LL << 21)" in LIBRARIES["linear"][1].read_text()
    assert _lib.MHC_LINEAR_MAX_K == 1 << 21
