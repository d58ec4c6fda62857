"""The built libraries' own gfx950 code, as it is in the .so files of this tree: every
library is held to the one full list of scalar memory writes that
test_build_guards.py keeps, whichever shorter ones other guards look for."""

from __future__ import annotations

import shutil
import subprocess
from pathlib import Path

import pytest

from hyper_connection_residual_mhc_amd import _build

guards = pytest.importorskip("test_build_guards")


@pytest.fixture(scope="module")
def objdump() -> str:
    beside = Path(_build.hipcc()).resolve().parent.parent / "llvm" / "bin" / "llvm-objdump"
    path = str(beside) if beside.exists() else shutil.which("llvm-objdump")
    if path is None:
        pytest.skip("no llvm-objdump beside hipcc")
    return path


@pytest.mark.parametrize("lib", [lib for lib, _ in _build.LIBRARIES.values()], ids=lambda p: p.stem)
def test_no_scalar_memory_writes(built_library, objdump, lib, tmp_path):
    shutil.copy(lib, tmp_path)
    subprocess.run([objdump, "--offloading", lib.name], cwd=tmp_path, check=True, capture_output=True)
    code, = tmp_path.glob("*gfx950*")
    asm = subprocess.run([objdump, "-d", "--no-show-raw-insn", str(code)], check=True, capture_output=True,
                         text=True).stdout
    # the listing has an instruction to a line, behind white space, as the list expects them
    assert "\n\ts_endpgm" in asm and asm.count("\n\ts_load_dword") > 1
    guards.test_no_scalar_memory_writes(asm)
