"""The functions that read a unit's fault flag belong to that unit: a flag is a
variable of its translation unit, so a function shared by the linker would read
one unit's flag for all of them (no GPU needed, nothing runs)."""
import os
import shutil
import subprocess

import pytest

from residual_add_rmsnorm_rmsq_gb300 import _build


@pytest.mark.skipif(shutil.which("nm") is None, reason="needs nm")
@pytest.mark.parametrize("header, reader", [("rmsq_attn_launch.cuh", "take_fault_of_unit"), ("rmsq_dispatch.cuh", "take_pipe_fault")])
def test_readers_of_fault_flags_are_local_to_their_unit(tmp_path, header, reader):
    """Compiled without inlining, the reader is a local symbol ("t"), not one that the
    linker may merge ("W") or export ("T")."""
    source, obj = tmp_path / "unit.cu", tmp_path / "unit.o"
    source.write_text(f'#include <cuda_runtime.h>\n#include "{header}"\n'
                      f"cudaError_t probe(unsigned int* out) {{ return rmsq::{reader}(out); }}\n")
    subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-Xcompiler", "-O0,-fno-inline", "-I", _build.INCLUDE, "-I", _build.CSRC,
                    "-c", os.fspath(source), "-o", os.fspath(obj)], check=True, capture_output=True)
    lines = subprocess.run(["nm", "-C", os.fspath(obj)], check=True, capture_output=True, text=True).stdout.splitlines()
    kinds = [line.split()[-2] if "(" not in line else line.split("rmsq::")[0].split()[-1] for line in lines if f"rmsq::{reader}(" in line]
    assert kinds == ["t"], kinds
