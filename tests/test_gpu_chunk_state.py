"""The chunk attention's state between calls: tests/chunk_state.cu."""
import os
import subprocess

import pytest

from compressed_paged_kv_gb300 import _build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_calls_after_one_that_gave_up(tmp_path):
    lib = _build.build()
    exe = str(tmp_path / "chunk_state")
    subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-O1", "-I", _build.INCLUDE, "-I",
                    _build.CSRC, os.path.join(ROOT, "tests", "chunk_state.cu"), "-o", exe, lib,
                    "-Xlinker", "-rpath", "-Xlinker", os.path.dirname(lib)],
                   check=True, capture_output=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout + res.stderr
