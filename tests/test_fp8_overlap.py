"""Chunk calls over an 8-bit cache whose kernels overlap: tests/fp8_overlap.cu on the host, and
tests/fp8_overlap_state.cu on a GPU."""
import os
import subprocess

import pytest

from compressed_paged_kv_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(tmp_path, name):
    lib = _build.build()
    exe = str(tmp_path / name)
    res = subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-O1", "-I", _build.INCLUDE, "-I",
                          _build.CSRC, os.path.join(ROOT, "tests", name + ".cu"), "-o", exe, lib,
                          "-Xlinker", "-rpath", "-Xlinker", os.path.dirname(lib)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout + res.stderr


def test_who_says_and_who_clears(tmp_path):
    run(tmp_path, "fp8_overlap")


@pytest.mark.gpu
def test_the_word_between_calls(tmp_path):
    run(tmp_path, "fp8_overlap_state")
