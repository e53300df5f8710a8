"""The weights that the draws' kernels form, two at a time: tests/sample_weights.cu."""
import os
import subprocess

import pytest

from compressed_paged_kv_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("where", ["host", pytest.param("gpu", marks=pytest.mark.gpu)])
def test_weights(tmp_path, where):
    exe = str(tmp_path / "sample_weights")
    # (each operation of the host's is rounded by itself)
    res = subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-O1", "-Xcompiler",
                          "-ffp-contract=off", "-I", _build.INCLUDE, "-I", _build.CSRC,
                          os.path.join(ROOT, "tests", "sample_weights.cu"), "-o", exe],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe, where], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout + res.stderr
