"""The draws from logits without a GPU: tests/sample_launch.cu, compiled and run on the host."""
import os
import subprocess

from compressed_paged_kv_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_launches_ask_for_no_more_than_was_set(tmp_path):
    exe = str(tmp_path / "sample_launch")
    res = subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-O1", "-Xcicc", "-O0",
                          "-Xptxas", "-O0", "-I", _build.INCLUDE, "-I", _build.CSRC,
                          os.path.join(ROOT, "tests", "sample_launch.cu"), "-o", exe],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout + res.stderr
