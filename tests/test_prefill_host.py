"""The compression at admission without a GPU: tests/prefill_launch.cu, run on the host."""
import os
import subprocess

from compressed_paged_kv_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_limit_of_shared_memory_is_the_same_in_every_call(tmp_path):
    exe = str(tmp_path / "prefill_launch")
    res = subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-O1", "-Xcicc", "-O0",
                          "-Xptxas", "-O0", "-I", _build.INCLUDE, "-I", _build.CSRC,
                          os.path.join(ROOT, "tests", "prefill_launch.cu"), "-o", exe],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout + res.stderr
