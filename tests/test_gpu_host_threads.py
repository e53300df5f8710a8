"""Calls that two host threads make at once: tests/host_threads.cu."""
import os
import subprocess

import pytest

from compressed_paged_kv_gb300 import _build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    lib = _build.build()
    out = str(tmp_path_factory.mktemp("host_threads") / "host_threads")
    subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-O1", "-I", _build.INCLUDE,
                    os.path.join(ROOT, "tests", "host_threads.cu"), "-o", out, lib, "-Xlinker",
                    "-rpath", "-Xlinker", os.path.dirname(lib)], check=True, capture_output=True)
    return out


@pytest.mark.parametrize("what", ["draws"])
def test_at_once(exe, what):
    res = subprocess.run([exe, what], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout + res.stderr
