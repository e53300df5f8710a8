"""The C ABI's host side without a GPU: tests/api_host.cu, compiled and run on
the host."""
import os
import subprocess

import pytest

from compressed_paged_kv_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    lib = _build.build()
    out = str(tmp_path_factory.mktemp("api_host") / "api_host")
    subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-O1", "-I", _build.INCLUDE, "-I",
                    _build.CSRC, os.path.join(ROOT, "tests", "api_host.cu"), "-o", out, lib,
                    "-Xlinker", "-rpath", "-Xlinker", os.path.dirname(lib)],
                   check=True, capture_output=True)
    return out


def _run(exe, what):
    res = subprocess.run([exe, what], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout + res.stderr


def test_a_status_clears_its_own_word_only(exe):
    _run(exe, "status")


def test_shared_memory_is_refused(exe):
    _run(exe, "shared")


def test_limits_of_a_verification(exe):
    _run(exe, "limits")
