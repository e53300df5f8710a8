"""The 8-bit cache and the draws from logits without a GPU: tests/fp8_host.cu, compiled and run on
the host; the binding's checks; the plain forms that the GPU tests compare with, by hand."""
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from compressed_paged_kv_gb300 import _build, zp
from tests.fp8_ref import attn_ref, draw_ref, filter_ref, scale_of
from tests.test_chunk_host import F32, I32, FakeStream, FakeTensor, _cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    lib = _build.build()
    out = str(tmp_path_factory.mktemp("fp8_host") / "fp8_host")
    res = subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-O1", "-I", _build.INCLUDE,
                          "-I", _build.CSRC, os.path.join(ROOT, "tests", "fp8_host.cu"), "-o", out,
                          lib, "-Xlinker", "-rpath", "-Xlinker", os.path.dirname(lib)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return out


@pytest.mark.parametrize("what", ["walk", "calls", "draws", "weights"])
def test_host(exe, what):
    res = subprocess.run([exe, what], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout + res.stderr


def _draw_args(**kw):
    a = dict(logits=FakeTensor((3, 100), F32, strides=(104, 1)), temperature=FakeTensor((3,), F32),
             top_k=FakeTensor((3,), I32), top_p=FakeTensor((3,), F32), min_p=FakeTensor((3,), F32),
             stream=FakeStream())
    a.update(kw)
    return a


BAD = [dict(logits=FakeTensor((300,), F32)), dict(logits=FakeTensor((3, 100), torch.float16)),
       dict(logits=FakeTensor((3, 100), F32, cuda=False)),
       dict(logits=FakeTensor((3, 100), F32, strides=(1, 3))),
       dict(temperature=FakeTensor((3,), torch.float64)), dict(top_k=FakeTensor((3,), torch.int64)),
       dict(top_p=FakeTensor((2,), F32)), dict(min_p=FakeTensor((4,), F32)),
       dict(temperature=FakeTensor((3,), F32, strides=(2,))), dict(req_idx=FakeTensor((2,), I32)),
       dict(req_idx=FakeTensor((3,), torch.int64)),
       dict(temperature=None, top_k=FakeTensor((2,), I32), top_p=None, min_p=None)]


@pytest.mark.parametrize("kw", BAD + [dict(u=FakeTensor((2,), F32)), dict(tokens=FakeTensor((3,), F32)),
                                      dict(tokens=FakeTensor((2,), I32))])
def test_sample_arguments(kw):
    a = dict(u=FakeTensor((3,), F32), tokens=FakeTensor((3,), I32))
    with pytest.raises(zp.ZpError):  # the null handle
        _cache().sample(**_draw_args(**a))
    a.update(kw)
    with pytest.raises(ValueError):
        _cache().sample(**_draw_args(**a))


@pytest.mark.parametrize("kw", BAD + [dict(probs=FakeTensor((2, 100), F32)),
                                      dict(probs=FakeTensor((3, 99), F32)),
                                      dict(probs=FakeTensor((3, 100), torch.float16))])
def test_token_probs_arguments(kw):
    a = dict(probs=FakeTensor((3, 100)))
    with pytest.raises(zp.ZpError):
        _cache().token_probs(**_draw_args(**a))
    a.update(kw)
    with pytest.raises(ValueError):
        _cache().token_probs(**_draw_args(**a))


# ------------------------------------------------------------ the plain forms

LOGITS = np.log([0.1, 0.4, 0.2, 0.3])


@pytest.mark.parametrize("kw,want", [
    (dict(), [0.1, 0.4, 0.2, 0.3]), (dict(k=2), [0, 0.4, 0, 0.3]), (dict(t=0.0), [0, 1, 0, 0]),
    (dict(p=0.41), [0, 0.4, 0, 0.3]), (dict(p=0.39), [0, 1, 0, 0]), (dict(m=0.51), [0, 0.4, 0, 0.3]),
    (dict(t=0.5), [0.01, 0.16, 0.04, 0.09]), (dict(k=3, p=0.77), [0, 0.4, 0, 0.3])])
def test_filters_by_hand(kw, want):
    w, want = filter_ref(LOGITS, **kw), np.asarray(want)
    assert np.allclose(w / w.sum(), want / want.sum())


def test_draws_by_hand():
    w = filter_ref(LOGITS)
    assert [draw_ref(w, u) for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.99)] == [
        0, 0, 1, 1, 2, 2, 3, 3]


def test_attention_by_hand():
    """Two keys with scores 0 and ln 3, the second hidden from the first token."""
    k = torch.tensor([[[0.0, 0.0]], [[math.log(3.0), 0.0]]])
    v = torch.tensor([[[4.0, 0.0]], [[0.0, 8.0]]])
    out, tol = attn_ref(torch.ones(2, 1, 2), k, v, 1.0)
    assert torch.allclose(out[:, 0], torch.tensor([[4.0, 0.0], [1.0, 6.0]], dtype=torch.float64))
    assert bool((tol < 0.1).all())


def test_scales_by_hand():
    x = torch.tensor([448.0, 449.0, 224.0, 1.0, 0.0, 2.0 ** -40, 3e38])
    assert scale_of(x).tolist() == [1.0, 2.0, 0.5, 2.0 ** -8, 2.0 ** -32, 2.0 ** -32, 2.0 ** 32]
