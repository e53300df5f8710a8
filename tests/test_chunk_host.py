"""The chunk calls without a GPU: the attention's work shares (tests/chunk_walk.cu,
compiled and run on the host), the binding's argument checks, and the plain
forms the GPU tests compare with, against worked examples."""
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from compressed_paged_kv_gb300 import _build, zp
from tests.chunk_ref import attn_ref, verify_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_work_shares_cover_every_tile_once(tmp_path):
    exe = str(tmp_path / "chunk_walk")
    subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-O1", "-I", _build.INCLUDE, "-I",
                    _build.CSRC, os.path.join(ROOT, "tests", "chunk_walk.cu"), "-o", exe],
                   check=True, capture_output=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.startswith("ok"), res.stdout


class FakeTensor:
    """As much of a CUDA tensor as the binding looks at."""

    def __init__(self, shape, dtype=torch.bfloat16, strides=None, cuda=True):
        self.shape, self.dtype, self.is_cuda = tuple(shape), dtype, cuda
        if strides is None:
            strides, n = [], 1
            for s in reversed(self.shape):
                strides.insert(0, n)
                n *= s
        self._strides = tuple(strides)

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self._strides

    def numel(self):
        return math.prod(self.shape)

    def is_contiguous(self):
        return self._strides == FakeTensor(self.shape)._strides

    def data_ptr(self):
        return 4096


def _cache():
    c = zp.Cache.__new__(zp.Cache)
    c.handle = None  # the library answers a null handle with an error
    c.Hq, c.Hkv, c.d = 4, 2, 64
    c.dtype, c.int32, c.float32 = torch.bfloat16, torch.int32, torch.float32
    return c


I32 = torch.int32
F32 = torch.float32


def _attn_args(**kw):
    a = dict(layer=0, q=FakeTensor((7, 4, 64), strides=(512, 64, 1)), starts=FakeTensor((3,), I32),
             block_tables=FakeTensor((2, 5), I32), lengths=FakeTensor((2,), I32), scale=0.125,
             out=FakeTensor((7, 4, 64)), stream=FakeStream())
    a.update(kw)
    return a


class FakeStream:
    cuda_stream = 0


@pytest.fixture(autouse=True)
def _built():
    _build.build()


def test_good_arguments_reach_the_library():
    with pytest.raises(zp.ZpError) as e:
        _cache().chunk_attn(**_attn_args())
    assert e.value.status == zp.ERR_INVALID_ARG  # the null handle


@pytest.mark.parametrize("kw", [
    dict(q=FakeTensor((7, 3, 64))), dict(q=FakeTensor((7, 4, 32))), dict(q=FakeTensor((7, 256))),
    dict(q=FakeTensor((7, 4, 64), torch.float16)), dict(q=FakeTensor((7, 4, 64), cuda=False)),
    dict(q=FakeTensor((7, 4, 64), strides=(256, 1, 4))),
    dict(q=FakeTensor((7, 4, 64), strides=(512, 128, 1))),
    dict(out=FakeTensor((6, 4, 64))), dict(out=FakeTensor((7, 4, 64), F32)),
    dict(out=FakeTensor((7, 4, 64), strides=(512, 64, 1))),
    dict(starts=FakeTensor((3,), torch.int64)), dict(starts=FakeTensor((4,), I32)),
    dict(lengths=FakeTensor((1,), I32)), dict(lengths=FakeTensor((2,), torch.int64)),
    dict(block_tables=FakeTensor((2, 5), I32, strides=(8, 1))),
    dict(req_idx=FakeTensor((1,), I32)), dict(req_idx=FakeTensor((2,), torch.int64))])
def test_attention_arguments(kw):
    with pytest.raises(ValueError):
        _cache().chunk_attn(**_attn_args(**kw))


@pytest.mark.parametrize("kw", [
    dict(k_new=FakeTensor((7, 4, 64))), dict(v_new=FakeTensor((6, 2, 64))),
    dict(v_new=FakeTensor((7, 2, 64), F32)), dict(k_new=FakeTensor((7, 2, 64), strides=(512, 96, 1))),
    dict(starts=FakeTensor((5,), I32))])
def test_append_arguments(kw):
    a = dict(layer=0, k_new=FakeTensor((7, 2, 64), strides=(512, 64, 1)), v_new=FakeTensor((7, 2, 64)),
             starts=FakeTensor((3,), I32), block_tables=FakeTensor((2, 5), I32),
             lengths=FakeTensor((2,), I32), stream=FakeStream())
    with pytest.raises(zp.ZpError):
        _cache().append_kv_chunk(**a)
    a.update(kw)
    with pytest.raises(ValueError):
        _cache().append_kv_chunk(**a)


@pytest.mark.parametrize("kw", [
    dict(tokens=FakeTensor((7,), torch.int64)), dict(tokens=FakeTensor((6,), I32)),
    dict(target_probs=FakeTensor((7, 100), torch.float16)), dict(target_probs=FakeTensor((700,), F32)),
    dict(target_probs=FakeTensor((7, 100), F32, strides=(1, 7))),
    dict(draft_probs=FakeTensor((7, 100), F32, strides=(104, 1))),
    dict(draft_probs=FakeTensor((6, 100), F32)), dict(draft_probs=FakeTensor((7, 99), F32)),
    dict(accept_u=FakeTensor((6,), F32)), dict(sample_u=FakeTensor((1,), F32)),
    dict(accepted=FakeTensor((1,), I32)), dict(next_tokens=FakeTensor((2,), F32)),
    dict(lengths=FakeTensor((1,), I32)), dict(lengths=FakeTensor((2,), torch.int64)),
    dict(lengths=FakeTensor((4,), I32), req_idx=FakeTensor((1,), I32))])
def test_verification_arguments(kw):
    a = dict(tokens=FakeTensor((7,), I32), starts=FakeTensor((3,), I32),
             target_probs=FakeTensor((7, 100), F32), accept_u=FakeTensor((7,), F32),
             sample_u=FakeTensor((2,), F32), accepted=FakeTensor((2,), I32),
             next_tokens=FakeTensor((2,), I32), draft_probs=FakeTensor((7, 100), F32),
             stream=FakeStream())
    with pytest.raises(zp.ZpError):
        _cache().verify_draft(**a)
    a.update(kw)
    with pytest.raises(ValueError):
        _cache().verify_draft(**a)


# ------------------------------------------------------------ the plain forms

def test_attention_by_hand():
    """Two keys with scores 0 and ln 3: weights 1/4 and 3/4; the first of two
    queries sees the first key alone."""
    k = torch.tensor([[[0.0, 0.0]], [[math.log(3.0), 0.0]]])
    v = torch.tensor([[[4.0, 0.0]], [[0.0, 8.0]]])
    q = torch.ones(2, 1, 2)
    out, tol = attn_ref(q, k, v, 1.0)
    assert torch.allclose(out[:, 0], torch.tensor([[4.0, 0.0], [1.0, 6.0]], dtype=torch.float64))
    assert bool((tol < 0.1).all())


@pytest.mark.parametrize("u,r,want", [
    (0.49, 0.0, (1, 0)),    # accepted (0.49 * 0.4 < 0.2); then row 1's first token
    (0.49, 0.99, (1, 2)),   # ... its last
    (0.51, 0.0, (0, 0)),    # rejected; p - q = (0.1, -0.2, 0.1): token 0 or 2, half each
    (0.51, 0.51, (0, 2))])
def test_verification_by_hand(u, r, want):
    p = np.array([[0.5, 0.2, 0.3], [0.25, 0.25, 0.5]])
    q = np.array([[0.4, 0.4, 0.2], [0.0, 0.0, 0.0]])
    acc, nxt = verify_ref([9, 1], [0, 2], p, q, [u, 0.0], [r])
    assert (acc[0], nxt[0]) == want


def test_verification_without_draft_rows_by_hand():
    p = np.array([[0.5, 0.2, 0.3], [0.25, 0.25, 0.5]])
    assert verify_ref([9, 1], [0, 2], p, None, [0.19, 0.0], [0.6]) == ([1], [2])
    # rejected: token 1 left out, 0.5 and 0.3 remain
    assert verify_ref([9, 1], [0, 2], p, None, [0.21, 0.0], [0.62]) == ([0], [0])
    assert verify_ref([9, 1], [0, 2], p, None, [0.21, 0.0], [0.63]) == ([0], [2])
