"""Tokens and filtered probabilities from logits, against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

from compressed_paged_kv_gb300 import zp
from tests.fp8_ref import border, draw_ref, filter_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from compressed_paged_kv_gb300 import _build
    _build.build()
    yield
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def cache():
    pool = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device=DEV)
    return zp.Cache([pool], [pool.clone()], 1, max_requests=4096, max_blocks_per_req=2)


def _f(x):
    return torch.tensor(x, dtype=torch.float32, device=DEV)


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def run(cache, logits, u, t=None, k=None, p=None, m=None, idx=None, prob=torch.float32):
    """Tokens and probabilities of rows of logits, filters given as lists."""
    R = logits.shape[0]
    kw = dict(temperature=None if t is None else _f(t), top_k=None if k is None else _i(k),
              top_p=None if p is None else _f(p), min_p=None if m is None else _f(m),
              req_idx=None if idx is None else _i(idx))
    tokens = torch.full((R,), -7, dtype=torch.int32, device=DEV)
    cache.sample(logits, _f(u), tokens, **kw)
    probs = torch.full((R, logits.shape[1] + 3), 9.0, dtype=prob, device=DEV)
    cache.token_probs(logits, probs[:, :logits.shape[1]], **kw)
    assert cache.status() == zp.OK
    assert bool((probs[:, logits.shape[1]:] == 9.0).all())
    return tokens.cpu().numpy(), probs[:, :logits.shape[1]].double().cpu().numpy()


def check(cache, logits, u, t=None, k=None, p=None, m=None, idx=None, prob=torch.float32):
    """Against 64 bits.  A token may differ only where u lies within 2^-38 of a border
    (weights are off by 2^-40 at most, and their sums by V times that at worst); a
    probability by 2^-18 of itself (the fp32 exponent's rounding, of at most 2^-24 times
    150, and the exponential's 2^-22), rounded to its type (2^-8 in bf16)."""
    R, V = logits.shape
    u = np.asarray(u, np.float32)
    got, probs = run(cache, logits, u, t, k, p, m, idx, prob)
    x = logits.double().cpu().numpy()
    rel = 2.0 ** -18 + (2.0 ** -8 if prob == torch.bfloat16 else 2.0 ** -24)
    at = np.arange(R) if idx is None else np.asarray(idx)
    for i in range(R):
        j = int(at[i])
        w = filter_ref(x[i], *(np.float64(np.float32(z[j])) if z is not None else dflt
                               for z, dflt in ((t, 1.0), (k, 0), (p, 1.0), (m, 0.0))))
        want = draw_ref(w, float(u[i]))
        assert got[i] == want or border(w, float(u[i])) < 2.0 ** -38, (i, got[i], want)
        w = w / w.sum()
        # below 2^-126 flushed to 0
        assert np.all(np.abs(probs[i] - w) <= rel * w + 2.0 ** -126), (
            i, np.abs(probs[i] - w).max(), int(((probs[i] > 0) != (w > 0)).sum()))


def rows(R, V, dtype=torch.float32, seed=0, sigma=3.0, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.zeros(R, V + pad, dtype=dtype, device=DEV)
    s = sigma * (0.3 + torch.rand(R, 1, generator=g, device=DEV))
    x[:, :V] = (s * torch.randn(R, V, generator=g, device=DEV)).to(dtype)
    return x[:, :V], np.random.default_rng(seed).random(R).astype(np.float32)


DTYPES = [torch.float32, torch.bfloat16]
SIZES = [1, 2, 3, 7, 8, 31, 100, 511, 513, 1000, 4097, 32000, 50257, 151936]


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("V", SIZES)
def test_no_filters(cache, V, dtype):
    x, u = rows(5, V, dtype, seed=V, pad=V % 3)
    check(cache, x, u)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("V", SIZES)
def test_filters(cache, V, dtype):
    R = 12
    x, u = rows(R, V, dtype, seed=V + 1, pad=1)
    check(cache, x, u, t=[1.0, 0.7, 0.0, 1.5, 1.0, 0.9, 0.2, 4.0, 1.0, 1.0, 0.5, 1.0],
          k=[50, 1, 0, 7, 0, 300, 2000, 0, V, -3, 5, 0],
          p=[1.0, 0.9, 0.5, 0.8, 0.95, 0.3, 0.999, 0.9, 2.0, 0.0, 0.7, 0.6],
          m=[0.0, 0.1, 0.2, 0.05, 0.0, 0.0, 0.01, 0.0, 0.5, 0.0, -1.0, 1.5])


@pytest.mark.parametrize("name", ["k", "p", "m", "t"])
def test_one_filter_alone(cache, name):
    x, u = rows(6, 20000, seed=4)
    kw = {"k": [1, 2, 1024, 1025, 5000, 19999], "p": [0.01, 0.5, 0.9, 0.99, 0.9999, 1.0],
          "m": [1.0, 0.5, 0.1, 1e-3, 1e-10, 0.0], "t": [0.0, 0.1, 0.5, 1.0, 2.0, 50.0]}
    check(cache, x, u, **{name: kw[name]})


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [10, 5000, 60000])
def test_ties(cache, V, dtype):
    """Rows of few values: cuts that fall among equal logits keep the lowest indices."""
    g = torch.Generator(device=DEV).manual_seed(V)
    R = 8
    x = torch.randint(0, 3, (R, V), generator=g, device=DEV).to(dtype)
    x[0] = 2.5
    x[1] = -4.0
    x[2, 3:] = -math.inf
    x[3] = torch.where(x[3] == 0, -0.0, 0.0)
    u = np.linspace(0.0, 0.999, R).astype(np.float32)
    # (sums that reach a quarter or half of the whole exactly, with equal weights)
    check(cache, x, u, k=[V // 2, 0, 2, 4, V // 3 + 1, 0, 3, V - 1],
          p=[1.0, 0.5, 1.0, 0.25, 0.77, 0.81, 1.0, 0.4], t=[1.0] * 4 + [0.8, 1.0, 2.0, 1.3])


def test_values_that_are_no_numbers(cache):
    V = 3000
    x, u = rows(8, V, seed=9)
    x[0, ::2] = math.nan
    x[1, 5] = math.inf
    x[2, 7] = x[2, 2900] = math.inf
    x[3] = -math.inf
    x[3, 1234] = -3.0
    x[4, :] = -math.inf
    x[4, :10] = 3e38
    x[4, 10:20] = -3e38
    x[5] = 1e-42
    x[5, 77] = 2e-42
    x[6] *= 1e30
    x[7, 1:] = math.nan
    check(cache, x, u)
    check(cache, x, u, k=[40] * 8, p=[0.9] * 8, m=[0.01] * 8, t=[0.8] * 8)


def test_wide_and_narrow_rows(cache):
    """Every logit within a few steps of its type, far outliers beside a narrow row,
    temperatures far from 1."""
    V = 40000
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(6, V, generator=g, device=DEV)
    x[0] = 1.0 + 1e-6 * x[0]
    x[1] = 1e-3 * x[1]
    x[1, 100] = -1e6
    x[2] = 1e4 + x[2]
    x[3] = 1e-5 * x[3]
    x[3, 3] = 5.0
    u = np.array([0.1, 0.3, 0.5, 0.7, 0.9, 0.99], np.float32)
    for t in (1.0, 1e-4, 1e3, 1e-30, 1e30):
        check(cache, x, u, t=[t] * 6, p=[0.7] * 6)
        check(cache, x, u, t=[t] * 6, k=[3000] * 6)
        check(cache, x, u, t=[t] * 6)


def test_filters_of_a_chunk(cache):
    """Rows that share a request's filters, in any order."""
    x, u = rows(30, 5000, torch.bfloat16, seed=11, pad=8)
    idx = [3, 3, 0, 1, 2, 2, 2, 4, 0, 3] * 3
    check(cache, x, u, t=[1.0, 0.5, 0.0, 0.9, 2.0], k=[0, 10, 0, 50, 3], p=[0.9, 1.0, 0.5, 0.8, 0.99],
          idx=idx, prob=torch.bfloat16)


def test_many_rows(cache):
    x, u = rows(1000, 777, seed=13)
    check(cache, x, u, k=[i % 40 for i in range(1000)], p=[0.5 + i % 7 / 12 for i in range(1000)])


def test_random_numbers_at_the_ends(cache):
    x, _ = rows(4, 900, seed=2)
    u = np.array([0.0, 1.0 - 2.0 ** -24, 2.0 ** -30, 2.0 ** -149], np.float32)
    check(cache, x, u)


def test_bad_entries_and_rows(cache):
    x, u = rows(6, 500, seed=6)
    x[5] = -math.inf
    tokens = torch.full((6,), -7, dtype=torch.int32, device=DEV)
    good = _f([1.0] * 6)
    for t, p, m, idx in (([1, -1, 1, 1, 1, 1], [1] * 6, [0] * 6, [0, 1, 2, 3, 4, 5]),
                         ([1, math.inf, 1, 1, 1, 1], [1] * 6, [0] * 6, [0, 1, 2, 3, 4, 5]),
                         ([1] * 6, [1, math.nan, 1, 1, 1, 1], [0] * 6, [0, 1, 2, 3, 4, 5]),
                         ([1] * 6, [1] * 6, [0, math.nan, 0, 0, 0, 0], [0, 1, 2, 3, 4, 5]),
                         ([1] * 6, [1] * 6, [0] * 6, [0, 6, 2, 3, 4, 5]),
                         ([1] * 6, [1] * 6, [0] * 6, [0, -1, 2, 3, 4, 5])):
        probs = torch.full((6, 500), 3.0, device=DEV)
        cache.sample(x, _f(u), tokens, _f(t), top_p=_f(p), min_p=_f(m), req_idx=_i(idx))
        assert cache.status() == zp.ERR_DEVICE_CHECK
        cache.token_probs(x, probs, _f(t), top_p=_f(p), min_p=_f(m), req_idx=_i(idx))
        assert cache.status() == zp.ERR_DEVICE_CHECK
        got = tokens.cpu().numpy()
        for i in range(6):
            if i in (1, 5):
                assert got[i] == -1 and bool((probs[i] == 0).all())
            else:
                w = filter_ref(x[i].double().cpu().numpy())
                assert got[i] == draw_ref(w, float(u[i]))
    del good


def test_refusals(cache):
    x, u = rows(3, 100)
    u = _f(u)
    tokens = torch.zeros(3, dtype=torch.int32, device=DEV)
    probs = torch.zeros(3, 100, device=DEV)
    assert cache.sample(x[:0], u[:0], tokens[:0]) == zp.OK
    with pytest.raises(ValueError):
        cache.sample(x.half(), u, tokens)
    with pytest.raises(ValueError):
        cache.sample(x, u, tokens.long())
    with pytest.raises(ValueError):
        cache.sample(x, u, tokens, temperature=_f([1.0, 1.0]))
    with pytest.raises(ValueError):
        cache.sample(x, u, tokens, temperature=_f([1.0] * 3), top_k=_i([1] * 4))
    with pytest.raises(ValueError):
        cache.token_probs(x, probs[:2])
    with pytest.raises(ValueError):
        cache.sample(x.t(), u, tokens)
    assert cache.token_probs(x, x, check=False) == zp.ERR_INVALID_ARG
    big = torch.zeros(1, 360449, device=DEV)
    assert cache.sample(big, u[:1], tokens[:1], check=False) == zp.ERR_UNSUPPORTED
    assert cache.sample(big[:, :360448], u[:1], tokens[:1]) == zp.OK
    assert cache.status() == zp.OK
