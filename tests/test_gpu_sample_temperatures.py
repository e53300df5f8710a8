"""Temperatures at the ends of the range that is taken as it is, 2^-120 to 2^120, and past them."""
import numpy as np
import pytest
import torch

from tests.fp8_ref import border, draw_ref, filter_ref
from tests.test_gpu_sample import DEV, _built, cache, run  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu
LOW, HIGH = 2.0 ** -120, 2.0 ** 120
U = np.array([0.1, 0.3, 0.5, 0.7, 0.9], np.float32)
FILTERS = dict(k=[0, 40, 0, 0, 700], p=[1.0, 1.0, 0.7, 1.0, 0.9], m=[0.0, 0.0, 0.0, 0.2, 0.05])


def check_as(cache, x, t, taken):  # noqa: F811
    """Rows at a temperature `t`, which is taken as `taken`.  A weight is off by 2^-40 of the largest,
    and by 2^-24 of itself above 2^100 (the low part of log2(e) / T, rounded to a multiple of 2^-149,
    puts an exponent of at most 48, a gap of 48 T ln 2 < 2^126, off by 2^-150 times that), and so are
    sums of them, by V times 2^-40 and by 2^-24 of themselves.  So a token may be kept or not whose
    place in the sum lies that near top_p's border (twice: of the sum and of the whole that top_p is a
    part of), and draws are free that near a border between tokens.  Probabilities as in
    tests/test_gpu_sample.py, to 2^-18."""
    got, probs = run(cache, x, U, [t] * 5, **FILTERS)
    V = x.shape[1]
    rel = 2.0 ** -24 if taken > 2.0 ** 100 else 0.0
    for i in range(5):
        k, p, m = (np.float64(np.float32(FILTERS[name][i])) for name in "kpm")
        row = x[i].double().cpu().numpy()
        w = filter_ref(row, taken, k, p, m)
        odd = (probs[i] > 0) != (w > 0)
        if odd.any():  # (or its probability is no normal fp32 number)
            order = np.argsort(-row, kind="stable")[:int(k) if 0 < k < V else V]
            by = np.exp((row[order] - row.max()) / taken)
            near = np.abs(np.cumsum(by) - by - p * by.sum()) <= 2 * (rel * by.sum() + V * 2.0 ** -40)
            free = set(order[near]) if p < 1.0 else set()
            lost = set(np.flatnonzero((w > 0) & (w < 2.0 ** -125 * w.sum())))
            assert set(np.flatnonzero(odd)) <= free | lost, i
            w = np.where(np.isin(np.arange(V), list(free)), np.where(
                probs[i] > 0, np.exp((row - row.max()) / taken), 0.0), w)
        total = w.sum()
        assert got[i] == draw_ref(w, float(U[i])) or border(w, float(U[i])) <= 2 * (
            rel + V * 2.0 ** -40 / total), i
        assert np.all(np.abs(probs[i] - w / total) <= (2.0 ** -18 + 2.0 ** -24) * w / total +
                      2.0 ** -126), i


@pytest.mark.parametrize("t", [1e-30, 1e-35, 2.0 ** -120, 1e-37, 1e-38, 1e-45])
@pytest.mark.parametrize("spread", [4.0, 1e-5])
def test_the_lowest(cache, t, spread):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(4)
    x = -spread * max(t, LOW) * torch.rand(5, 3000, generator=g, device=DEV)
    check_as(cache, x, t, max(float(np.float32(t)), LOW))


@pytest.mark.parametrize("t", [1e30, 2.0 ** 100, 1e31, 1e35, 2.0 ** 120, 3e38])
@pytest.mark.parametrize("size", [1.0, 1e30, 1e36, 1e38])
def test_the_highest(cache, t, size):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(5)
    x = size * torch.randn(5, 3000, generator=g, device=DEV).clamp(-3.4, 3.4)
    x[:, 5] = -3e38
    check_as(cache, x, t, min(float(np.float32(t)), HIGH))
