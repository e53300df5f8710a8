"""Draws and filtered probabilities of the largest vocabulary: values and ties there, rows of equal
logits, whose weights' sums are the largest."""
import math

import numpy as np
import pytest
import torch

from tests.fp8_ref import border, draw_ref, filter_ref
from tests.test_gpu_sample import DEV, _built, cache, rows, run  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu
MOST = 352 * 1024


def check(cache, logits, u, t=None, k=None, p=None, m=None):  # noqa: F811
    """Against 64 bits.  A weight is off by 2^-40 of the largest at most, so a sum of V of them by
    `off` = V 2^-40 of it, 3.3e-7 here; a small temperature and a top_p near 1 leave single weights
    far below that (0.3 and 0.99999: 9e-9).  So a token may be kept or not whose place, the sum of
    those before it, lies within `off` (twice: of the sum and of the whole that top_p is a part
    of) of the border; probabilities and draws follow the kept ones, and draws are free within
    `off` of a border between tokens."""
    R, V = logits.shape
    got, probs = run(cache, logits, u, t, k, p, m)
    x = logits.double().cpu().numpy()
    off = V * 2.0 ** -40
    for i in range(R):
        f = [np.float64(np.float32(z[i])) if z is not None else dflt
             for z, dflt in ((t, 1.0), (k, 0), (p, 1.0), (m, 0.0))]
        w = filter_ref(x[i], *f)
        kept, odd = probs[i] > 0, (probs[i] > 0) != (w > 0)
        if odd.any():
            assert f[2] < 1.0 and 0 < f[0]
            top = x[i].max()
            order = np.argsort(-x[i], kind="stable")
            k_i = int(f[1]) if 0 < f[1] < V else V
            by = np.exp((x[i][order[:k_i]] - top) / f[0])
            before = np.cumsum(by) - by
            near = np.abs(before - f[2] * by.sum()) <= 2 * off
            assert set(np.flatnonzero(odd)) <= set(order[:k_i][near]), i
            w = np.where(kept, np.exp((x[i] - top) / f[0]), 0.0)
        u_i = float(np.float32(u[i]))
        assert got[i] == draw_ref(w, u_i) or border(w, u_i) <= 2 * off / w.sum(), i
        w = w / w.sum()
        # 2^-18 and 2^-24 as for smaller vocabularies, and the sum's error
        assert np.all(np.abs(probs[i] - w) <= (2.0 ** -18 + 2.0 ** -24 + 2 * off) * w + 2.0 ** -126), i


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [MOST, MOST - 7])
def test_the_largest_vocabulary(cache, V, dtype):  # noqa: F811
    x, u = rows(6, V, dtype, seed=V, pad=V % 5)
    check(cache, x, u, t=[1.0, 0.8, 1.0, 2.0, 0.3, 1.0], k=[0, 40, 0, 9000, 0, V - 1],
          p=[1.0, 0.9, 0.9, 1.0, 0.99999, 0.5], m=[0.0, 0.0, 0.0, 0.001, 0.0, 1e-6])


def test_equal_logits_of_the_largest_vocabulary(cache):  # noqa: F811
    x = torch.zeros(3, MOST, device=DEV)
    x[1] = -3e38
    x[2, ::2] = -math.inf
    u = np.array([0.999, 0.5, 0.25], np.float32)
    check(cache, x, u, p=[0.75, 1.0, 0.5], k=[0, MOST // 2, 0])
    check(cache, x, u)
