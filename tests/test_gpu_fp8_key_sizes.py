"""Attention over an 8-bit cache whose keys are zeros, tiny or huge, under queries that are zero,
ordinary or huge: every path (single tokens, few rows, one tile, two heads at a time, pairs of
tiles, blocks widened to bf16) against 64 bits."""
import math

import pytest
import torch

from compressed_paged_kv_gb300 import zp
from tests.fp8_ref import B, E4M3, WIDE_ROWS, Batch8, attn_ref, scale_of

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from compressed_paged_kv_gb300 import _build
    _build.build()
    yield
    torch.cuda.empty_cache()


# (spans, Hkv): a group has four heads
PATHS = {"single": ([(1, 20 * i + 1) for i in range(20)], 2),
         "few": ([(4, 70), (3, 200), (1, 33), (2, 2)], 2),
         "tile": ([(20, 300), (30, 40), (16, 16)], 2),
         "heads": ([(9, 130 + i) for i in range(80)], 4),
         "pairs": ([(100, 500), (60, 60)], 2),
         "widened": ([(400, 700)], 2)}


def batch(path, d):
    spans, Hkv = PATHS[path]
    return Batch8(spans, Hkv=Hkv, Hq=4 * Hkv, d=d, seed=d + len(spans), packed=False)


def set_keys(b, sizes, change=lambda x: x):
    """Keys of normal deviation `sizes`, block after block in turn (0: zeros), as an append would
    round them; slots past the length hold NaN."""
    g = torch.Generator(device=DEV).manual_seed(17)
    pool, scale = b.kp[0].view(torch.uint8), b.ks[0]
    for i, (_, T) in enumerate(b.spans):
        m = -(-T // B)
        blocks = b.tables[b.order[i], :m].long()
        size = torch.tensor([sizes[j % len(sizes)] for j in range(m)], device=DEV)
        x = change(torch.randn(m, b.Hkv, B, b.d, generator=g, device=DEV) * size[:, None, None, None])
        s = scale_of(x.abs().amax((2, 3))).float()
        y = (x / s[..., None, None]).to(E4M3).view(torch.uint8)
        if T % B:
            y[-1, :, T % B:] = 0x7f
        pool[blocks], scale[blocks] = y, s


def run(b, path):
    c = b.cache()
    b.decode(c) if path == "single" else b.attn(c)
    assert c.status() == zp.OK


KEYS = {"zeros": [0.0], "2^-40": [2.0 ** -40], "1e-6": [1e-6], "2^30": [2.0 ** 30],
        "mixed": [0.0, 1.0, 2.0 ** -40, 1e-6]}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q", ["zeros", "ordinary", "huge", "scale 0"])
@pytest.mark.parametrize("keys", KEYS)
@pytest.mark.parametrize("path", PATHS)
def test_keys_of_every_size(path, keys, q, d):
    b = batch(path, d)
    set_keys(b, KEYS[keys])
    if keys == "2^30":
        b.scale *= 2.0 ** -30  # (scores stay below 2^20)
    if q == "zeros":
        b.q[::2] = 0
    elif q == "huge":
        b.q = (b.q.float() * 2.0 ** 90).bfloat16()
        b.scale *= 2.0 ** -90
    elif q == "scale 0":
        b.scale = 0.0
    run(b, path)
    b.check_attn(split=0.0 if path == "single" else 2.0 ** -17)


def check_a_query_that_meets_no_key(path, d):
    """Every score is 0: the query has one element, a power of two (so that its rounding loses
    nothing), where the keys have zeros; the two scales' product is no fp32 number."""
    def without_first(x):
        x[..., 0] = 0
        return x

    b = batch(path, d)
    set_keys(b, [2.0 ** 38, 1.0], without_first)  # (4.5 deviations: 2^40.2, below 448 times 2^32)
    b.q.zero_()
    b.q[..., 0] = 2.0 ** 120
    run(b, path)
    for i, (n, T) in enumerate(b.spans):
        a = int(b.starts_np[i])
        k, v = b.rows_of(i)
        assert bool(k.isfinite().all())
        want, tol = attn_ref(b.q[a:a + n], k, v, b.scale, 0.0,
                             2.0 ** -8 if n * 4 >= WIDE_ROWS else 2.0 ** -11)
        err = (b.out[a:a + n].double() - want).abs()
        assert bool((err <= tol).all()), (i, float((err / tol).nan_to_num(math.inf).max()))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("path", ["tile", "heads", "pairs", "widened"])
def test_huge_keys_that_a_huge_query_does_not_meet(path, d):
    check_a_query_that_meets_no_key(path, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("path", ["single", "few"])
def test_few_rows_of_huge_queries_that_meet_no_key(path, d):
    check_a_query_that_meets_no_key(path, d)
