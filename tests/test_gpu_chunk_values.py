"""Values that are not finite in a chunk's attention: they reach the rows that
see them, in their dims, and no others; and a call with them costs a few times
a clean one at most."""
import math

import pytest
import torch

from compressed_paged_kv_gb300 import zp
from tests.chunk_ref import B, Batch, attn_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from compressed_paged_kv_gb300 import _build
    _build.build()
    yield
    torch.cuda.empty_cache()


def _poison(b, share, early, seed):
    """Puts NaN, inf and -inf into a `share` of the value elements of each
    request's own chunk and, where `early`, into one dim of one key before it;
    every third request stays clean."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    bad = torch.tensor([math.nan, math.inf, -math.inf], device=DEV).bfloat16()
    for i, (n, T) in enumerate(b.spans):
        if n == 0 or i % 3 == 2:
            continue
        blocks = b.tables[b.order[i]].long()
        pos = torch.arange(T - n, T, device=DEV)
        v = b.vp[0][blocks[pos // B], :, pos % B]
        hit = torch.rand(v.shape, generator=g, device=DEV) < share
        pick = bad[torch.randint(0, 3, v.shape, generator=g, device=DEV)]
        b.vp[0][blocks[pos // B], :, pos % B] = torch.where(hit, pick, v)
        if early and T > n:
            t = int(torch.randint(0, T - n, (1,), generator=g, device=DEV))
            b.vp[0][blocks[t // B], i % b.Hkv, t % B, i % b.d] = bad[i % 2]


def _check(b):
    """Finite elements within the bound of the 64-bit result without the values
    that are not finite; the others of the sign (or NaN) that the rows' sums
    have."""
    for i, (n, T) in enumerate(b.spans):
        if n == 0:
            continue
        a = int(b.starts_np[i])
        k, v = b.rows_of(i)
        want, tol = attn_ref(b.q[a:a + n], k, torch.where(torch.isfinite(v), v, 0.0), b.scale)
        up = (~(v < math.inf)).cumsum(0)[T - n:] > 0     # [n, Hkv, d]: inf or NaN seen
        down = (~(v > -math.inf)).cumsum(0)[T - n:] > 0
        up, down = (x.repeat_interleave(b.Hq // b.Hkv, 1) for x in (up, down))
        got = b.out[a:a + n].double()
        assert bool(torch.isnan(got)[up & down].all()), i
        assert bool((got == math.inf)[up & ~down].all()), i
        assert bool((got == -math.inf)[down & ~up].all()), i
        ok = (got - want).abs() <= tol
        assert bool(ok[~up & ~down].all()), (i, n, T)


SHAPES = [([(64, 900)] * 100, 2, 8), ([(3, 700)] * 400, 2, 8), ([(200, 3000)], 1, 4),
          ([(5, 4000)], 2, 8), ([(200, 300), (255, 255), (256, 700)] * 12, 1, 1),
          ([(40, 130), (1, 17), (0, 5), (130, 517), (7, 128)] * 5, 2, 14),
          ([(9, 2000), (300, 333)] * 3, 1, 16), ([(700, 700), (1, 900), (33, 40)], 8, 32)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("early", [False, True])
@pytest.mark.parametrize("spans,Hkv,Hq", SHAPES)
def test_rows_see_what_is_theirs(spans, Hkv, Hq, early, d):
    b = Batch(spans, Hkv, Hq, d, seed=51, permute=True, heavy=0.0)
    _poison(b, 0.002, early, 52)
    cache = b.cache()
    b.attn(cache)
    assert cache.status() == zp.OK
    _check(b)
    first = b.out.clone()
    for _ in range(2):
        b.out.fill_(7.0)
        b.attn(cache)
        assert torch.equal(b.out.view(torch.int16), first.view(torch.int16))


def test_every_value_hidden_and_not_finite():
    """All values of the chunk but its first token's: one row of it is finite."""
    b = Batch([(130, 1000), (40, 40)], 2, 8, 128, seed=53, heavy=0.0)
    _poison(b, 2.0, False, 54)
    for i, (n, T) in enumerate(b.spans):
        blk = b.tables[i, (T - n) // B].long()
        b.vp[0][blk, :, (T - n) % B] = 0.5
    cache = b.cache()
    b.attn(cache)
    assert cache.status() == zp.OK
    _check(b)


def test_clean_calls_after_it_are_as_before():
    b = Batch([(64, 900)] * 30 + [(5, 3000)], 2, 8, 128, seed=55)
    cache = b.cache()
    b.attn(cache)
    first, v = b.out.clone(), b.vp[0].clone()
    _poison(b, 0.01, True, 56)
    b.attn(cache)
    b.vp[0].copy_(v)
    for _ in range(3):
        b.attn(cache)
        assert cache.status() == zp.OK
        assert torch.equal(b.out.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("where", ["first key", "last key", "chunk"])
@pytest.mark.parametrize("spans,Hkv,Hq,d", [([(64, 2000)] * 160, 2, 8, 128), ([(5, 9000)] * 8, 8, 32, 128),
                                            ([(2000, 2000)] * 8, 2, 8, 64), ([(400, 2000)] * 9, 2, 2, 64)])
def test_cost(spans, Hkv, Hq, d, where):
    """Two walks of the shares: at most a few times the clean call's time."""
    b = Batch(spans, Hkv, Hq, d, seed=57)
    cache = b.cache()

    def time():
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        best = math.inf
        for _ in range(4):
            e[0].record()
            b.attn(cache)
            e[1].record()
            torch.cuda.synchronize()
            best = min(best, e[0].elapsed_time(e[1]))
        return best

    clean = time()
    for i, (n, T) in enumerate(spans):
        t = {"first key": 0, "last key": T - 1, "chunk": T - n}[where]
        hit = slice(None) if where == "chunk" else i % d
        stop = T if where == "chunk" else t + 1
        pos = torch.arange(t, stop, device=DEV)
        b.vp[0][b.tables[i].long()[pos // B], :, pos % B, hit] = math.inf
    slow = time()
    assert cache.status() == zp.OK
    print(f"clean {clean * 1e3:.0f} us, {where} {slow * 1e3:.0f} us")
    assert slow < 8 * clean + 0.05


@pytest.mark.parametrize("spans,Hkv,Hq", [([(70, 600)], 1, 4), ([(64, 900)] * 100, 2, 8),
                                          ([(3, 2000)] * 3, 2, 8), ([(5, 700)] * 300, 1, 7)])
@pytest.mark.parametrize("power", [124, 110, 60, -60])
@pytest.mark.parametrize("d", [64, 128])
def test_large_and_small_values(spans, Hkv, Hq, power, d):
    """Values near the largest bf16 number (124: up to about 2^126) and small
    ones, under scores that climb by 12 powers of e along a row (less than what
    makes the kernel change its reference): sums of weights above 1 overflow."""
    b = Batch(spans, Hkv, Hq, d, seed=58, heavy=0.0)
    b.q.copy_(torch.ones_like(b.q))
    for i, (n, T) in enumerate(spans):
        m = -(-T // B)
        blocks = b.tables[i, :m].long()
        t = torch.arange(m * B, device=DEV).view(m, 1, B, 1)
        k = b.kp[0][blocks].float() * 0.05 + t * (12.0 / T / math.sqrt(d))
        b.kp[0][blocks] = torch.where(t < T, k, math.nan).bfloat16()
        b.vp[0][blocks] = (b.vp[0][blocks].float() * 2.0 ** power).bfloat16()
    cache = b.cache()
    b.attn(cache)
    assert cache.status() == zp.OK
    b.check_attn()


@pytest.mark.parametrize("scale", [0.0, 1e-40, -1e-37, 2.0 ** -110])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_near_zero_and_large_scores(scale, d):
    """Scores of up to 1e35: a scale of zero makes every visible key weigh the
    same, a tiny one counts as it is."""
    spans = [(70, 600), (3, 400), (200, 200)]
    b = Batch(spans, 2, 8, d, seed=59, heavy=0.0)
    b.scale = scale
    b.q.mul_(2.0 ** 55)
    b.kp[0].mul_(2.0 ** 55)
    cache = b.cache()
    b.attn(cache)
    assert cache.status() == zp.OK
    b.check_attn()


@pytest.mark.parametrize("spans", [[(64, 900)] * 40, [(5, 4000), (9, 70), (200, 3000)]])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_minus_infinity(spans, d):
    """A request all of whose scores are -infinity gets zeros; in the others such
    keys have no weight."""
    b = Batch(spans, 2, 8, d, seed=60, heavy=0.0)
    b.q.copy_(b.q.abs() + 0.1)
    want = {}
    for i, (n, T) in enumerate(spans):
        a = int(b.starts_np[i])
        blocks = b.tables[i].long()
        k, v = b.rows_of(i)
        gone = torch.arange(0 if i % 3 == 0 else T // 3, T - n if i % 3 else T, device=DEV)
        b.kp[0][blocks[gone // B], :, gone % B] = -math.inf
        if i % 3:  # the 64-bit form on finite keys: far below the others
            k = k.clone()
            k[gone] = -3e4
            want[i] = attn_ref(b.q[a:a + n], k, v, b.scale)
    cache = b.cache()
    b.attn(cache)
    assert cache.status() == zp.OK
    for i, (n, T) in enumerate(spans):
        got = b.out[int(b.starts_np[i]):int(b.starts_np[i + 1])].double()
        if i % 3 == 0:
            assert not bool(got.any()), i
        else:  # keys that have no weight lend none to the bound's spread
            k, v = b.rows_of(i)
            seen = torch.isfinite(k).all(2).all(1).nonzero()[:, 0]
            first = int((seen < T - n).sum())
            _, tol = attn_ref(b.q[int(b.starts_np[i]):int(b.starts_np[i + 1])], k[seen], v[seen],
                              b.scale)
            assert first + n == seen.numel()
            assert bool(((got - want[i][0]).abs() <= tol).all()), i
