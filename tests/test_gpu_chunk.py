"""Ragged chunks of new tokens over the paged cache: the K/V append and the
attention, against plain 64-bit forms (tests/chunk_ref.py)."""
import math

import pytest
import torch

from compressed_paged_kv_gb300 import zp
from tests.chunk_ref import B, Batch, attn_ref

pytestmark = pytest.mark.gpu

RAGGED = [(5, 5), (1, 1), (0, 9), (1, 17), (16, 16), (17, 33), (3, 300), (64, 64), (130, 517),
          (0, 0), (33, 700), (1, 1500)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from compressed_paged_kv_gb300 import _build
    _build.build()
    yield
    torch.cuda.empty_cache()


def _bits(t):
    return t.contiguous().view(torch.int16)


# ------------------------------------------------------------------- append

@pytest.mark.parametrize("Hkv,Hq,d", [(2, 4, 64), (8, 32, 128), (1, 1, 128), (3, 3, 64)])
@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("spans", [RAGGED, [(1, 1)], [(40, 40)], [(1, 5)] * 70 + [(9, 20)] * 3,
                                   [(2, 16)] * 1100])
def test_append_writes_only_its_slots(Hkv, Hq, d, packed, spans):
    b = Batch(spans, Hkv, Hq, d, seed=1, permute=True, pad=3, packed=packed, L=2, layer=1)
    cache = b.cache()
    want = []
    for pools, new in ((b.kp, b.k_new), (b.vp, b.v_new)):
        w = [p.clone() for p in pools]
        for i, (n, T) in enumerate(spans):
            a = int(b.starts_np[i])
            pos = torch.arange(T - n, T, device=b.dev)
            blk = b.tables[b.order[i]].long()[pos // B]
            w[1][blk, :, pos % B] = new[a:a + n]
        want.append(w)
    b.append(cache)
    assert cache.status() == zp.OK
    for got, w in zip((b.kp, b.vp), want):
        for x, y in zip(got, w):
            assert torch.equal(_bits(x), _bits(y))


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("Hkv,Hq,d", [(2, 4, 64), (8, 32, 128), (1, 1, 128), (2, 32, 64),
                                      (1, 7, 128), (2, 10, 128), (3, 3, 64)])
@pytest.mark.parametrize("packed", [True, False])
def test_ragged_batch(Hkv, Hq, d, packed):
    b = Batch(RAGGED, Hkv, Hq, d, seed=2, permute=True, pad=5, packed=packed, L=2, layer=1)
    cache = b.cache()
    b.attn(cache)
    assert cache.status() == zp.OK
    b.check_attn()


@pytest.mark.parametrize("n,T", [(1, 1), (1, 2), (2, 2), (1, 16), (7, 127), (7, 128), (7, 129),
                                 (31, 31), (32, 32), (33, 33), (63, 255), (64, 256), (65, 257),
                                 (128, 128), (129, 129), (257, 400), (513, 513), (1, 5000),
                                 (40, 9000)])
@pytest.mark.parametrize("Hkv,Hq,d", [(2, 8, 128), (1, 2, 64)])
def test_one_request(n, T, Hkv, Hq, d):
    b = Batch([(n, T)], Hkv, Hq, d, seed=n * 10007 + T)
    cache = b.cache()
    b.attn(cache)
    assert cache.status() == zp.OK
    b.check_attn()


@pytest.mark.parametrize("spans", [[(2000, 2000)], [(1500, 4000), (1, 33), (1, 4000)],
                                   [(5, 2040)] * 8, [(1 + i % 9, 100 + 7 * i) for i in range(300)],
                                   [(1, 1 + i % 40) for i in range(1200)],
                                   [(300, 300 + 40 * i) for i in range(12)]])
def test_larger_batches(spans):
    b = Batch(spans, 2, 8, 128, seed=3)
    cache = b.cache()
    b.attn(cache)
    assert cache.status() == zp.OK
    b.check_attn()


@pytest.mark.parametrize("rise", [1, -1])
def test_scores_that_climb_or_fall(rise):
    """Keys whose scores grow (or shrink) by a few units every key: the running
    maximum moves all along the row (or never again)."""
    b = Batch([(150, 1500), (3, 1200)], 1, 4, 128, seed=4, heavy=0.0)
    b.q.copy_(torch.ones_like(b.q))
    for i, (n, T) in enumerate(b.spans):
        m = -(-T // B)
        blocks = b.tables[i, :m].long()
        t = torch.arange(m * B, device=b.dev).view(m, 1, B, 1)
        step = t if rise > 0 else T - t
        k = b.kp[0][blocks].float() * 0.05 + step * (2.0 / math.sqrt(128))
        b.kp[0][blocks] = torch.where(t < T, k, math.nan).bfloat16()
    cache = b.cache()
    b.attn(cache)
    assert cache.status() == zp.OK
    b.check_attn()


@pytest.mark.parametrize("scale", [-0.09, 0.0, 1e-6, 0.7])
@pytest.mark.parametrize("d", [64, 128])
def test_other_scales(scale, d):
    b = Batch([(70, 600), (3, 400), (200, 200)], 2, 8, d, seed=15, heavy=0.0)
    b.scale = scale
    cache = b.cache()
    b.attn(cache)
    assert cache.status() == zp.OK
    b.check_attn()


def test_hidden_tokens_do_not_reach_a_row():
    """Not-finite keys and values at positions a token does not see leave its
    output within the bound of the clean 64-bit result (rows that shared a tile
    with them are computed again in another order of additions)."""
    spans = [(40, 200), (130, 130), (300, 1000), (9, 515)]
    b = Batch(spans, 2, 8, 128, seed=5)
    cache = b.cache()
    want = []
    for i, (n, T) in enumerate(spans):
        k, v = b.rows_of(i)
        a = int(b.starts_np[i])
        want.append(attn_ref(b.q[a:a + n], k, v, b.scale))
    for i, (n, T) in enumerate(spans):
        cut = T - n // 2  # positions from here on are poisoned
        for pool, bad in ((b.kp[0], math.nan), (b.vp[0], math.inf)):
            pos = torch.arange(cut, T, device=b.dev)
            blk = b.tables[i].long()[pos // B]
            pool[blk, :, pos % B] = bad
    b.attn(cache)
    assert cache.status() == zp.OK
    for i, (n, T) in enumerate(spans):
        a = int(b.starts_np[i])
        m = n - n // 2
        err = (b.out[a:a + m].double() - want[i][0][:m]).abs()
        assert bool((err <= want[i][1][:m]).all()), i
        assert not bool(torch.isfinite(b.out[a + m:a + n]).any()), i


@pytest.mark.parametrize("t", [0, 100, 255, 299])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_visible_value_that_is_not_finite(t, bad):
    b = Batch([(60, 300)], 1, 4, 64, seed=6, heavy=0.0)
    cache = b.cache()
    k, v = b.rows_of(0)
    want, tol = attn_ref(b.q, k, v, b.scale)
    b.vp[0][b.tables[0, t // B].long(), 0, t % B, 5] = bad
    b.attn(cache)
    assert cache.status() == zp.OK
    hit = torch.zeros(60, 4, 64, dtype=torch.bool, device=b.dev)
    hit[max(0, t - 240):, :, 5] = True
    assert not bool(torch.isfinite(b.out[hit]).any())
    assert bool(((b.out.double() - want).abs() <= tol)[~hit].all())


def test_query_that_is_not_finite_stays_in_its_row():
    b = Batch([(70, 90), (3, 40)], 2, 4, 64, seed=7)
    cache = b.cache()
    b.attn(cache)
    clean = b.out.clone()
    b.q[11, 2, 9] = math.nan
    b.attn(cache)
    assert bool(torch.isnan(b.out[11, 2]).all())
    keep = torch.ones_like(clean, dtype=torch.bool)
    keep[11, 2] = False
    assert torch.equal(_bits(b.out[keep]), _bits(clean[keep]))


def test_single_tokens_match_the_decode_attention():
    spans = [(1, T) for T in (1, 15, 16, 17, 100, 1000, 2040)]
    b = Batch(spans, 8, 32, 128, seed=8, permute=True, packed=False)
    cache = b.cache()
    b.attn(cache)
    dec = torch.empty_like(b.out)
    cache.decode(0, b.q, b.tables, b.lengths, b.scale, dec, req_idx=b.req_idx)
    assert cache.status() == zp.OK
    b.check_attn()
    for i in range(len(spans)):  # both within the bound of the same 64-bit result
        k, v = b.rows_of(i)
        want, tol = attn_ref(b.q[i:i + 1], k, v, b.scale)
        assert bool(((dec[i:i + 1].double() - want).abs() <= tol).all())


def test_same_row_twice_and_a_repeat_are_the_same():
    b = Batch([(20, 500), (9, 64)], 2, 8, 128, seed=9)
    b.req_idx = torch.tensor([0, 0], dtype=torch.int32, device=b.dev)
    b.q[20:29] = b.q[11:20].clone()  # the last nine tokens of row 0, twice
    cache = b.cache()
    b.attn(cache)
    assert cache.status() == zp.OK
    first = b.out.clone()
    k, v = b.rows_of(0)
    want, tol = attn_ref(b.q[:20], k, v, b.scale)
    assert bool(((b.out[:20].double() - want).abs() <= tol).all())
    assert bool(((b.out[20:29].double() - want[11:]).abs() <= tol[11:]).all())
    for _ in range(3):
        b.attn(cache)
        assert torch.equal(_bits(b.out), _bits(first))


def test_offsets_past_32_bits():
    """Pools of more than 2^31 elements, all blocks in use near their end."""
    nb = (1 << 31) // (8 * B * 128) + 600
    b = Batch([(50, 900), (1, 2000), (200, 333)], 8, 32, 128, seed=10, num_blocks=nb,
              first_block=nb - 300)
    cache = b.cache()
    b.append(cache)
    b.attn(cache)
    assert cache.status() == zp.OK
    for i, (n, T) in enumerate(b.spans):
        k, v = b.rows_of(i)
        a = int(b.starts_np[i])
        assert torch.equal(_bits(k[T - n:]), _bits(b.k_new[a:a + n]))
        assert torch.equal(_bits(v[T - n:]), _bits(b.v_new[a:a + n]))
    b.check_attn()


def test_another_stream_and_a_slice_of_the_requests():
    b = Batch([(30, 200), (4, 100), (90, 90)], 2, 8, 128, seed=11)
    cache = b.cache()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.append_kv_chunk(0, b.k_new, b.v_new, b.starts, b.tables, b.lengths)
        b.attn(cache)
    side.synchronize()
    assert cache.status(stream=side) == zp.OK
    b.check_attn()


def test_captured_call_follows_the_device_arrays():
    """One captured append and attention, replayed on other chunk offsets and
    lengths (a padded batch): equal to the eager calls on them, bit for bit."""
    full = [(64, 900), (40, 333), (100, 700), (1, 50)]
    b = Batch(full, 2, 8, 128, seed=12)
    cache = b.cache()
    b.append(cache)
    b.attn(cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.append(cache)
        b.attn(cache)
    for step, spans in enumerate([full, [(5, 841), (6, 299), (0, 0), (1, 50)],
                                  [(1, 1), (0, 300), (100, 700), (0, 0)], [(0, 0)] * 4]):
        counts = [n for n, _ in spans]
        starts = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32)
        b.starts.copy_(starts)
        b.lengths.copy_(torch.tensor([T for _, T in spans], dtype=torch.int32))
        b.spans, b.starts_np = spans, starts.numpy()
        b.out.fill_(7.0)
        b.append(cache)
        b.attn(cache)
        eager = b.out.clone()
        b.out.fill_(7.0)
        graph.replay()
        assert cache.status() == zp.OK
        assert torch.equal(_bits(b.out), _bits(eager)), step
        b.check_attn()


# ----------------------------------------------------------------- refusals

def test_refused_on_the_host():
    b = Batch([(8, 40), (3, 20)], 2, 4, 64, seed=13, packed=False)
    cache = b.cache()
    s = torch.cuda.current_stream().cuda_stream

    def attn(layer=0, q=None, qs=256, total=11, stride=None, rows=2, R=2, scale=0.125, out=None,
             starts=None):
        return zp.zp_paged_chunk_attn(
            cache.handle, layer, b.q.data_ptr() if q is None else q, qs,
            b.starts.data_ptr() if starts is None else starts, total, b.tables.data_ptr(),
            b.tables.shape[1] if stride is None else stride, rows, b.lengths.data_ptr(), 0, R,
            scale, b.out.data_ptr() if out is None else out, s)

    def append(layer=0, k=None, ks=128, vs=128, total=11, R=2):
        return zp.zp_append_kv_chunk(
            cache.handle, layer, b.k_new.data_ptr() if k is None else k, ks, b.v_new.data_ptr(),
            vs, b.starts.data_ptr(), total, b.tables.data_ptr(), b.tables.shape[1], 2,
            b.lengths.data_ptr(), 0, R, s)

    before = [b.kp[0].clone(), b.vp[0].clone()]
    bad = zp.ERR_INVALID_ARG
    assert attn(layer=1) == bad and attn(layer=-1) == bad
    assert attn(q=b.q.data_ptr() + 2) == bad and attn(out=b.out.data_ptr() + 16) == bad
    assert attn(qs=255) == bad and attn(qs=260) == bad and attn(qs=-256) == bad
    assert attn(total=-1) == bad and attn(R=-1) == bad and attn(R=3) == bad
    assert attn(stride=0) == bad and attn(rows=0) == bad and attn(starts=0) == bad
    assert attn(scale=math.inf) == bad and attn(scale=math.nan) == bad
    assert attn(stride=1 << 27) == zp.ERR_UNSUPPORTED
    assert attn(R=0) == zp.OK and attn(total=0) == zp.OK
    assert append(layer=1) == bad and append(k=b.k_new.data_ptr() + 8) == bad
    assert append(ks=120) == bad and append(vs=132) == bad and append(total=-1) == bad
    assert append(R=0) == zp.OK and append(total=0) == zp.OK
    for f in (lambda: cache.chunk_attn(0, b.q[:, :3], b.starts, b.tables, b.lengths, 1.0, b.out),
              lambda: cache.chunk_attn(0, b.q.float(), b.starts, b.tables, b.lengths, 1.0, b.out),
              lambda: cache.chunk_attn(0, b.q.transpose(0, 1), b.starts, b.tables, b.lengths, 1.0,
                                       b.out),
              lambda: cache.chunk_attn(0, b.q, b.starts.long(), b.tables, b.lengths, 1.0, b.out),
              lambda: cache.chunk_attn(0, b.q, b.starts, b.tables, b.lengths, 1.0, b.out[:5]),
              lambda: cache.append_kv_chunk(0, b.k_new, b.v_new[:3], b.starts, b.tables,
                                            b.lengths)):
        with pytest.raises(ValueError):
            f()
    assert cache.status() == zp.OK
    assert bool((b.out == 7.0).all())
    assert torch.equal(_bits(before[0]), _bits(b.kp[0]))
    assert torch.equal(_bits(before[1]), _bits(b.vp[0]))


@pytest.mark.parametrize("what", ["row", "negative_row", "short_length", "long_length",
                                  "offsets_fall", "offsets_past_total", "block", "negative_block"])
def test_refused_on_the_device(what):
    """A request that does not fit is recorded and skipped; the others are
    computed."""
    b = Batch([(8, 40), (30, 200), (3, 20)], 2, 4, 64, seed=14)
    b.req_idx = torch.arange(3, dtype=torch.int32, device=b.dev)
    cache = b.cache()
    skip = {1}
    if what == "row":
        b.req_idx[1] = 3
    elif what == "negative_row":
        b.req_idx[1] = -1
    elif what == "short_length":
        b.lengths[1] = 29
    elif what == "long_length":
        b.lengths[1] = b.tables.shape[1] * B + 1
    elif what == "offsets_fall":
        b.starts[2] = 5  # chunk 1 is [8, 5), chunk 2 [5, 41) is longer than its row
        skip = {1, 2}
    elif what == "offsets_past_total":
        b.starts[3] = 42
        skip = {2}
    elif what == "block":
        b.tables[1, 11] = b.kp[0].shape[0]
    else:
        b.tables[1, 11] = -1
    before = [b.kp[0].clone(), b.vp[0].clone()]
    good = [i for i in range(3) if i not in skip]
    spans = b.spans
    b.append(cache)
    assert cache.status() == zp.ERR_DEVICE_CHECK
    for pool, new, old in ((b.kp[0], b.k_new, before[0]), (b.vp[0], b.v_new, before[1])):
        for i in good:
            n, T = spans[i]
            a = int(b.starts_np[i])
            pos = torch.arange(T - n, T, device=b.dev)
            blk = b.tables[i].long()[pos // B]
            old[blk, :, pos % B] = new[a:a + n]
        if what == "offsets_fall":  # rows 5 .. 7 are claimed by two chunks
            pos = torch.arange(37, 40, device=b.dev)
            blk = b.tables[0].long()[pos // B]
            old[blk, :, pos % B] = pool[blk, :, pos % B]
        if "block" in what:  # the chunk's tokens in its other blocks are written
            pos = torch.arange(170, 200, device=b.dev)
            pos = pos[pos // B != 11]
            blk = b.tables[1].long()[pos // B]
            old[blk, :, pos % B] = new[8 + pos - 170]
        assert torch.equal(_bits(pool), _bits(old))
    b.attn(cache)
    assert cache.status() == zp.ERR_DEVICE_CHECK
    if "block" in what:
        b.out[8:38] = 7.0  # undefined there
    b.check_attn(skip=skip)
    assert cache.status() == zp.OK
