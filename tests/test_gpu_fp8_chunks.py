"""Chunks over an 8-bit cache by the number of their query rows: few (a kernel of their own), one
tile in large batches (kv heads two at a time), many; NaN among keys and values; requests that
are none."""
import math

import pytest
import torch

from compressed_paged_kv_gb300 import zp
from tests.fp8_ref import Batch8, attn_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN8 = 0x7f


@pytest.fixture(scope="module", autouse=True)
def _built():
    from compressed_paged_kv_gb300 import _build
    _build.build()
    yield
    torch.cuda.empty_cache()


def run(b, **kw):
    c = b.cache()
    b.attn(c, **kw)
    assert c.status() == zp.OK
    return c


SHAPES = [(64, 2, 2), (64, 3, 6), (128, 2, 8), (64, 1, 5), (128, 1, 7), (128, 2, 16), (64, 1, 16)]


@pytest.mark.parametrize("d,Hkv,Hq", SHAPES)
@pytest.mark.parametrize("rows", [8, 16, 20, 24])
def test_few_rows(d, Hkv, Hq, rows):
    """Every length around the ends of blocks, pairs of them and a warp's turn; chunks as long as
    the row itself, and up to `rows` rows of queries."""
    most = max(1, rows // (Hq // Hkv))
    spans = []
    for i, T in enumerate([1, 2, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 127, 128, 129, 130, 255, 257,
                           300, 511, 513, 1000]):
        spans += [(min(T, most), T), (min(T, 1 + i % most), T)]
    b = Batch8(spans, Hkv=Hkv, Hq=Hq, d=d, permute=True, pad=3, seed=rows)
    run(b)
    b.check_attn()


@pytest.mark.parametrize("R,n,T", [(1, 1, 1), (1, 2, 40), (1, 4, 2000), (1, 5, 4000), (2, 3, 2500),
                                   (5, 4, 700), (1, 4, 8000)])
def test_few_rows_over_splits(R, n, T):
    b = Batch8([(n, T + 3 * i) for i in range(R)], Hkv=4, Hq=16, d=128, seed=T)
    run(b)
    b.check_attn()


def test_a_table_much_wider_than_the_row():
    """The splits share out the row, not the table."""
    b = Batch8([(4, 1000), (1, 3)], Hkv=2, Hq=8, d=64)
    wide = torch.full((2, 900), -1, dtype=torch.int32, device=DEV)
    wide[:, :b.tables.shape[1]] = b.tables
    b.tables = wide
    run(b)
    b.check_attn()


@pytest.mark.parametrize("spans", [
    [(4, 300)] * 30 + [(60, 700)] + [(0, 50)] * 3,             # one for the other kernel
    [(0, 0), (5, 900), (0, 7), (1, 1), (7, 7), (3, 129)] * 8,  # some of them just above
    [(1, 200)] * 40 + [(200, 200)],
    [(6, 1000)] * 3 + [(0, 16)] * 20,
])
def test_both_kernels(spans):
    b = Batch8(spans, Hkv=2, Hq=8, d=128, permute=True, seed=len(spans))
    run(b)
    b.check_attn()


@pytest.mark.parametrize("d,Hkv,G", [(64, 8, 4), (128, 8, 4), (128, 4, 8), (64, 5, 4)])
@pytest.mark.parametrize("long", [False, True])
def test_one_tile_each_of_a_large_batch(d, Hkv, G, long):
    """Above 20 rows, up to a tile of 128: kv heads two at a time where their number is even."""
    spans = [(6 + i % (128 // G - 5), 6 + i % (128 // G - 5) + 11 * i) for i in range(78)]
    if long:  # and requests of more than a tile beside them
        spans[3], spans[40] = (300, 800), (77, 77)
    b = Batch8(spans, Hkv=Hkv, Hq=Hkv * G, d=d, permute=True, seed=G)
    run(b)
    b.check_attn()


# (spans, Hkv, Hq): few rows; one tile; heads by two; more than a tile; widened to bf16
NANS = [([(4, 70), (3, 33), (2, 200)], 2, 8),
        ([(5, 40), (4, 513)], 1, 4),
        ([(1, 90)] * 3, 2, 2),
        ([(20, 70), (12, 300)], 2, 8),
        ([(9, 150 + i) for i in range(80)], 4, 16),
        ([(90, 300), (200, 200)], 2, 8),
        ([(400, 700)], 2, 8)]


@pytest.mark.parametrize("spans,Hkv,Hq", NANS, ids=[str(i) for i in range(len(NANS))])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_values(spans, Hkv, Hq, d):
    """A value that is NaN: NaN in its dim for the tokens that see its key, nothing for those
    before it."""
    b = Batch8(spans, Hkv=Hkv, Hq=Hq, d=d, seed=d)
    G = Hq // Hkv
    pool = b.vp[0].view(torch.uint8)
    put = []  # (request, key, head, dim)
    for i in range(0, len(spans), max(1, len(spans) // 4)):
        n, T = spans[i]
        for t, h, e in ((T - 1, 0, 3), (T - n // 2 - 1, Hkv - 1, d - 1), (T - n, 0, 8),
                        (max(0, T - n - 1), Hkv - 1, 17), (0, 0, 40)):
            put.append((i, t, h, e))
    put += put[:2]
    for i, t, h, e in put:
        blk = int(b.tables[b.order[i], t // 16])
        pool[blk, h, t % 16, e] = NAN8 | (0x80 if t & 1 else 0)
    run(b)
    for i, (n, T) in enumerate(spans):
        a = int(b.starts_np[i])
        k, v = b.rows_of(i)
        want, tol = attn_ref(b.q[a:a + n], k, v.nan_to_num(0.0), b.scale, 2.0 ** -17,
                             2.0 ** -8 if n * G >= 1536 else 2.0 ** -11)
        got = b.out[a:a + n].double()
        seen = torch.zeros(n, Hq, d, dtype=torch.bool, device=DEV)
        for j, t, h, e in put:
            if j == i:
                seen[max(0, t - (T - n)):, h * G:(h + 1) * G, e] = True
        assert torch.equal(torch.isnan(got), seen), i
        assert bool((((got - want).abs() <= tol) | seen).all()), i


@pytest.mark.parametrize("spans,Hkv,Hq", NANS, ids=[str(i) for i in range(len(NANS))])
def test_nan_keys_and_queries(spans, Hkv, Hq):
    """NaN in a key: NaN for the tokens that see it.  NaN or an infinity in a row of q: NaN for
    that row alone (an infinity makes it NaN or a limit; never a wrong number beside it)."""
    d, G = 64, Hq // Hkv
    b = Batch8(spans, Hkv=Hkv, Hq=Hq, d=d, seed=7)
    n, T = spans[-1]
    t, i = T - (n + 1) // 2, len(spans) - 1
    blk = int(b.tables[b.order[i], t // 16])
    b.kp[0].view(torch.uint8)[blk, Hkv - 1, t % 16, 5] = NAN8
    b.q[0, 0, 9] = math.nan
    b.q[0, Hq - 1, 60] = math.inf
    run(b)
    for j, (n, T) in enumerate(spans):
        a = int(b.starts_np[j])
        k, v = b.rows_of(j)
        want, tol = attn_ref(b.q[a:a + n].nan_to_num(0.0, 0.0, 0.0), k.nan_to_num(0.0), v, b.scale,
                             2.0 ** -17, 2.0 ** -8 if n * G >= 1536 else 2.0 ** -11)
        got = b.out[a:a + n].double()
        bad = torch.zeros(n, Hq, d, dtype=torch.bool, device=DEV)
        if j == i:
            bad[t - (T - n):, (Hkv - 1) * G:] = True
        if j == 0:
            bad[0, 0] = True
        free = bad.clone()
        if j == 0:
            free[0, Hq - 1] = True
        assert bool(torch.isnan(got)[bad].all()), j
        assert bool((((got - want).abs() <= tol) | free).all()), j


@pytest.mark.parametrize("n", [3, 30])
def test_requests_that_are_none(n):
    """Rows out of the table, lengths below the chunk's and past the table, block ids out of the
    pool: reported, the other requests' rows right, the refused ones' as they were."""
    b = Batch8([(n, 100 + 20 * i) for i in range(8)], Hkv=2, Hq=8, d=64, permute=True)
    b.req_idx[1] = 99
    b.req_idx[2] = -1
    b.lengths[int(b.order[4])] = n - 1
    b.lengths[int(b.order[5])] = b.tables.shape[1] * 16 + 1
    c = b.cache()
    b.attn(c)
    assert c.status() == zp.ERR_DEVICE_CHECK
    b.check_attn(skip=(1, 2, 4, 5))
    b.out.fill_(7.0)
    b.tables[int(b.order[6]), 2] = b.kp[0].shape[0]
    b.tables[int(b.order[7]), 0] = -7
    c = b.cache()
    b.attn(c)
    assert c.status() == zp.ERR_DEVICE_CHECK
    for i in (6, 7):
        a = int(b.starts_np[i])
        b.out[a:a + n] = 7.0
    b.check_attn(skip=(1, 2, 4, 5, 6, 7))


@pytest.mark.parametrize("n", [2, 30])
def test_offsets_that_are_none(n):
    """Offsets past the rows, falling ones and negative ones."""
    b = Batch8([(n, 60)] * 6, Hkv=2, Hq=8, d=64)
    s = b.starts_np.copy()
    s[3] = b.total + 5  # request 2 ends past the rows, request 3 falls
    b.starts = torch.from_numpy(s).to(DEV)
    c = b.cache()
    b.attn(c)
    assert c.status() == zp.ERR_DEVICE_CHECK
    b.check_attn(skip=(2, 3))


MIXES = [[(4, 70), (3, 200), (1, 33)], [(20, 300), (30, 40)], [(9, 130 + i) for i in range(80)],
         [(100, 500), (60, 60)], [(400, 700)]]


@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-30, 2.0])
@pytest.mark.parametrize("spans", MIXES, ids=[str(i) for i in range(len(MIXES))])
def test_scales_of_the_logits(spans, scale):
    b = Batch8(spans, Hkv=4, Hq=16, d=64, seed=5)
    b.scale = scale
    run(b)
    b.check_attn()


@pytest.mark.parametrize("power", [-90, 90])
@pytest.mark.parametrize("spans", MIXES, ids=[str(i) for i in range(len(MIXES))])
def test_queries_of_every_size(spans, power):
    """Rows of q from 2^-90 to 2^90, taken back by the scale; rows of zeros."""
    b = Batch8(spans, Hkv=2, Hq=8, d=128, seed=6, packed=False)
    b.q = (b.q.float() * 2.0 ** power).bfloat16()
    b.q[::5] = 0
    b.scale *= 2.0 ** -power
    run(b)
    b.check_attn()


@pytest.mark.parametrize("spans", MIXES, ids=[str(i) for i in range(len(MIXES))])
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_every_size(spans, d):
    """Blocks of values whose scales lie up to 2^50 apart."""
    b = Batch8(spans, Hkv=2, Hq=8, d=d, seed=8, spread=50)
    run(b)
    b.check_attn()


@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens_of_every_size(d):
    b = Batch8([(1, 20 * i + 1) for i in range(40)], Hkv=2, Hq=8, d=d, seed=8, spread=50,
               packed=False)
    b.scale = -0.3
    b.decode(b.cache())
    b.check_attn(split=0.0)


@pytest.mark.parametrize("n,scale", [(1, 1e33), (1, -1e33), (4, 1e33), (4, -1e33), (30, 1e4),
                                     (30, -1e4), (400, 1e4), (400, -1e4)])
def test_the_first_key_alone_at_any_score(n, scale):
    """The first token of a prompt sees its own key, whose weight is 1 however low its score is.
    (Chunks of many rows take p in one step from a product and the maximum, whose rounding
    is within the 2 that fp16 leaves above 2^15 for scores below 2^23 in base 2: the header
    allows 2^20, and |q . k| is below 2^6 here.)"""
    b = Batch8([(n, n)] * 3, Hkv=2, Hq=8, d=64, seed=4, packed=False)
    b.scale = scale
    c = run(b)
    if n == 1:
        want = b.out.clone()
        b.out.fill_(7.0)
        b.decode(c)
        assert c.status() == zp.OK and torch.equal(b.out, want)
    for i in range(3):
        _, v = b.rows_of(i)
        got = b.out[int(b.starts_np[i])].double().view(2, 4, 64)
        # p v / p: p rounded for the product (2^-11 in fp16, 2^-8 in bf16) and not in the sum, then
        # the result (2^-8); twice the fp32 roundings of both
        rel = 2.0 ** -8 + (2.0 ** -8 if 4 * n >= 1536 else 2.0 ** -11) * (1 + 2.0 ** -8) + 2.0 ** -20
        assert bool(((got - v[0][:, None]).abs() <= v[0][:, None].abs() * rel).all())


@pytest.mark.parametrize("d", [64, 128])
def test_short_items_before_long_ones(d):
    """Many items a CTA of one key tile, which one stream has no part in, and of several, odd and
    even numbers of them, single ones, pairs and two heads at a time."""
    spans = []
    for i in range(240):
        n = 6 + i % 20
        spans.append((n, n + (i * 37 % 90 if i % 3 else 130 + i * 53 % 900)))
    spans[50] = spans[170] = (70, 500)
    for Hkv in (3, 2):
        b = Batch8(spans, Hkv=Hkv, Hq=4 * Hkv, d=d, seed=Hkv)
        c = run(b)
        b.check_attn()
        want = b.out.clone()
        for _ in range(5):
            b.out.fill_(7.0)
            b.attn(c)
            assert torch.equal(b.out, want)
