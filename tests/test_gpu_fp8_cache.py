"""The 8-bit cache: rows rounded into it, scales, copies of shared tails, and the
attention of single tokens and of chunks over it, against plain 64-bit forms."""
import math

import pytest
import torch

from compressed_paged_kv_gb300 import zp
from tests.fp8_ref import B, E4M3, Batch8

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from compressed_paged_kv_gb300 import _build
    _build.build()
    yield
    torch.cuda.empty_cache()


def _ints(x):
    return torch.tensor(x, dtype=I32, device=DEV)


SPANS = [(1, 1), (5, 21), (16, 16), (0, 40), (17, 33), (3, 100), (30, 47), (1, 32), (2, 17)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("permute", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_append(d, permute, packed):
    b = Batch8(SPANS, Hkv=3, Hq=6, d=d, permute=permute, packed=packed, pad=4, seed=d)
    want = b.expected_append()
    c = b.cache()
    b.append(c)
    assert c.status() == zp.OK
    b.check_append(want)
    b.append(c)  # the same rows again: nothing changes
    assert c.status() == zp.OK
    b.check_append(want)


@pytest.mark.parametrize("spans", [[(1, 16 * i + 1 + i % 16) for i in range(40)],
                                   [(700, 700), (333, 900), (1, 5)],
                                   [(9, 9 + i) for i in range(33)]])
def test_append_batches(spans):
    b = Batch8(spans, Hkv=2, Hq=2, d=128, seed=len(spans))
    want = b.expected_append()
    c = b.cache()
    b.append(c)
    assert c.status() == zp.OK
    b.check_append(want)


@pytest.mark.parametrize("d", [64, 128])
def test_append_one_token_each(d):
    b = Batch8([(1, 1 + 7 * i) for i in range(50)], Hkv=4, Hq=4, d=d, permute=True, packed=False)
    want = b.expected_append()
    c = b.cache()
    c.append_kv(0, b.k_new, b.v_new, b.tables, b.lengths, req_idx=b.req_idx)
    assert c.status() == zp.OK
    b.check_append(want)


def test_append_values_of_every_size():
    """Rows of zeros, of the smallest and the largest numbers, NaN, infinities, borders of
    the scale (448 and the next bf16 numbers)."""
    b = Batch8([(1, 1)] * 12 + [(1, 18)] * 12 + [(16, 16)], Hkv=1, Hq=1, d=64, packed=False)
    rows = [0.0, 448.0, 450.0, 446.0, 2.0 ** -127, 3e38, 1e-30, 7.0, 7.02, math.nan, math.inf, 1.0]
    for x in (b.k_new, b.v_new):
        for i, v in enumerate(rows):
            x[i] *= v if math.isfinite(v) else 1.0
            x[i, 0, 3] = v
            x[12 + i] = x[i]
        x[24:40, 0, ::2] = math.nan
        x[30, 0] = math.nan
        x[31, 0, 5] = -math.inf
    want = b.expected_append()
    c = b.cache()
    b.append(c)
    assert c.status() == zp.OK
    b.check_append(want)


def test_append_token_by_token():
    """Blocks filled one token at a time, their scales growing on the way."""
    b = Batch8([(0, 0)], Hkv=2, Hq=2, d=64, num_blocks=6)
    b.tables = _ints([[3, 1, 4, -1]])
    c = b.cache()
    g = torch.Generator(device=DEV).manual_seed(3)
    for t in range(40):
        b.spans, b.starts_np = [(1, t + 1)], [0, 1]
        b.lengths = _ints([t + 1])
        grow = 2.0 ** (t % 16 / 2.0)
        b.k_new, b.v_new = ((torch.randn(1, 2, 64, generator=g, device=DEV) * grow).bfloat16()
                            for _ in range(2))
        want = b.expected_append()
        c.append_kv(0, b.k_new, b.v_new, b.tables, b.lengths)
        b.check_append(want)
    assert c.status() == zp.OK


def test_append_bad_requests():
    b = Batch8([(3, 20), (4, 30), (2, 40), (5, 50)], Hkv=2, Hq=2, d=64, permute=True)
    want = b.expected_append()
    keep = [x.clone() for x in (b.kp[0].view(torch.uint8), b.ks[0])]
    c = b.cache()
    order = [int(x) for x in b.order]
    bad = b.tables.clone()
    bad[order[1], 1] = 10_000
    c.append_kv_chunk(0, b.k_new, b.v_new, b.starts, bad, b.lengths, req_idx=b.req_idx)
    assert c.status() == zp.ERR_DEVICE_CHECK
    c.append_kv_chunk(0, b.k_new, b.v_new, _ints([0, 3, 2, 9, 14]), b.tables, b.lengths,
                      req_idx=b.req_idx)
    assert c.status() == zp.ERR_DEVICE_CHECK
    one = _ints([99, -1, order[2], order[3]])
    c.append_kv(0, b.k_new[:4].contiguous(), b.v_new[:4].contiguous(), b.tables, b.lengths, req_idx=one)
    assert c.status() == zp.ERR_DEVICE_CHECK
    b.kp[0].view(torch.uint8).copy_(keep[0])
    b.ks[0].copy_(keep[1])
    del want


@pytest.mark.parametrize("d,Hkv,Hq", [(64, 2, 4), (128, 8, 32), (64, 1, 16), (128, 4, 28),
                                      (128, 3, 3), (64, 2, 10)])
def test_decode(d, Hkv, Hq):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 127, 128, 129, 500, 511, 513, 1000, 2047]
    b = Batch8([(1, n) for n in lens], Hkv=Hkv, Hq=Hq, d=d, permute=True, packed=False, seed=Hq)
    c = b.cache()
    b.decode(c)
    assert c.status() == zp.OK
    b.check_attn(split=0.0)


@pytest.mark.parametrize("T", [1, 40, 333, 5000, 30001])
def test_decode_one_request(T):
    """Work split over the length."""
    b = Batch8([(1, T)], Hkv=2, Hq=8, d=128, packed=False, seed=T)
    c = b.cache()
    b.decode(c)
    assert c.status() == zp.OK
    b.check_attn(split=0.0)


def test_decode_zero_length_and_bad_rows():
    b = Batch8([(1, 20), (1, 30), (1, 40), (1, 50)], Hkv=2, Hq=4, d=64, packed=False)
    c = b.cache()
    b.lengths[1] = 0
    b.decode(c)
    assert c.status() == zp.OK
    assert bool((b.out[1] == 0).all())
    b.out[1] = 7.0
    b.check_attn(skip=(1,), split=0.0)
    b.lengths[1] = 10_000
    b.decode(c)
    assert c.status() == zp.ERR_DEVICE_CHECK
    b.lengths[1] = 30
    c.decode(0, b.q.contiguous(), b.tables, b.lengths, b.scale, b.out, req_idx=_ints([0, 9, 2, 3]))
    assert c.status() == zp.ERR_INVALID_ARG
    b.tables[2, 1] = 10_000
    b.decode(c)
    assert c.status() == zp.ERR_DEVICE_CHECK


CHUNKS = [[(1, 1)], [(5, 100)], [(1, 33), (7, 7), (64, 200), (0, 20), (130, 130), (17, 1000)],
          [(3, 50 + 17 * i) for i in range(20)], [(300, 2200), (1, 700)]]


@pytest.mark.parametrize("d,Hkv,Hq", [(64, 2, 4), (128, 2, 8), (64, 1, 16), (128, 4, 28),
                                      (128, 2, 10)])
@pytest.mark.parametrize("spans", CHUNKS, ids=[str(len(x)) for x in CHUNKS])
def test_chunk(spans, d, Hkv, Hq):
    b = Batch8(spans, Hkv=Hkv, Hq=Hq, d=d, permute=len(spans) > 3, pad=3, seed=Hq)
    c = b.cache()
    b.attn(c)
    assert c.status() == zp.OK
    b.check_attn()


@pytest.mark.parametrize("d,Hkv,Hq", [(64, 2, 4), (128, 2, 8), (64, 1, 16), (128, 4, 28)])
@pytest.mark.parametrize("permute", [False, True])
def test_chunk_long_beside_short(d, Hkv, Hq, permute):
    """Long chunks, whose blocks are widened, beside short ones and single tokens."""
    b = Batch8([(1, 300), (900, 1500), (0, 20), (5, 40), (2000, 2000), (1, 1), (17, 500),
                (770, 771)], Hkv=Hkv, Hq=Hq, d=d, permute=permute, pad=5, seed=d + Hq)
    c = b.cache()
    b.attn(c)
    assert c.status() == zp.OK
    b.check_attn()
    first = b.out.clone()
    b.out.fill_(7.0)
    b.attn(c)
    assert torch.equal(first.view(torch.int16), b.out.view(torch.int16))


def test_chunk_more_long_ones_than_the_workspace_holds():
    """Requests past the widened blocks' room go the short ones' way."""
    b = Batch8([(1600, 16000)] * 6 + [(3, 50)], Hkv=8, Hq=8, d=128, seed=5)
    c = b.cache()
    b.attn(c)
    assert c.status() == zp.OK
    b.check_attn()


def test_refusals():
    b = Batch8([(2, 40)], Hkv=2, Hq=4, d=64)
    c = b.cache()
    free, count, refs = _ints([0]), _ints([1]), _ints([0] * b.kp[0].shape[0])
    wq = torch.zeros(1, 1, 4, 8, 64, dtype=torch.bfloat16, device=DEV)
    assert c.compress(b.tables, b.lengths, wq, 2, 8, 0.5, free, count, refs,
                      check=False) == zp.ERR_UNSUPPORTED
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    assert c.compress_prefill(b.tables, b.lengths, wq, 2, 8, 0.5, free, count, refs, ws,
                              check=False) == zp.ERR_UNSUPPORTED
    red = torch.zeros(1, 1, 2, b.tables.shape[1] * B, device=DEV)
    for gram in (False, True):
        assert c.global_redundancy(b.tables, b.lengths, red, check=False,
                                   gram=gram) == zp.ERR_UNSUPPORTED
    out = b.kp[0].view(torch.bfloat16).view(-1)[:2 * 4 * 64].view(2, 4, 64)
    assert c.chunk_attn(0, b.q, b.starts, b.tables, b.lengths, 1.0, out,
                        check=False) == zp.ERR_INVALID_ARG
    with pytest.raises(ValueError):  # bf16 pools with scales
        zp.Cache([b.kp[0].to(torch.bfloat16)], [b.vp[0].to(torch.bfloat16)], 4, 1, 4,
                 k_scales=b.ks, v_scales=b.vs)
    with pytest.raises(ValueError):  # 8-bit pools without
        zp.Cache(b.kp, b.vp, 4, 1, 4)
    with pytest.raises(ValueError):
        zp.Cache(b.kp, b.vp, 4, 1, 4, k_scales=b.ks)
    with pytest.raises(ValueError):
        zp.Cache(b.kp, b.vp, 4, 1, 4, k_scales=[b.ks[0][:-1]], v_scales=b.vs)
    assert b.kp[0].dtype == E4M3
