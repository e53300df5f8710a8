"""Verification of drafted tokens against the plain 64-bit form: accepted
counts and next tokens are whole numbers and equal."""
import math

import numpy as np
import pytest
import torch

from compressed_paged_kv_gb300 import zp
from tests.chunk_ref import verify_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from compressed_paged_kv_gb300 import _build
    _build.build()
    yield
    torch.cuda.empty_cache()


def _cache(R):
    pool = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device=DEV)
    return zp.Cache([pool], [pool.clone()], 1, max_requests=R, max_blocks_per_req=2)


class Draft:
    def __init__(self, counts, V, dtype=torch.float32, draft=True, pad=0, offset=0, seed=0,
                 noise=0.4, width=3.0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.counts = counts
        total, R = sum(counts), len(counts)
        self.starts = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)

        def rows():  # rows of V probabilities, V + pad apart, `offset` elements into a buffer
            buf = torch.full((total * (V + pad) + offset + 8,), math.nan, dtype=dtype, device=DEV)
            return buf[offset:offset + total * (V + pad)].view(total, V + pad)[:, :V]

        logits = width * torch.randn(total, V, generator=g, device=DEV)
        noisy = logits + noise * torch.randn(total, V, generator=g, device=DEV)
        self.p, self.q = rows(), None
        self.p.copy_(torch.softmax(logits, 1))
        q = torch.softmax(noisy, 1)
        if draft:
            self.q = rows()
            self.q.copy_(q)
        picked = torch.multinomial(q, 1, generator=g)[:, 0] if draft else noisy.argmax(1)
        self.tokens = torch.full((total,), -5, dtype=torch.int32, device=DEV)
        for i, n in enumerate(counts):  # token 0 of a chunk is not read
            a = int(self.starts[i])
            if n > 1:
                self.tokens[a + 1:a + n] = picked[a:a + n - 1].int()
        self.accept_u = torch.rand(total, generator=g, device=DEV)
        self.sample_u = torch.rand(R, generator=g, device=DEV)
        self.accepted = torch.full((R,), -7, dtype=torch.int32, device=DEV)
        self.next = torch.full((R,), -7, dtype=torch.int32, device=DEV)

    def run(self, cache, **kw):
        return cache.verify_draft(self.tokens, self.starts, self.p, self.accept_u, self.sample_u,
                                  self.accepted, self.next, draft_probs=self.q, **kw)

    def check(self):
        acc, nxt = verify_ref(self.tokens.cpu().numpy(), self.starts.cpu().numpy(),
                              self.p.cpu().double().numpy(),
                              None if self.q is None else self.q.cpu().double().numpy(),
                              self.accept_u.cpu().numpy(), self.sample_u.cpu().numpy())
        assert self.accepted.tolist() == [-7 if x is None else x for x in acc]
        assert self.next.tolist() == [-7 if x is None else x for x in nxt]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V,pad,offset", [(1, 0, 0), (2, 1, 0), (7, 0, 1), (31, 2, 3), (1000, 0, 0),
                                          (1000, 24, 5), (4097, 0, 0), (32000, 0, 0),
                                          (50257, 0, 1), (128001, 7, 0)])
def test_against_64_bits(dtype, draft, V, pad, offset):
    counts = [5, 1, 0, 2, 9, 3, 1, 4]
    d = Draft(counts, V, dtype, draft, pad, offset, seed=V + pad)
    cache = _cache(len(counts))
    d.run(cache)
    assert cache.status() == zp.OK
    d.check()


@pytest.mark.parametrize("draft", [True, False])
def test_a_large_batch(draft):
    counts = [1 + i % 7 for i in range(300)]
    d = Draft(counts, 2003, draft=draft, seed=5)
    cache = _cache(300)
    d.run(cache)
    assert cache.status() == zp.OK
    d.check()
    first = d.accepted.clone(), d.next.clone()
    for _ in range(3):
        d.run(cache)
        assert torch.equal(d.accepted, first[0]) and torch.equal(d.next, first[1])


def test_flat_rows_and_extreme_numbers():
    """Nearly equal probabilities (borders as close as they get), sample_u at 0
    and just below 1."""
    counts = [2] * 12
    d = Draft(counts, 151936, seed=6, width=0.01, noise=0.01)
    top = 1.0 - 2.0 ** -24
    d.sample_u[:4] = torch.tensor([0.0, top, 0.0, top])
    d.accept_u[0:24:2] = torch.tensor([0.0, 0.0, top, top] + [0.5] * 8)
    cache = _cache(12)
    d.run(cache)
    assert cache.status() == zp.OK
    d.check()


def test_greedy_rows():
    """One-hot target rows: a drafted token is accepted exactly when it is the
    target's, and the next token is the target's."""
    V, counts = 1003, [6] * 9
    d = Draft(counts, V, draft=False, seed=7)
    best = torch.randint(0, V, (54,), device=DEV)
    d.p.zero_()
    d.p[torch.arange(54, device=DEV), best] = 1.0
    for i in range(9):  # the first i % 6 drafted tokens are right, then one is wrong
        for j in range(5):
            d.tokens[6 * i + j + 1] = (best[6 * i + j] + (1 if j == i % 6 else 0)) % V
    cache = _cache(9)
    d.run(cache)
    assert cache.status() == zp.OK
    d.check()
    assert d.accepted.tolist() == [min(i % 6, 5) for i in range(9)]
    assert d.next.tolist() == [int(best[6 * i + min(i % 6, 5)]) for i in range(9)]


def test_nothing_left_of_a_rejected_row():
    """p <= q everywhere: drawn from p; NaN, negative and infinite weights count
    as zero; a row of zeros is recorded."""
    V = 40
    d = Draft([2, 2, 1, 1, 2], V, seed=8)
    d.p[0] = 0.5 * d.q[0]
    d.accept_u[0] = 0.9                      # rejected, nothing left
    d.q[2] = 0.0
    d.p[2] = 0.0                             # no weight at all
    d.p[4, 3], d.p[4, 9], d.p[4, 11] = math.nan, -1.0, math.inf
    d.p[5] = 0.0
    d.q[6] = math.nan                        # u * NaN < p is false: rejected, drawn from p
    cache = _cache(5)
    d.run(cache)
    assert cache.status() == zp.ERR_DEVICE_CHECK  # requests 1 and 3
    d.check()
    assert d.next[1] == -1 and d.next[3] == -1 and int(d.next[0]) >= 0 and int(d.next[4]) >= 0


def test_kept_tokens_follow_the_target():
    """Over a grid of drafted tokens and random numbers, the first token kept
    has the target's frequencies: sum_x q(x) [accepted x or resampled] = p."""
    V, n = 5, 48
    p = torch.tensor([0.42, 0.03, 0.25, 0.3, 0.0], device=DEV)
    q = torch.tensor([0.2, 0.4, 0.3, 0.1, 0.0], device=DEV)
    R = 4 * n * n
    grid = ((torch.arange(n, device=DEV) + 0.5) / n)
    x = torch.arange(4, device=DEV).repeat_interleave(n * n)
    counts = torch.arange(R + 1, device=DEV, dtype=torch.int32) * 2
    tokens = torch.zeros(2 * R, dtype=torch.int32, device=DEV)
    tokens[1::2] = x.int()
    u = torch.zeros(2 * R, device=DEV)
    u[0::2] = grid.repeat_interleave(n).repeat(4)
    r = grid.repeat(4 * n)
    acc = torch.zeros(R, dtype=torch.int32, device=DEV)
    nxt = torch.zeros(R, dtype=torch.int32, device=DEV)
    cache = _cache(R)
    cache.verify_draft(tokens, counts, p.expand(2 * R, V).contiguous(), u, r, acc, nxt,
                       draft_probs=q.expand(2 * R, V).contiguous())
    assert cache.status() == zp.OK
    kept = torch.where(acc == 1, x.int(), nxt).long()
    weight = q[x].double() / (n * n)
    freq = torch.zeros(V, dtype=torch.float64, device=DEV).index_add_(0, kept, weight)
    # each border of the two grids is met within half a cell: 1/(2n) an acceptance
    # (4 drafted tokens, weights q) and 1/(2n) a resampled token (2 borders)
    assert float((freq - p.double()).abs().max()) <= 2.0 / n


def test_lengths_are_committed():
    counts = [5, 1, 0, 3]
    d = Draft(counts, 300, seed=9)
    rows = torch.tensor([4, 0, 3, 1], dtype=torch.int32, device=DEV)
    lengths = torch.tensor([10, 20, 30, 40, 50, 60], dtype=torch.int32, device=DEV)
    cache = _cache(4)
    d.run(cache, lengths=lengths, req_idx=rows)
    assert cache.status() == zp.OK
    d.check()
    a = d.accepted.tolist()
    assert lengths.tolist() == [10, 20 - (2 - a[3]), 30, 40, 50 - (4 - a[0]), 60]


def test_refused_on_the_host():
    d = Draft([3, 2], 100, seed=10, pad=4)
    cache = _cache(2)
    s = torch.cuda.current_stream().cuda_stream

    def call(handle=None, tokens=None, target=None, dtype=zp.DTYPE_F32, vocab=100, stride=104, R=2,
             total=5, lengths=0, rows=0, acc=None):
        return zp.zp_verify_draft(
            cache.handle if handle is None else handle,
            d.tokens.data_ptr() if tokens is None else tokens, d.starts.data_ptr(), total,
            d.p.data_ptr() if target is None else target, d.q.data_ptr(), dtype, vocab, stride,
            d.accept_u.data_ptr(), d.sample_u.data_ptr(), lengths, rows, 0, R,
            d.accepted.data_ptr() if acc is None else acc, d.next.data_ptr(), s)

    bad = zp.ERR_INVALID_ARG
    assert call(tokens=0) == bad and call(target=0) == bad and call(acc=0) == bad
    assert call(vocab=0) == bad and call(stride=99) == bad and call(total=-1) == bad
    assert call(R=-1) == bad and call(R=3) == bad
    assert call(target=d.p.data_ptr() + 2) == bad and call(tokens=d.tokens.data_ptr() + 1) == bad
    assert call(lengths=d.starts.data_ptr(), rows=0) == bad
    assert call(dtype=2) == zp.ERR_UNSUPPORTED
    assert call(R=0) == zp.OK and call(total=0) == zp.OK
    args = (d.tokens, d.starts, d.p, d.accept_u, d.sample_u, d.accepted, d.next)
    for kw in (dict(draft_probs=d.q.contiguous()), dict(draft_probs=d.q.double()),
               dict(draft_probs=d.q[:4])):
        with pytest.raises(ValueError):
            cache.verify_draft(*args, **kw)
    for i, t in ((0, d.tokens.long()), (0, d.tokens[:4]), (2, d.p.half()), (2, d.p.t()),
                 (3, d.accept_u[:3]), (5, d.accepted[:1])):
        with pytest.raises(ValueError):
            cache.verify_draft(*args[:i], t, *args[i + 1:])
    assert cache.status() == zp.OK
    assert d.accepted.tolist() == [-7, -7]


def test_refused_on_the_device():
    d = Draft([3, 2, 4], 100, seed=11)
    cache = _cache(3)
    d.run(cache)
    good = d.accepted.clone(), d.next.clone()
    # a drafted token outside the vocabulary
    d.accept_u[3] = 0.0
    d.tokens[4] = 100
    d.run(cache)
    assert cache.status() == zp.ERR_DEVICE_CHECK
    assert d.accepted.tolist() == [int(good[0][0]), 0, int(good[0][2])]
    assert d.next.tolist() == [int(good[1][0]), -1, int(good[1][2])]
    # offsets past the rows: nothing is written for that request
    d.starts[3] = 10
    d.accepted.fill_(-7)
    d.run(cache)
    assert cache.status() == zp.ERR_DEVICE_CHECK
    assert d.accepted.tolist() == [int(good[0][0]), 0, -7]
    # a row and a length that do not fit: the outputs are right, the length stays
    d = Draft([3, 2, 4], 100, seed=11)
    for rows, lens in (([0, 3, 2], [9, 9, 9]), ([0, 1, 2], [9, 1, 9])):
        lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
        d.run(cache, lengths=lengths,
              req_idx=torch.tensor(rows, dtype=torch.int32, device=DEV))
        assert cache.status() == zp.ERR_DEVICE_CHECK
        d.check()
        a = d.accepted.tolist()
        assert lengths.tolist() == [9 - (2 - a[0]), lens[1], 9 - (3 - a[2])]


def test_captured_call():
    d = Draft([5, 3, 1], 5001, seed=12)
    cache = _cache(3)
    d.run(cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.run(cache)
    for seed in (13, 14):
        e = Draft([5, 3, 1], 5001, seed=seed)
        for name in ("p", "q", "tokens", "accept_u", "sample_u"):
            getattr(d, name).copy_(getattr(e, name))
        d.accepted.fill_(-7)
        graph.replay()
        assert cache.status() == zp.OK
        d.check()


@pytest.mark.parametrize("draft", [True, False])
def test_kept_tokens_have_the_targets_frequencies(draft):
    """As above with borders that lie on the grid's lines, so the frequencies are
    exact: p and q in 16ths.  u q < p and the draw from (3, 0, 0, 3) / 6 split 30
    cells a side without a rest; without q, u < p splits 16, and the draws from
    10, 15, 12 and 11 16ths (p without the drafted token) split 660."""
    V = 5
    p = torch.tensor([6, 1, 4, 5, 0], device=DEV) / 16
    q = torch.tensor([3, 6, 5, 2, 0], device=DEV) / 16
    n, m = (30, 30) if draft else (16, 660)
    R = 4 * n * m
    x = torch.arange(4, device=DEV).repeat_interleave(n * m)
    starts = torch.arange(R + 1, device=DEV, dtype=torch.int32) * 2
    tokens = torch.zeros(2 * R, dtype=torch.int32, device=DEV)
    tokens[1::2] = x.int()
    u = torch.zeros(2 * R, device=DEV)
    u[0::2] = ((torch.arange(n, device=DEV) + 0.5) / n).repeat_interleave(m).repeat(4)
    r = ((torch.arange(m, device=DEV) + 0.5) / m).repeat(4 * n)
    acc, nxt = (torch.zeros(R, dtype=torch.int32, device=DEV) for _ in range(2))
    cache = _cache(R)
    cache.verify_draft(tokens, starts, p.expand(2 * R, V).contiguous(), u, r, acc, nxt,
                       draft_probs=q.expand(2 * R, V).contiguous() if draft else None)
    assert cache.status() == zp.OK
    kept = torch.where(acc == 1, x.int(), nxt).long()
    count = torch.zeros(4, V, dtype=torch.int64, device=DEV)
    count.index_put_((x, kept), torch.ones_like(kept), accumulate=True)
    if draft:  # weighted by q, the kept tokens are the target's
        total = (count * (q[:4, None] * 16).long()).sum(0)
        assert total.tolist() == (p * 16 * n * m).long().tolist()
    else:  # whatever token was drafted
        for row in count.tolist():
            assert row == (p * n * m).long().tolist()
