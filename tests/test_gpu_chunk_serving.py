"""The chunk calls as a serving loop makes them -- blocks reserved, a prompt in
pieces, its compression, speculative steps, a decode step -- against plain
64-bit forms at every step; two calls at once; calls the other files do not
make."""
import math

import numpy as np
import pytest
import torch

from compressed_paged_kv_gb300 import zp
from tests.chunk_ref import B, Batch, attn_ref, verify_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from compressed_paged_kv_gb300 import _build
    _build.build()
    yield
    torch.cuda.empty_cache()


def _bits(t):
    return t.contiguous().view(torch.int16)


def _ints(x):
    return torch.tensor(x, dtype=I32, device=DEV)


class Engine:
    """A few layers' pools with their block pool, and beside them the rows as
    plain tensors [T, Hkv, d]."""

    def __init__(self, rows, L=2, Hkv=2, Hq=8, d=64, nb=160, width=24, seed=0):
        self.L, self.Hkv, self.Hq, self.d, self.width = L, Hkv, Hq, d, width
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)
        self.kp = [torch.full((nb, Hkv, B, d), math.nan, dtype=torch.bfloat16, device=DEV)
                   for _ in range(L)]
        self.vp = [k.clone() for k in self.kp]
        self.tables = torch.full((rows, width), -1, dtype=I32, device=DEV)
        self.lengths = torch.zeros(rows, dtype=I32, device=DEV)
        self.free = torch.randperm(nb, generator=self.g, device=DEV).int()
        self.count = _ints([nb])
        self.refs = torch.zeros(nb, dtype=I32, device=DEV)
        self.pool = (self.free, self.count, self.refs)
        self.cache = zp.Cache(self.kp, self.vp, Hq, max_requests=rows, max_blocks_per_req=width)
        self.scale = 1.0 / math.sqrt(d)
        self.K = [[torch.empty(0, Hkv, d, dtype=torch.bfloat16, device=DEV)] * rows
                  for _ in range(L)]
        self.V = [list(x) for x in self.K]

    def tokens(self, n):
        """One layer's packed projections of n tokens: q, k, v."""
        x = torch.randn(max(n, 1), self.Hq + 2 * self.Hkv, self.d, generator=self.g, device=DEV)
        x = x.bfloat16()[:n]
        return x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]

    def step(self, rows, counts, lengths, pad=0):
        """Appends and attends one chunk a row, every layer, checked; returns
        the queries of each layer."""
        starts = np.concatenate([[0], np.cumsum(counts)])
        total, queries = int(starts[-1]) + pad, []
        s, ri = _ints(starts.tolist()), _ints(rows)
        for l in range(self.L):
            q, k, v = self.tokens(total)
            out = torch.full((total, self.Hq, self.d), 7.0, dtype=torch.bfloat16, device=DEV)
            self.cache.append_kv_chunk(l, k, v, s, self.tables, lengths, req_idx=ri)
            self.cache.chunk_attn(l, q, s, self.tables, lengths, self.scale, out, req_idx=ri)
            for i, row in enumerate(rows):
                a, b = int(starts[i]), int(starts[i + 1])
                if a == b:
                    continue
                self.K[l][row] = torch.cat([self.K[l][row], k[a:b]])
                self.V[l][row] = torch.cat([self.V[l][row], v[a:b]])
                want, tol = attn_ref(q[a:b], self.K[l][row], self.V[l][row], self.scale)
                assert bool(((out[a:b].double() - want).abs() <= tol).all()), (l, row)
            assert bool((out[int(starts[-1]):] == 7.0).all())
            queries.append(q)
        assert self.cache.status() == zp.OK
        return queries

    def check_cache(self, rows):
        for row in rows:
            T = int(self.lengths[row])
            for l in range(self.L):
                assert self.K[l][row].shape[0] == T
                blocks = self.tables[row, :-(-T // B)].long()
                for pool, want in ((self.kp[l], self.K[l][row]), (self.vp[l], self.V[l][row])):
                    got = pool[blocks].permute(0, 2, 1, 3).reshape(-1, self.Hkv, self.d)[:T]
                    assert torch.equal(_bits(got), _bits(want))


def test_a_serving_run():
    e = Engine(4)
    rows, prompt = [2, 0, 3], [200, 37, 118]
    ri = _ints(rows)
    e.cache.alloc_rows(e.tables, e.lengths, _ints(prompt), *e.pool, req_idx=ri)
    # the prompts in pieces of at most 64 tokens, padded to one shape
    done = [0, 0, 0]
    progress = torch.zeros_like(e.lengths)
    tail = {}
    while done != prompt:
        n = [min(64, p - x) for p, x in zip(prompt, done)]
        done = [x + y for x, y in zip(done, n)]
        progress[ri.long()] = _ints(done)
        qs = e.step(rows, n, progress, pad=3 * 64 - sum(n))
        at = np.concatenate([[0], np.cumsum(n)])
        for i, row in enumerate(rows):
            if n[i] >= 8:
                tail[row] = [q[at[i + 1] - 8:at[i + 1]] for q in qs]
    e.check_cache(rows)
    # row 2 is longer than six blocks: compressed to five
    N, w, row = 6, 8, 2
    wq = torch.stack([q.permute(1, 0, 2) for q in tail[row]])[:, None].contiguous()
    ws = torch.empty(e.cache.prefill_workspace_bytes(1, e.width), dtype=torch.uint8, device=DEV)
    kept = torch.empty(e.L, 1, e.Hkv, (N - 1) * B, dtype=I32, device=DEV)
    e.cache.compress_prefill(e.tables, e.lengths, wq, N, w, 0.2, *e.pool, ws,
                             req_idx=_ints([row]), kept_out=kept)
    assert e.cache.status() == zp.OK and int(e.lengths[row]) == (N - 1) * B
    for l in range(e.L):
        for x in (e.K, e.V):
            x[l][row] = torch.stack([x[l][row][kept[l, 0, h].long(), h] for h in range(e.Hkv)], 1)
    e.check_cache(rows)
    # speculative steps: k drafted tokens behind the last accepted one
    vocab = 500
    kept_tokens = 0
    for step, k in enumerate([4, 0, 2, 7, 3]):
        for _ in range(k + 1):
            e.cache.append_slots(e.tables, e.lengths, 0, *e.pool, req_idx=ri)
        n = [k + 1] * 3
        e.step(rows, n, e.lengths)
        total = 3 * (k + 1)
        logits = 2 * torch.randn(total, vocab, generator=e.g, device=DEV)
        p = torch.softmax(logits, 1)
        q = torch.softmax(logits + 0.3 * torch.randn(total, vocab, generator=e.g, device=DEV), 1)
        toks = torch.randint(0, vocab, (total,), generator=e.g, device=DEV).int()
        toks.view(3, k + 1)[:, 1:] = torch.multinomial(q, 1, generator=e.g).int().view(3, k + 1)[:, :-1]
        starts = _ints([i * (k + 1) for i in range(4)])
        u, r = (torch.rand(m, generator=e.g, device=DEV) for m in (total, 3))
        acc, nxt = torch.empty(3, dtype=I32, device=DEV), torch.empty(3, dtype=I32, device=DEV)
        draft = q if step % 2 == 0 else None
        e.cache.verify_draft(toks, starts, p, u, r, acc, nxt, draft_probs=draft,
                             lengths=e.lengths, req_idx=ri)
        assert e.cache.status() == zp.OK
        want = verify_ref(toks.cpu().numpy(), starts.cpu().numpy(), p.cpu().double().numpy(),
                          None if draft is None else draft.cpu().double().numpy(),
                          u.cpu().numpy(), r.cpu().numpy())
        assert (acc.tolist(), nxt.tolist()) == want
        for i, a in enumerate(acc.tolist()):
            for l in range(e.L):
                keep = e.K[l][rows[i]].shape[0] - (k - a)
                e.K[l][rows[i]] = e.K[l][rows[i]][:keep]
                e.V[l][rows[i]] = e.V[l][rows[i]][:keep]
            kept_tokens += a
        e.check_cache(rows)
    assert kept_tokens > 0
    # one plain decode step on the same rows
    e.cache.append_slots(e.tables, e.lengths, 0, *e.pool, req_idx=ri)
    for l in range(e.L):
        q, k, v = (t.contiguous() for t in e.tokens(3))
        out = torch.empty(3, e.Hq, e.d, dtype=torch.bfloat16, device=DEV)
        e.cache.append_kv(l, k, v, e.tables, e.lengths, req_idx=ri)
        e.cache.decode(l, q, e.tables, e.lengths, e.scale, out, req_idx=ri)
        for i, row in enumerate(rows):
            e.K[l][row] = torch.cat([e.K[l][row], k[i:i + 1]])
            e.V[l][row] = torch.cat([e.V[l][row], v[i:i + 1]])
            want, tol = attn_ref(q[i:i + 1], e.K[l][row], e.V[l][row], e.scale)
            assert bool(((out[i:i + 1].double() - want).abs() <= tol).all())
    # every block comes back
    e.cache.release_rows(e.tables, e.lengths, *e.pool, req_idx=ri)
    assert e.cache.status() == zp.OK
    assert int(e.count) == 160 and not bool(e.refs.any())


def test_a_prompt_shared_by_two_samples():
    """A forked row's speculative step writes its own copy of the shared
    partial block."""
    e = Engine(3, seed=1)
    e.cache.alloc_rows(e.tables, e.lengths, _ints([75]), *e.pool, req_idx=_ints([0]))
    e.step([0], [75], e.lengths)
    e.cache.fork_rows(e.tables, e.lengths, e.refs, _ints([0, 0]), _ints([1, 2]))
    for l in range(e.L):
        e.K[l][1] = e.K[l][2] = e.K[l][0]
        e.V[l][1] = e.V[l][2] = e.V[l][0]
    for _ in range(6):
        e.cache.append_slots(e.tables, e.lengths, 0, *e.pool, req_idx=_ints([1, 2]))
    e.step([2, 1], [6, 6], e.lengths)
    e.check_cache([0, 1, 2])


def test_calls_at_once_on_disjoint_requests():
    """Decode and single-token append on one stream beside chunk append, chunk
    attention and verification on another, one handle."""
    spans = [(70, 900), (1, 1500), (5, 333), (130, 2000), (1, 777), (1, 40)]
    b = Batch(spans, 2, 8, 128, seed=21, L=2)
    cache = b.cache()
    chunk = dict(starts=_ints([0, 70, 70, 75, 205, 205, 205]))
    rows = _ints([1, 4, 5])
    q1, k1, v1 = (torch.randn(3, h, 128, device=DEV).bfloat16() for h in (8, 2, 2))
    vocab = 5000
    p = torch.softmax(torch.randn(205, vocab, device=DEV), 1)
    u, r = torch.rand(205, device=DEV), torch.rand(6, device=DEV)
    toks = torch.randint(0, vocab, (205,), device=DEV).int()

    def side_a(out):
        for l in range(2):
            cache.append_kv(l, k1, v1, b.tables, b.lengths, req_idx=rows)
            cache.decode(l, q1, b.tables, b.lengths, b.scale, out[l], req_idx=rows)

    def side_b(out, acc, nxt):
        for l in range(2):
            cache.append_kv_chunk(l, b.k_new[:205], b.v_new[:205], chunk["starts"], b.tables,
                                  b.lengths)
            cache.chunk_attn(l, b.q[:205], chunk["starts"], b.tables, b.lengths, b.scale, out[l])
        cache.verify_draft(toks, chunk["starts"], p, u, r, acc, nxt)

    def buffers():
        return (torch.full((2, 3, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV),
                torch.full((2, 205, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV),
                torch.full((6,), -7, dtype=I32, device=DEV),
                torch.full((6,), -7, dtype=I32, device=DEV))

    want = buffers()
    side_a(want[0])
    side_b(*want[1:])
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = buffers()
        torch.cuda.synchronize()
        with torch.cuda.stream(s[0]):
            side_a(got[0])
        with torch.cuda.stream(s[1]):
            side_b(*got[1:])
        torch.cuda.synchronize()
        assert cache.status() == zp.OK
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_chunks_beside_a_compression():
    """zp_compress of two full rows on one stream, a chunk's append and
    attention of the others on another, one handle: as one after the other."""
    N, w = 8, 8
    spans = [(70, 900), (5, 333), (130, 2000), (0, N * B), (0, N * B)]
    wq = torch.randn(1, 2, 8, w, 128, device=DEV).bfloat16()
    results = []
    for at_once in (False, True, True, True):
        b = Batch(spans, 2, 8, 128, seed=29)
        nb = b.kp[0].shape[0]
        cache = b.cache()
        refs = torch.zeros(nb, dtype=I32, device=DEV)
        refs[b.tables[b.tables >= 0].long()] = 1
        unused = torch.nonzero(refs == 0).flatten().int()
        free = torch.cat([unused, torch.zeros(nb - unused.numel(), dtype=I32, device=DEV)])
        count = _ints([unused.numel()])
        s = [torch.cuda.Stream(), torch.cuda.Stream()] if at_once else [None, None]
        torch.cuda.synchronize()
        cache.compress(b.tables, b.lengths, wq, N, w, 0.5, free, count, refs,
                       req_idx=_ints([3, 4]), stream=s[0])
        for _ in range(3):
            b.append(cache, stream=s[1])
            b.attn(cache, stream=s[1])
        torch.cuda.synchronize()
        assert cache.status() == zp.OK
        assert b.lengths.tolist()[3:] == [(N - 1) * B] * 2
        results.append([b.out, b.kp[0], b.vp[0], b.tables])
        for got, want in zip(results[-1], results[0]):
            view = (lambda t: _bits(t)) if got.dtype == torch.bfloat16 else (lambda t: t)
            assert torch.equal(view(got), view(want))


def test_two_handles_at_once():
    """Two handles over the same pools (each its own workspace), their chunk
    attentions on two streams."""
    b = Batch([(300, 4000), (5, 2500), (1, 6000)], 2, 8, 128, seed=22)
    caches = [b.cache(), b.cache()]
    b.attn(caches[0])
    want = b.out.clone()
    outs = [torch.empty_like(want), torch.empty_like(want)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, o, st in zip(caches, outs, s):
            c.chunk_attn(0, b.q, b.starts, b.tables, b.lengths, b.scale, o, stream=st)
    torch.cuda.synchronize()
    for c, o in zip(caches, outs):
        assert c.status() == zp.OK
        assert torch.equal(_bits(o), _bits(want))


def test_two_graphs_of_one_handle():
    """Two captured graphs share the handle's workspace; replayed in turn."""
    b = Batch([(300, 4000), (5, 2500)], 2, 8, 128, seed=23)
    c = Batch([(1, 3000), (64, 64), (9, 5000)], 2, 8, 128, seed=24)
    nb = max(b.kp[0].shape[0], c.kp[0].shape[0])  # one pool size a handle

    def grow(x):
        y = torch.full((nb,) + tuple(x.shape[1:]), math.nan, dtype=x.dtype, device=DEV)
        y[:x.shape[0]] = x
        return y

    for t in (b, c):
        t.kp, t.vp = [grow(x) for x in t.kp], [grow(x) for x in t.vp]
    cache = zp.Cache(b.kp + c.kp, b.vp + c.vp, 8, max_requests=4, max_blocks_per_req=400)

    def run(t, layer):
        cache.chunk_attn(layer, t.q, t.starts, t.tables, t.lengths, t.scale, t.out)

    graphs, want = [], []
    for layer, t in enumerate((b, c)):
        run(t, layer)
        want.append(t.out.clone())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(t, layer)
        graphs.append(graph)
    for k in (0, 1, 1, 0, 0, 1):
        t = (b, c)[k]
        t.out.fill_(7.0)
        graphs[k].replay()
        assert cache.status() == zp.OK
        assert torch.equal(_bits(t.out), _bits(want[k]))
        t.check_attn()


def test_a_long_row_of_queries_that_are_not_finite():
    """Every query NaN, or every value of a long row: NaN out, and in time."""
    b = Batch([(600, 60000)], 1, 4, 128, seed=25)
    cache = b.cache()
    keep = b.q.clone()
    b.q.fill_(math.nan)
    b.attn(cache)
    assert cache.status() == zp.OK and bool(torch.isnan(b.out).all())
    b.q.copy_(keep)
    b.vp[0][b.tables[0, 3].long(), 0, 5] = math.nan
    b.attn(cache)
    assert cache.status() == zp.OK and bool(torch.isnan(b.out).all())


def test_hidden_values_behind_a_long_row():
    """Rows computed twice because of an infinity hidden behind them, over a
    long cache: right, and no wait of the others runs out."""
    b = Batch([(60, 30000)], 1, 4, 128, seed=26)
    k, v = b.rows_of(0)
    want, tol = attn_ref(b.q, k, v, b.scale)
    pos = torch.arange(29970, 30000, device=DEV)
    b.vp[0][b.tables[0].long()[pos // B], 0, pos % B] = math.inf
    cache = b.cache()
    b.attn(cache)
    assert cache.status() == zp.OK
    assert bool(((b.out.double() - want).abs() <= tol)[:30].all())
    assert not bool(torch.isfinite(b.out[30:]).any())


@pytest.mark.parametrize("spans", [[(200, 1000)], [(3, 4000)] * 5])
@pytest.mark.parametrize("d", [64, 128])
def test_a_second_result_is_within_the_same_bound(spans, d):
    """Rows with a hidden infinity, in items cut between CTAs and whole ones."""
    b = Batch(spans, 2, 16, d, seed=27)
    want = []
    for i, (n, T) in enumerate(spans):
        k, v = b.rows_of(i)
        a = int(b.starts_np[i])
        want.append(attn_ref(b.q[a:a + n], k, v, b.scale))
        b.vp[0][b.tables[i, (T - 1) // B].long(), :, (T - 1) % B, ::3] = -math.inf
    cache = b.cache()
    b.attn(cache)
    assert cache.status() == zp.OK
    for i, (n, T) in enumerate(spans):
        a = int(b.starts_np[i])
        ok = (b.out[a:a + n - 1].double() - want[i][0][:-1]).abs() <= want[i][1][:-1]
        assert bool(ok.all())


@pytest.mark.parametrize("n,T,Hkv,Hq,d", [(9000, 9000, 1, 2, 64), (7001, 12345, 1, 5, 128)])
def test_a_long_prompt(n, T, Hkv, Hq, d):
    """A whole prompt of thousands of tokens, and a piece as long."""
    b = Batch([(n, T)], Hkv, Hq, d, seed=41)
    cache = b.cache()
    b.attn(cache)
    assert cache.status() == zp.OK
    b.check_attn()


def test_packed_rows_past_32_bits():
    """The last rows of packed tensors of more than 2^27 rows (2^33 elements)."""
    n, T, total = 21, 90, (1 << 27) + 40
    b = Batch([(n, T)], 1, 1, 64, seed=28)
    big = torch.empty(total, 1, 64, dtype=torch.bfloat16, device=DEV)
    big[-n - 2:-2] = b.k_new
    starts = _ints([total - n - 2, total - 2])
    cache = b.cache()
    cache.append_kv_chunk(0, big, big, starts, b.tables, b.lengths)
    assert cache.status() == zp.OK
    k, v = b.rows_of(0)
    assert torch.equal(_bits(k[T - n:]), _bits(b.k_new))
    assert torch.equal(_bits(v[T - n:]), _bits(b.k_new))
    big[-n - 2:-2] = b.q
    out = torch.empty_like(big)
    out[-2:] = 7.0
    out[-n - 3] = 7.0
    cache.chunk_attn(0, big, starts, b.tables, b.lengths, b.scale, out)
    assert cache.status() == zp.OK
    want, tol = attn_ref(b.q, k, v, b.scale)
    assert bool(((out[-n - 2:-2].double() - want).abs() <= tol).all())
    assert bool((out[-2:] == 7.0).all() and (out[-n - 3] == 7.0).all())


# ------------------------------------------------------------- verification

def _verify(cache, tokens, starts, p, q, u, r, R=None, **kw):
    R = starts.numel() - 1 if R is None else R
    acc, nxt = (torch.full((R,), -7, dtype=I32, device=DEV) for _ in range(2))
    cache.verify_draft(tokens, starts, p, u, r, acc, nxt, draft_probs=q, **kw)
    return acc, nxt


def _plain(tokens, starts, p, q, u, r):
    acc, nxt = verify_ref(tokens.cpu().numpy(), starts.cpu().numpy(), p.cpu().double().numpy(),
                          None if q is None else q.cpu().double().numpy(), u.cpu().numpy(),
                          r.cpu().numpy())
    return [-7 if x is None else x for x in acc], [-7 if x is None else x for x in nxt]


def _pool_cache(R):
    pool = torch.zeros(1, 1, B, 64, dtype=torch.bfloat16, device=DEV)
    return zp.Cache([pool], [pool.clone()], 1, max_requests=R, max_blocks_per_req=2)


@pytest.mark.parametrize("dtype,shift", [(torch.float32, 1), (torch.float32, 3),
                                         (torch.bfloat16, 1), (torch.bfloat16, 4)])
def test_rows_aligned_unlike(dtype, shift):
    """p and q at different offsets from 16 bytes."""
    V, total = 3001, 12
    g = torch.Generator(device=DEV)
    g.manual_seed(31)
    buf = torch.empty(2, total * V + 8, dtype=dtype, device=DEV)
    p = buf[0, :total * V].view(total, V)
    q = torch.empty(total * V + 8, dtype=dtype, device=DEV)[shift:shift + total * V].view(total, V)
    x = 2 * torch.randn(total, V, generator=g, device=DEV)
    p.copy_(torch.softmax(x, 1))
    q.copy_(torch.softmax(x + 0.5 * torch.randn(total, V, generator=g, device=DEV), 1))
    toks = torch.multinomial(q.float(), 1, generator=g)[:, 0].int().roll(1)
    u, r = torch.rand(total, generator=g, device=DEV), torch.rand(3, generator=g, device=DEV)
    starts = _ints([0, 4, 7, 12])
    cache = _pool_cache(3)
    acc, nxt = _verify(cache, toks, starts, p, q, u, r)
    assert cache.status() == zp.OK
    assert (acc.tolist(), nxt.tolist()) == _plain(toks, starts, p, q, u, r)


@pytest.mark.parametrize("stop", [0, 31, 32, 33, 63, 64, 99, 100])
def test_long_drafts(stop):
    """100 drafted tokens, the first `stop` of them accepted."""
    V, n = 64, 101
    g = torch.Generator(device=DEV)
    g.manual_seed(32)
    p = torch.softmax(torch.randn(n, V, generator=g, device=DEV), 1)
    q = p.clone()
    toks = torch.randint(0, V, (n,), generator=g, device=DEV).int()
    u = torch.rand(n, generator=g, device=DEV) * 0.99
    if stop < n - 1:
        q[stop, int(toks[stop + 1])] = 4.0
        u[stop] = 0.9
    starts, r = _ints([0, n]), torch.rand(1, generator=g, device=DEV)
    cache = _pool_cache(1)
    lengths = _ints([500])
    acc, nxt = _verify(cache, toks, starts, p, q, u, r, lengths=lengths)
    assert cache.status() == zp.OK
    assert (acc.tolist(), nxt.tolist()) == _plain(toks, starts, p, q, u, r)
    assert acc.tolist() == [stop] and lengths.tolist() == [500 - (100 - stop)]


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [37, 5000, 70001])
def test_weights_that_are_not_finite(draft, V):
    """Infinities and NaN of either sign, in p and in q, in the deciding row."""
    g = torch.Generator(device=DEV)
    g.manual_seed(33)
    total, R = 24, 12
    x = torch.randn(total, V, generator=g, device=DEV)
    p = torch.softmax(x, 1)
    q = torch.softmax(x + torch.randn(total, V, generator=g, device=DEV), 1)
    toks = torch.randint(10, V, (total,), generator=g, device=DEV).int()
    bad = [math.nan, math.inf, -math.inf, -0.5]
    for row in range(total):
        for k in range(5):
            at = int(torch.randint(0, 10 if k else V, (1,), generator=g, device=DEV))
            if k == 0 and at in toks.tolist():
                continue
            (p if (row + k) % 2 or not draft else q)[row, at] = bad[(row // 2 + k) % 4]
    u, r = torch.rand(total, generator=g, device=DEV), torch.rand(R, generator=g, device=DEV)
    starts = _ints([2 * i for i in range(R + 1)])
    cache = _pool_cache(R)
    q = q if draft else None
    acc, nxt = _verify(cache, toks, starts, p, q, u, r)
    assert cache.status() == zp.OK
    assert (acc.tolist(), nxt.tolist()) == _plain(toks, starts, p, q, u, r)


@pytest.mark.parametrize("dtype,draft", [(torch.float32, True), (torch.float32, False),
                                         (torch.bfloat16, True), (torch.bfloat16, False)])
@pytest.mark.parametrize("R,V", [(700, 500), (320, 40000), (160, 40001), (64, 9001), (30, 70003),
                                 (3, 33000)])
def test_every_cluster_size(dtype, draft, R, V):
    """Batches and vocabularies for clusters of one, two, four and eight CTAs of
    either size."""
    g = torch.Generator(device=DEV)
    g.manual_seed(39)
    total = 2 * R
    x = 2 * torch.randn(total, V, generator=g, device=DEV)
    p = torch.softmax(x, 1).to(dtype)
    q = torch.softmax(x + 0.5 * torch.randn(total, V, generator=g, device=DEV), 1).to(dtype)
    toks = torch.multinomial(q.float(), 1, generator=g)[:, 0].int().roll(1)
    u, r = torch.rand(total, generator=g, device=DEV), torch.rand(R, generator=g, device=DEV)
    starts = _ints([2 * i for i in range(R + 1)])
    q = q if draft else None
    cache = _pool_cache(R)
    acc, nxt = _verify(cache, toks, starts, p, q, u, r)
    assert cache.status() == zp.OK
    assert (acc.tolist(), nxt.tolist()) == _plain(toks, starts, p, q, u, r)


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [5000, 70001])
def test_16_bit_weights_that_are_not_finite(draft, V):
    g = torch.Generator(device=DEV)
    g.manual_seed(40)
    total, R = 16, 8
    x = torch.randn(total, V, generator=g, device=DEV)
    p = torch.softmax(x, 1).bfloat16()
    q = torch.softmax(x + torch.randn(total, V, generator=g, device=DEV), 1).bfloat16()
    toks = torch.randint(10, V, (total,), generator=g, device=DEV).int()
    for row in range(total):  # positions no drafted token has
        t = p if row % 3 or not draft else q
        t[row, row % 10] = [math.nan, math.inf, -math.inf, -0.5][row % 4]
    u, r = torch.rand(total, generator=g, device=DEV), torch.rand(R, generator=g, device=DEV)
    starts = _ints([2 * i for i in range(R + 1)])
    q = q if draft else None
    cache = _pool_cache(R)
    acc, nxt = _verify(cache, toks, starts, p, q, u, r)
    assert cache.status() == zp.OK
    assert (acc.tolist(), nxt.tolist()) == _plain(toks, starts, p, q, u, r)


def test_verification_of_a_padded_batch_on_another_stream():
    g = torch.Generator(device=DEV)
    g.manual_seed(34)
    V, total = 1009, 40
    p = torch.softmax(torch.randn(total, V, generator=g, device=DEV), 1)
    toks = torch.randint(0, V, (total,), generator=g, device=DEV).int()
    u, r = torch.rand(total, generator=g, device=DEV), torch.rand(8, generator=g, device=DEV)
    starts = _ints([3, 8, 8, 17, 20, 20, 20, 20, 20])  # rows 0-2 and 20-39 of no chunk
    cache = _pool_cache(8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        acc, nxt = _verify(cache, toks, starts, p, None, u, r)
    side.synchronize()
    assert cache.status(stream=side) == zp.OK
    assert (acc.tolist(), nxt.tolist()) == _plain(toks, starts, p, None, u, r)
    # offsets that fall: that request alone is refused
    starts[3] = 6
    acc, nxt = _verify(cache, toks, starts, p, None, u, r)
    assert cache.status() == zp.ERR_DEVICE_CHECK
    want = _plain(toks, _ints([3, 8, 8]), p, None, u, r[:2])
    assert acc.tolist()[:3] == [want[0][0], -7, -7]
    last = _plain(toks, _ints([6, 20]), p, None, u, r[3:4])
    assert (acc.tolist()[3], nxt.tolist()[3]) == (last[0][0], last[1][0])


def test_probability_rows_past_32_bits():
    """Rows beyond 2^31 elements, a vocabulary of 2^20 + 5."""
    V, total = (1 << 20) + 5, 2060
    g = torch.Generator(device=DEV)
    g.manual_seed(35)
    p = torch.empty(total, V, device=DEV)
    q = torch.empty(total, V, device=DEV)
    x = torch.randn(7, V, generator=g, device=DEV)
    p[-7:] = torch.softmax(x, 1)
    q[-7:] = torch.softmax(x + 0.3 * torch.randn(7, V, generator=g, device=DEV), 1)
    toks = torch.zeros(total, dtype=I32, device=DEV)
    toks[-6:] = torch.multinomial(q[-7:-1], 1, generator=g)[:, 0].int()
    u, r = torch.rand(total, generator=g, device=DEV), torch.rand(2, generator=g, device=DEV)
    starts = _ints([total - 7, total - 3, total])
    cache = _pool_cache(2)
    acc, nxt = _verify(cache, toks, starts, p, q, u, r)
    assert cache.status() == zp.OK
    want = _plain(toks[-7:], _ints([0, 4, 7]), p[-7:], q[-7:], u[-7:], r)
    assert (acc.tolist(), nxt.tolist()) == want


def test_shared_memory_is_refused():
    """Outputs that lie in inputs or in each other, and K/V rows inside the
    pools they are copied to."""
    b = Batch([(8, 40), (3, 20)], 2, 4, 64, seed=36, packed=False)
    cache = b.cache()
    before = b.kp[0].clone()
    args = (b.starts, b.tables, b.lengths)
    V = 50
    p = torch.rand(11, V, device=DEV)
    u, r = torch.rand(11, device=DEV), torch.rand(2, device=DEV)
    toks = torch.zeros(11, dtype=I32, device=DEV)
    acc, nxt = torch.zeros(2, dtype=I32, device=DEV), torch.zeros(2, dtype=I32, device=DEV)
    both = torch.zeros(3, dtype=I32, device=DEV)
    keep = b.q.clone()

    def verify(tokens=toks, accepted=acc, next_tokens=nxt, lengths=None, uu=u):
        return cache.verify_draft(tokens, b.starts, p, uu, r, accepted, next_tokens,
                                  lengths=lengths)

    calls = [lambda: cache.chunk_attn(0, b.q, *args, b.scale, b.q),
             lambda: cache.append_kv_chunk(0, b.kp[0].view(-1, 2, 64)[:11], b.v_new, *args),
             lambda: cache.append_kv_chunk(0, b.k_new, b.vp[0].view(-1, 2, 64)[-11:], *args),
             lambda: verify(next_tokens=acc), lambda: verify(next_tokens=toks[:2]),
             lambda: verify(accepted=toks[9:]), lambda: verify(accepted=both[:2],
                                                               next_tokens=both[1:]),
             lambda: verify(lengths=toks), lambda: verify(accepted=b.starts[1:]),
             lambda: verify(accepted=p.view(-1)[:2].view(I32)),
             lambda: verify(accepted=u[4:6].view(I32))]
    for f in calls:
        with pytest.raises(zp.ZpError) as err:
            f()
        assert err.value.status == zp.ERR_INVALID_ARG
    assert cache.status() == zp.OK
    assert torch.equal(_bits(b.q), _bits(keep)) and torch.equal(_bits(b.kp[0]), _bits(before))
    assert not bool(acc.any()) and not bool(toks.any())


def test_batches_of_nothing():
    """No packed row at all (tensors without memory), and no request."""
    b = Batch([(0, 40), (0, 0)], 2, 4, 64, seed=38)
    cache = b.cache()
    lengths = b.lengths.clone()
    none = torch.empty(0, dtype=I32, device=DEV)
    f32 = torch.empty(0, device=DEV)
    for starts, R in ((b.starts, 2), (b.starts[:1], 0)):
        b.starts = starts
        b.append(cache)
        b.attn(cache)
        acc, nxt = _verify(cache, none, starts, torch.empty(0, 10, device=DEV), None, f32,
                           torch.rand(R, device=DEV), R=R, lengths=b.lengths)
        assert acc.tolist() == [-7] * R and nxt.tolist() == [-7] * R
    assert cache.status() == zp.OK
    assert torch.equal(b.lengths, lengths)


def test_sizes_beyond_the_limits_are_refused():
    b = Batch([(8, 40)], 2, 4, 64, seed=37, packed=False)
    cache = b.cache()
    s = torch.cuda.current_stream().cuda_stream
    for stride, want in (((1 << 26) + 1, zp.ERR_UNSUPPORTED), (b.tables.shape[1], zp.OK)):
        assert zp.zp_paged_chunk_attn(cache.handle, 0, b.q.data_ptr(), 256, b.starts.data_ptr(), 8,
                                      b.tables.data_ptr(), stride, 1, b.lengths.data_ptr(), 0, 1,
                                      0.1, b.out.data_ptr(), s) == want
        assert zp.zp_append_kv_chunk(cache.handle, 0, b.k_new.data_ptr(), 128, b.v_new.data_ptr(),
                                     128, b.starts.data_ptr(), 8, b.tables.data_ptr(), stride, 1,
                                     b.lengths.data_ptr(), 0, 1, s) == want
    x = torch.zeros(64, device=DEV)
    y = torch.zeros(64, dtype=I32, device=DEV)
    assert zp.zp_verify_draft(cache.handle, y.data_ptr(), b.starts.data_ptr(), 8, x.data_ptr(), 0,
                              zp.DTYPE_F32, (1 << 30) + 1, 1 << 31, x.data_ptr(), x.data_ptr(), 0,
                              0, 0, 1, y.data_ptr() + 128, y.data_ptr() + 192, s) \
        == zp.ERR_UNSUPPORTED
    assert cache.status() == zp.OK
