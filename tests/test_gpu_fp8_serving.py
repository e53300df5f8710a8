"""An 8-bit cache and the draws from logits as a serving loop uses them: blocks reserved, prompts
in pieces, samples forked from one prompt, speculative steps drawn, verified and cut back, single
tokens; graphs replayed, calls beside each other, other streams."""
import math

import numpy as np
import pytest
import torch

from compressed_paged_kv_gb300 import zp
from tests.chunk_ref import verify_ref
from tests.fp8_ref import B, E4M3, Batch8, attn_ref, values

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


class Engine8:
    """A few layers' 8-bit pools with their block pool, and beside them the rows as they were
    before their rounding, [T, Hkv, d] in fp32."""

    def __init__(self, rows, L=2, Hkv=2, Hq=8, d=64, nb=160, width=24, seed=0):
        self.L, self.Hkv, self.Hq, self.d = L, Hkv, Hq, d
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.kp = [torch.full((nb, Hkv, B, d), 0x7f, dtype=torch.uint8, device=DEV).view(E4M3)
                   for _ in range(L)]
        self.vp = [k.clone() for k in self.kp]
        self.ks = [torch.full((nb, Hkv), math.nan, device=DEV) for _ in range(L)]
        self.vs = [s.clone() for s in self.ks]
        self.tables = torch.full((rows, width), -1, dtype=I32, device=DEV)
        self.lengths = torch.zeros(rows, dtype=I32, device=DEV)
        self.free = torch.randperm(nb, generator=self.g, device=DEV).int()
        self.count = _ints([nb])
        self.refs = torch.zeros(nb, dtype=I32, device=DEV)
        self.pool = (self.free, self.count, self.refs)
        self.cache = zp.Cache(self.kp, self.vp, Hq, max_requests=64, max_blocks_per_req=width,
                              k_scales=self.ks, v_scales=self.vs)
        self.scale = 1.0 / math.sqrt(d)
        empty = torch.empty(0, Hkv, d, device=DEV)
        self.K = [[empty] * rows for _ in range(L)]
        self.V = [[empty] * rows for _ in range(L)]

    def tokens(self, n):
        x = torch.randn(max(n, 1), self.Hq + 2 * self.Hkv, self.d, generator=self.g, device=DEV)
        x = x.bfloat16()[:n]
        return x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]

    def held(self, l, row, T):
        """K and V as the cache holds them."""
        blocks = self.tables[row, :-(-T // B)].long()
        return (values(p[l], s[l], blocks)[:T] for p, s in ((self.kp, self.ks), (self.vp, self.vs)))

    def check_cache(self, rows):
        """Every row within what the roundings may take: half a step (2^-4 of the value, or of the
        smallest normal number, 2^-10 of the scale) for the first, and for each time the scale
        doubled half a step of its numbers below the normal ones, the next scale's 2^-10: together
        less than 2^-9 of the last scale."""
        for row in rows:
            T = int(self.lengths[row])
            for l in range(self.L):
                blocks = self.tables[row, :-(-T // B)].long()
                for got, want, s in zip(self.held(l, row, T), (self.K[l][row], self.V[l][row]),
                                        (self.ks[l], self.vs[l])):
                    assert want.shape[0] == T
                    step = s[blocks].double().repeat_interleave(B, 0)[:T, :, None] * 2.0 ** -9
                    err = (got - want.double()).abs()
                    assert bool((err <= want.double().abs() * 2.0 ** -4 + step).all())

    def step(self, rows, counts, lengths, pad=0):
        starts = np.concatenate([[0], np.cumsum(counts)])
        total = int(starts[-1]) + pad
        s, ri = _ints(starts.tolist()), _ints(rows)
        G = self.Hq // self.Hkv
        for l in range(self.L):
            q, k, v = self.tokens(total)
            out = torch.full((total, self.Hq, self.d), 7.0, dtype=torch.bfloat16, device=DEV)
            self.cache.append_kv_chunk(l, k, v, s, self.tables, lengths, req_idx=ri)
            self.cache.chunk_attn(l, q, s, self.tables, lengths, self.scale, out, req_idx=ri)
            for i, row in enumerate(rows):
                a, b = int(starts[i]), int(starts[i + 1])
                if a == b:
                    continue
                self.K[l][row] = torch.cat([self.K[l][row], k[a:b].float()])
                self.V[l][row] = torch.cat([self.V[l][row], v[a:b].float()])
                kk, vv = self.held(l, row, int(lengths[row]))
                wide = (b - a) * G >= 1536
                want, tol = attn_ref(q[a:b], kk, vv, self.scale, 2.0 ** -17,
                                     2.0 ** -8 if wide else 2.0 ** -11)
                assert bool(((out[a:b].double() - want).abs() <= tol).all()), (l, row)
            assert bool((out[int(starts[-1]):] == 7.0).all())
        assert self.cache.status() == zp.OK

    def cut(self, row, n):
        for x in (self.K, self.V):
            for l in range(self.L):
                x[l][row] = x[l][row][:n]


def test_a_serving_run():
    e = Engine8(4)
    rows, prompt = [2, 0, 3], [200, 37, 118]
    ri = _ints(rows)
    e.cache.alloc_rows(e.tables, e.lengths, _ints(prompt), *e.pool, req_idx=ri)
    done = [0, 0, 0]
    progress = torch.zeros_like(e.lengths)
    while done != prompt:
        n = [min(64, p - x) for p, x in zip(prompt, done)]
        done = [x + y for x, y in zip(done, n)]
        progress[ri.long()] = _ints(done)
        e.step(rows, n, progress, pad=3 * 64 - sum(n))
    e.check_cache(rows)
    # speculative steps: drafted tokens drawn from their filtered probabilities
    V, R = 700, 3
    temp, top_k = torch.tensor([0.8, 1.0, 1.3, 0.5], device=DEV), _ints([0, 50, 0, 20])
    top_p, min_p = torch.tensor([0.9, 1.0, 0.95, 1.0], device=DEV), torch.zeros(4, device=DEV)
    kw = dict(temperature=temp, top_k=top_k, top_p=top_p, min_p=min_p)
    kept_tokens = 0
    for k in [4, 0, 2, 7]:
        for _ in range(k + 1):
            e.cache.append_slots(e.tables, e.lengths, 0, *e.pool, req_idx=ri)
        e.step(rows, [k + 1] * R, e.lengths)
        total = R * (k + 1)
        target = 2 * torch.randn(total, V, generator=e.g, device=DEV)
        draft = target + 0.3 * torch.randn(total, V, generator=e.g, device=DEV)
        idx = ri.repeat_interleave(k + 1)
        p, q = torch.empty_like(target), torch.empty_like(target)
        toks = torch.empty(total, dtype=I32, device=DEV)
        u = torch.rand(total, generator=e.g, device=DEV)
        e.cache.token_probs(target, p, req_idx=idx, **kw)
        e.cache.token_probs(draft, q, req_idx=idx, **kw)
        e.cache.sample(draft, u, toks, req_idx=idx, **kw)
        for i in range(total):  # a drawn token has a probability
            assert float(q[i, int(toks[i])]) > 0
        assert bool(((p.double().sum(1) - 1).abs() < 1e-5).all())
        drafted = toks.view(R, k + 1).roll(1, 1).contiguous().view(-1)
        starts = _ints([i * (k + 1) for i in range(R + 1)])
        au, su = torch.rand(total, generator=e.g, device=DEV), torch.rand(R, generator=e.g, device=DEV)
        acc, nxt = torch.empty(R, dtype=I32, device=DEV), torch.empty(R, dtype=I32, device=DEV)
        e.cache.verify_draft(drafted, starts, p, au, su, acc, nxt, draft_probs=q, lengths=e.lengths,
                             req_idx=ri)
        assert e.cache.status() == zp.OK
        want = verify_ref(drafted.cpu().numpy(), starts.cpu().numpy(), p.cpu().double().numpy(),
                          q.cpu().double().numpy(), au.cpu().numpy(), su.cpu().numpy())
        assert (acc.tolist(), nxt.tolist()) == want
        for i, a in enumerate(acc.tolist()):
            e.cut(rows[i], e.K[0][rows[i]].shape[0] - (k - a))
            kept_tokens += a
    assert kept_tokens > 0
    # single tokens
    for _ in range(3):
        e.cache.append_slots(e.tables, e.lengths, 0, *e.pool, req_idx=ri)
        for l in range(e.L):
            q, k, v = (t.contiguous() for t in e.tokens(R))
            out = torch.empty(R, e.Hq, e.d, dtype=torch.bfloat16, device=DEV)
            e.cache.append_kv(l, k, v, e.tables, e.lengths, req_idx=ri)
            e.cache.decode(l, q, e.tables, e.lengths, e.scale, out, req_idx=ri)
            for i, row in enumerate(rows):
                kk, vv = e.held(l, row, int(e.lengths[row]))
                want, tol = attn_ref(q[i:i + 1], kk, vv, e.scale)
                assert bool(((out[i:i + 1].double() - want).abs() <= tol).all())
    assert e.cache.status() == zp.OK
    e.cache.release_rows(e.tables, e.lengths, *e.pool, req_idx=ri)
    assert e.cache.status() == zp.OK
    assert int(e.count) == 160 and not bool(e.refs.any())


def test_a_prompt_shared_by_two_samples():
    """A forked row writes its own copy of the shared partial block, numbers and scales; the block
    that was shared keeps its bytes."""
    e = Engine8(3, seed=1)
    e.cache.alloc_rows(e.tables, e.lengths, _ints([75]), *e.pool, req_idx=_ints([0]))
    e.step([0], [75], e.lengths)
    e.cache.fork_rows(e.tables, e.lengths, e.refs, _ints([0, 0]), _ints([1, 2]))
    for x in (e.K, e.V):
        for l in range(e.L):
            x[l][1] = x[l][2] = x[l][0]
    tail = int(e.tables[0, 4])
    before = [x[tail].view(torch.uint8).clone() if x.dtype == E4M3 else x[tail].clone()
              for x in e.kp + e.vp + e.ks + e.vs]
    e.cache.append_slots(e.tables, e.lengths, 0, *e.pool, req_idx=_ints([1, 2]))
    for row in (1, 2):  # copied, to the byte
        own = int(e.tables[row, 4])
        assert own != tail
        for x, y in zip(e.kp + e.vp + e.ks + e.vs, before):
            got = x[own].view(torch.uint8) if x.dtype == E4M3 else x[own]
            upto = (slice(None), slice(0, 75 % B)) if x.dtype == E4M3 else slice(None)
            assert torch.equal(got[upto], y[upto])
    for _ in range(5):
        e.cache.append_slots(e.tables, e.lengths, 0, *e.pool, req_idx=_ints([1, 2]))
    e.step([2, 1], [6, 6], e.lengths)
    e.check_cache([0, 1, 2])
    for x, y in zip(e.kp + e.vp + e.ks + e.vs, before):
        got = x[tail].view(torch.uint8) if x.dtype == E4M3 else x[tail]
        assert torch.equal(got, y)
    assert e.cache.status() == zp.OK


def _mixed(seed=3):
    """Few rows, a tile, and one long enough to be widened."""
    b = Batch8([(400, 900), (5, 300), (1, 40), (450, 460), (700, 1200)], Hkv=2, Hq=8, d=128,
               seed=seed)
    few = Batch8([(1 + i % 4, 30 + 57 * i) for i in range(9)], Hkv=2, Hq=8, d=128, seed=seed + 1)
    return b, few


def test_two_graphs_of_one_handle():
    """Captured calls replayed in turn give what the calls gave, with the cache's rows, its lengths
    and the random numbers changed in between."""
    b, few = _mixed()
    V, R = 5000, 7
    logits = 3 * torch.randn(2, R, V, device=DEV)
    u = torch.rand(R, device=DEV)
    top_p = torch.full((R,), 0.9, device=DEV)
    toks = [torch.empty(R, dtype=I32, device=DEV) for _ in range(2)]
    probs = torch.empty(R, V, device=DEV)
    c, f = b.cache(max_requests=64), few.cache()
    q1 = few.q[:9].contiguous()
    dec = torch.empty(9, 8, 128, dtype=torch.bfloat16, device=DEV)

    def first():
        b.append(c)
        b.attn(c)
        c.sample(logits[0], u, toks[0], top_p=top_p)

    def second():
        few.attn(f)
        f.decode(0, q1, few.tables, few.lengths, few.scale, dec)
        few.attn(c2)
        c.sample(logits[1], u, toks[1])
        c.token_probs(logits[1], probs, top_p=top_p)

    c2 = zp.Cache(few.kp, few.vp, 8, max_requests=9, max_blocks_per_req=few.tables.shape[1],
                  k_scales=few.ks, v_scales=few.vs)
    first(), second()
    graphs = []
    for fn in (first, second):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn()
        graphs.append(g)
    for turn in range(3):
        u.copy_(torch.rand(R, device=DEV))
        few.lengths[8 - turn] -= 16
        b.lengths[1] -= 1
        first(), second()
        want = [x.clone() for x in (b.out, few.out, dec, *toks, probs)]
        for x in (b.out, few.out, dec, *toks, probs):
            x.fill_(7)
        for k in ((0, 1), (1, 0), (0, 0, 1))[turn]:
            graphs[k].replay()
        for x, y in zip((b.out, few.out, dec, *toks, probs), want):
            assert torch.equal(x, y)
    for cache in (c, c2, f):
        assert cache.status() == zp.OK


def test_calls_beside_each_other():
    """One handle: single tokens on one stream, chunks on another, draws on a third."""
    b, few = _mixed(9)
    c = b.cache(max_requests=64)
    rows = _ints([1, 2])
    q1, k1, v1 = (torch.randn(2, h, 128, device=DEV).bfloat16() for h in (8, 2, 2))
    logits = 3 * torch.randn(5, 40000, device=DEV)
    u, top_k = torch.rand(5, device=DEV), _ints([0, 3, 1000, 40, 0])
    starts = _ints([0, 400, 400, 400, 850, 1550])

    def single(out):
        c.append_kv(0, k1, v1, b.tables, b.lengths, req_idx=rows)
        c.decode(0, q1, b.tables, b.lengths, b.scale, out, req_idx=rows)

    def chunk(out):
        c.append_kv_chunk(0, b.k_new[:1550], b.v_new[:1550], starts, b.tables, b.lengths)
        c.chunk_attn(0, b.q[:1550], starts, b.tables, b.lengths, b.scale, out)

    def draws(out):
        c.sample(logits, u, out, top_k=top_k)

    def buffers():
        return (torch.full((2, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV),
                torch.full((1550, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV),
                torch.full((5,), -7, dtype=I32, device=DEV))

    want = buffers()
    for fn, x in zip((single, chunk, draws), want):
        fn(x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        got = buffers()
        torch.cuda.synchronize()
        for fn, s, x in zip((single, chunk, draws), streams, got):
            with torch.cuda.stream(s):
                fn(x)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    assert c.status() == zp.OK


def test_two_handles_on_two_streams():
    b, few = _mixed(17)
    caches = b.cache(), few.cache()
    for x, c in zip((b, few), caches):
        x.attn(c)
    want = b.out.clone(), few.out.clone()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        b.out.fill_(7), few.out.fill_(7)
        torch.cuda.synchronize()
        for x, c, s in zip((b, few), caches, streams):
            with torch.cuda.stream(s):
                x.attn(c)
        torch.cuda.synchronize()
        assert torch.equal(b.out, want[0]) and torch.equal(few.out, want[1])


def test_the_same_bits_again():
    """Atomics hand out places and arrivals; no result depends on their order."""
    b, few = _mixed(21)
    c, f = b.cache(max_requests=64), few.cache()
    logits = 3 * torch.randn(64, 50257, device=DEV).bfloat16()
    p = torch.empty(64, 50257, device=DEV)
    kw = dict(top_p=torch.linspace(0.3, 0.99, 64, device=DEV), min_p=torch.full((64,), 1e-4, device=DEV))
    first = None
    for _ in range(8):
        b.attn(c), few.attn(f), c.token_probs(logits, p, **kw)
        now = [x.clone() for x in (b.out, few.out, p)]
        if first is None:
            first = now
        assert all(torch.equal(x, y) for x, y in zip(first, now))


def test_one_request_in_many_rows():
    """The filters' entries taken again and again, and out of order."""
    c = Batch8([(1, 1)], dev=DEV).cache(max_requests=64)
    V = 999
    logits = 2 * torch.randn(12, V, device=DEV)
    idx = _ints([2, 2, 0, 0, 2, 1, 1, 0, 2, 0, 1, 2])
    t, p = torch.tensor([0.5, 1.0, 2.0], device=DEV), torch.tensor([0.6, 0.9, 1.0], device=DEV)
    k = _ints([0, 40, 7])
    u = torch.rand(12, device=DEV)
    got, all_got = torch.empty(12, dtype=I32, device=DEV), torch.empty(12, dtype=I32, device=DEV)
    c.sample(logits, u, got, temperature=t, top_p=p, top_k=k, req_idx=idx)
    at = idx.long()
    c.sample(logits, u, all_got, temperature=t[at].contiguous(), top_p=p[at].contiguous(),
             top_k=k[at].contiguous())
    assert torch.equal(got, all_got) and c.status() == zp.OK


def test_offsets_past_32_bits():
    """Blocks and logits whose byte offsets pass 2^32: a pool of more than 4 GB with the rows in
    its last blocks, the last rows of 5 GB of logits."""
    nb = (1 << 32) // (8 * B * 128) + 64
    b = Batch8([(3, 130), (1, 50), (40, 300), (400, 410)], Hkv=8, Hq=32, d=128, num_blocks=nb,
               first_block=nb - 64)
    c = b.cache(max_requests=64)
    b.append(c)
    b.attn(c)
    b.check_attn()
    assert c.status() == zp.OK
    for i, (n, T) in enumerate(b.spans):
        a = int(b.starts_np[i])
        for got, new, s in zip(b.rows_of(i), (b.k_new, b.v_new), (b.ks[0], b.vs[0])):
            new = new[a:a + n].double()
            step = s[b.tables[i, :-(-T // B)].long()].double().repeat_interleave(B, 0)[T - n:T]
            assert bool(((got[T - n:] - new).abs() <= new.abs() * 2.0 ** -4 +
                         step[..., None] * 2.0 ** -10).all())
    del b, c
    torch.cuda.empty_cache()
    R, V = 9, 151936
    pad = (5 << 30) // 4 // R // 8 * 8
    big = torch.empty(R * pad, device=DEV)
    logits = big.view(R, pad)[:, :V]
    logits.copy_(3 * torch.randn(R, V, device=DEV))
    small = logits.contiguous()
    c = Batch8([(1, 1)], dev=DEV).cache(max_requests=64)
    u = torch.rand(R, device=DEV)
    got = [torch.empty(R, dtype=I32, device=DEV) for _ in range(2)]
    top_p = torch.full((R,), 0.8, device=DEV)
    c.sample(logits, u, got[0], top_p=top_p)
    c.sample(small, u, got[1], top_p=top_p)
    assert torch.equal(*got) and c.status() == zp.OK


def test_launches_that_overlap():
    """A large batch of chunks of all lengths goes to three kernels that run into each other; what
    the calls around them write and read is in order: q, lengths and rows change right before a
    call, and its output is read, and written over, right behind it."""
    R = 160
    b = Batch8([(1 + i * 7 % 12, 30 + i * 29 % 500) for i in range(R)], Hkv=8, Hq=32, d=128, seed=31)
    c = b.cache()
    g = torch.Generator(device=DEV).manual_seed(5)
    qs = [torch.randn(b.total, 32, 128, generator=g, device=DEV).bfloat16() for _ in range(4)]
    cuts = [torch.zeros_like(b.lengths), (b.lengths > 40).int() * 13]
    full, q = b.lengths.clone(), torch.empty_like(qs[0])
    b.q = q

    def call(k):
        q.copy_(qs[k % 4])
        b.lengths.copy_(full - cuts[k % 2])
        b.attn(c)

    want = []
    for k in range(4):
        call(k)
        torch.cuda.synchronize()
        want.append(b.out.clone())
        b.lengths.copy_(full)
        if k % 2 == 0:
            b.check_attn()
    got = [torch.empty_like(b.out) for _ in range(24)]
    torch.cuda.synchronize()
    for k in range(24):  # no host wait in between
        call(k)
        got[k].copy_(b.out)
        b.out.fill_(7.0)
    torch.cuda.synchronize()
    for k in range(24):
        assert torch.equal(got[k], want[k % 4]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for k in range(4):
            call(k)
            got[k].copy_(b.out)
            b.out.fill_(7.0)
    for _ in range(5):
        for k in range(4):
            got[k].fill_(0.0)
        graph.replay()
        torch.cuda.synchronize()
        for k in range(4):
            assert torch.equal(got[k], want[k]), k
    assert c.status() == zp.OK
