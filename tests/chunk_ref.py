"""Plain 64-bit forms of the calls on ragged chunks of new tokens, and the
bounds their kernels are held to.  Test infrastructure only."""
import math

import numpy as np
import torch

from compressed_paged_kv_gb300 import zp

B = 16


class Batch:
    """A ragged batch over its own pools: spans = (new tokens, cached tokens
    with them) of each request.  Every pool slot no token fills holds NaN (the
    slots of partial blocks and the unused blocks), every table entry past a
    row's blocks is -1."""

    def __init__(self, spans, Hkv=2, Hq=4, d=64, seed=0, dev="cuda", permute=False, pad=0,
                 heavy=0.02, packed=True, L=1, layer=0, num_blocks=None, first_block=0,
                 extra_rows=0):
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.spans, self.Hkv, self.Hq, self.d, self.dev, self.layer = spans, Hkv, Hq, d, dev, layer
        R = len(spans)
        need = [-(-T // B) for _, T in spans]
        nb = num_blocks or sum(need) + 3
        width = max(need + [1]) + 1
        rows = R + extra_rows + (2 if permute else 0)
        order = rng.permutation(rows)[:R] if permute else np.arange(R)
        ids = first_block + rng.permutation(nb - first_block)
        tables = np.full((rows, width), -1, np.int32)
        lengths = np.zeros(rows, np.int32)
        at = 0
        for i, m in enumerate(need):
            tables[order[i], :m] = ids[at:at + m]
            lengths[order[i]] = spans[i][1]
            at += m
        self.order = order
        self.tables = torch.from_numpy(tables).to(dev)
        self.lengths = torch.from_numpy(lengths).to(dev)
        self.req_idx = torch.from_numpy(order.astype(np.int32)).to(dev) if permute else None
        counts = [n for n, _ in spans]
        self.starts_np = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.starts = torch.from_numpy(self.starts_np).to(dev)
        self.total = int(self.starts_np[-1]) + pad
        self.kp, self.vp = [], []
        for _ in range(L):
            k = torch.empty(nb, Hkv, B, d, dtype=torch.bfloat16, device=dev)
            v = torch.empty(nb, Hkv, B, d, dtype=torch.bfloat16, device=dev)
            if num_blocks is None:
                k.fill_(math.nan)
                v.fill_(math.nan)
            for i, (_, T) in enumerate(spans):
                m = need[i]
                if not m:
                    continue
                blocks = self.tables[order[i], :m].long()
                x = torch.randn(m, Hkv, B, d, generator=g, device=dev)
                hot = torch.rand(m, Hkv, B, 1, generator=g, device=dev) < heavy
                x = torch.where(hot, x * 8, x)
                y = torch.randn(m, Hkv, B, d, generator=g, device=dev)
                if T % B:
                    x[-1, :, T % B:] = math.nan
                    y[-1, :, T % B:] = math.nan
                k[blocks], v[blocks] = x.bfloat16(), y.bfloat16()
            self.kp.append(k)
            self.vp.append(v)
        h = Hq + 2 * Hkv
        if packed:
            x = torch.randn(max(self.total, 1), h, d, generator=g, device=dev).bfloat16()
            x = x[:self.total]
            self.q, self.k_new, self.v_new = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            self.q, self.k_new, self.v_new = (
                torch.randn(self.total, m, d, generator=g, device=dev).bfloat16()
                for m in (Hq, Hkv, Hkv))
        self.scale = 1.0 / math.sqrt(d)
        self.out = torch.full((self.total, Hq, d), 7.0, dtype=torch.bfloat16, device=dev)

    def cache(self, **kw):
        return zp.Cache(self.kp, self.vp, self.Hq,
                        max_requests=kw.get("max_requests", max(len(self.spans), 1)),
                        max_blocks_per_req=max(2, self.tables.shape[1]))

    def attn(self, cache, **kw):
        return cache.chunk_attn(self.layer, self.q, self.starts, self.tables, self.lengths,
                                self.scale, self.out, req_idx=self.req_idx, **kw)

    def append(self, cache, **kw):
        return cache.append_kv_chunk(self.layer, self.k_new, self.v_new, self.starts, self.tables,
                                     self.lengths, req_idx=self.req_idx, **kw)

    def rows_of(self, i):
        """K and V of request i in token order, [T, Hkv, d]."""
        T = self.spans[i][1]
        blocks = self.tables[self.order[i], :-(-T // B)].long()
        return (p[self.layer][blocks].permute(0, 2, 1, 3).reshape(-1, self.Hkv, self.d)[:T]
                for p in (self.kp, self.vp))

    def check_attn(self, skip=()):
        """The output against 64 bits, within the bound of `attn_ref`; the rows
        of no chunk (and of the requests in `skip`) still hold 7."""
        seen = torch.zeros(self.total, dtype=torch.bool, device=self.dev)
        worst = 0.0
        for i, (n, T) in enumerate(self.spans):
            if n == 0 or i in skip:
                continue
            a = int(self.starts_np[i])
            k, v = self.rows_of(i)
            want, tol = attn_ref(self.q[a:a + n], k, v, self.scale)
            err = (self.out[a:a + n].double() - want).abs()
            assert bool((err <= tol).all()), (
                i, n, T, float((err / tol).nan_to_num(math.inf).max()))
            worst = max(worst, float((err / tol).max()))
            seen[a:a + n] = True
        assert bool((self.out[~seen] == 7.0).all()), "rows of no chunk were written"
        return worst


def attn_ref(q, k, v, scale):
    """(out, bound) of one chunk in 64 bits: q [n, Hq, d], k and v [T, Hkv, d].

    The bound counts: the result's rounding to bf16 (half a step, 2^-8 of the
    value); each probability's rounding to bf16 for the product with V (2^-8 of
    sum p |v|); the fp32 logit, a sum of d products (d + 2 roundings of 2^-23 --
    the matrix unit may truncate -- of scale |q| . |k|), which enters a
    probability and the sum it is divided by (twice); and 2^-11 of sum p |v| for
    the exponential (2^-22), the T-term fp32 sums and the joining of partial
    results."""
    n, Hq, d = q.shape
    T, Hkv, _ = k.shape
    G = Hq // Hkv
    q, k, v = q.double(), k.double(), v.double()
    hidden = torch.arange(T, device=q.device)[None] > torch.arange(T - n, T, device=q.device)[:, None]
    out = torch.empty_like(q)
    tol = torch.empty_like(q)
    for hq in range(Hq):
        h = hq // G
        s = (q[:, hq] @ k[:, h].T) * scale
        mag = (q[:, hq].abs() @ k[:, h].abs().T) * abs(scale)
        p = torch.softmax(s.masked_fill(hidden, -math.inf), 1)
        spread = 2 * (d + 2) * 2.0 ** -23 * mag.masked_fill(hidden, 0).amax(1, keepdim=True)
        out[:, hq] = p @ v[:, h]
        pv = p @ v[:, h].abs()
        tol[:, hq] = 2.0 ** -8 * out[:, hq].abs() + (2.0 ** -8 + 2.0 ** -11 + spread) * pv
    return out, tol


def verify_ref(tokens, starts, p, q, accept_u, sample_u):
    """(accepted, next) in 64 bits; p and q [total, vocab] numpy, q may be None."""
    accepted, following = [], []
    p = np.asarray(p, np.float64)
    q = None if q is None else np.asarray(q, np.float64)
    for i in range(len(starts) - 1):
        a, n = int(starts[i]), int(starts[i + 1] - starts[i])
        if n == 0:
            accepted.append(None)
            following.append(None)
            continue
        j = 0
        while j < n - 1:
            x = int(tokens[a + j + 1])
            if not float(accept_u[a + j]) * (1.0 if q is None else q[a + j, x]) < p[a + j, x]:
                break
            j += 1
        w = p[a + j].copy()
        if j < n - 1:
            if q is None:
                w[int(tokens[a + j + 1])] = 0.0
            else:
                w = w - q[a + j]
        w = _weights(w)
        if w.sum() == 0.0:
            w = _weights(p[a + j])
        c = np.cumsum(w)
        accepted.append(j)
        following.append(int(np.argmax(c > float(sample_u[i]) * c[-1])) if c[-1] > 0 else -1)
    return accepted, following


def _weights(w):
    w = np.where(np.isfinite(w), w, 0.0)
    return np.maximum(w, 0.0)
