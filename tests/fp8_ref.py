"""Plain 64-bit forms of the calls on an 8-bit cache and of the draws from logits,
and the bounds their kernels are held to.  Test infrastructure only."""
import math

import numpy as np
import torch

from compressed_paged_kv_gb300 import zp

B = 16
E4M3 = torch.float8_e4m3fn
MIN_EXP, MAX_EXP = -32, 32
WIDE_ROWS = 1536  # query rows from which on a chunk's attention may be the bf16 kernel's


def scale_of(most):
    """The least power of two, 2^-32 .. 2^32, that takes `most` into 448 (64 bits)."""
    most = most.double()
    e = torch.full_like(most, MIN_EXP)
    for x in range(MIN_EXP, MAX_EXP):
        e = torch.where(most > 448.0 * 2.0 ** x, x + 1.0, e)
    return torch.exp2(e)


def e4m3(x):
    """x (64 bits) to the nearest e4m3 number, ties to even, saturating, NaN kept."""
    e = torch.frexp(x.nan_to_num(0.0, 448.0, -448.0))[1].clamp(min=-5) - 4
    step = torch.exp2(e.double())
    y = ((x.nan_to_num(0.0, 448.0, -448.0) / step).round() * step).clamp(-448.0, 448.0)
    return torch.where(x.isnan(), math.nan, y)


def put(numbers, scale, first, rows):
    """One slab after an append: numbers [16, d] (64 bits), its scale, the first slot and
    the new rows [n, d]; returns the new (numbers, scale)."""
    a = rows.double().abs().nan_to_num(0.0, math.inf).amax()
    s = scale_of(a)
    numbers = numbers.clone()
    if first:
        s = torch.maximum(s, scale.double())
        numbers[:first] = e4m3(numbers[:first] * (scale.double() / s))
    numbers[first:first + len(rows)] = e4m3(rows.double() / s)
    return numbers, s


class Batch8:
    """A ragged batch over an 8-bit cache of its own: spans = (new tokens, cached tokens with
    them) of each request.  Slots that no token fills hold NaN, and so do the scales of
    blocks without any."""

    def __init__(self, spans, Hkv=2, Hq=4, d=64, seed=0, dev="cuda", permute=False, pad=0,
                 heavy=0.02, packed=True, L=1, layer=0, num_blocks=None, first_block=0,
                 spread=6):
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.spans, self.Hkv, self.Hq, self.d, self.dev, self.layer = spans, Hkv, Hq, d, dev, layer
        R = len(spans)
        need = [-(-T // B) for _, T in spans]
        nb = num_blocks or sum(need) + 3
        rows = R + (2 if permute else 0)
        order = rng.permutation(rows)[:R] if permute else np.arange(R)
        ids = first_block + rng.permutation(nb - first_block)
        tables = np.full((rows, max(need + [1]) + 1), -1, np.int32)
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
        self.kp, self.vp, self.ks, self.vs = [], [], [], []
        for _ in range(L):
            for pools, scales in ((self.kp, self.ks), (self.vp, self.vs)):
                pool = torch.empty(nb, Hkv, B, d, dtype=torch.uint8, device=dev)
                scale = torch.full((nb, Hkv), math.nan, device=dev)
                if num_blocks is None:
                    pool.fill_(0x7f)  # NaN
                for i, (_, T) in enumerate(spans):
                    m = need[i]
                    if not m:
                        continue
                    blocks = self.tables[order[i], :m].long()
                    x = torch.randn(m, Hkv, B, d, generator=g, device=dev)
                    hot = torch.rand(m, Hkv, B, 1, generator=g, device=dev) < heavy
                    x = torch.where(hot, x * 8, x)
                    # scales of all sizes: rows of a block within `spread` binades
                    if pools is self.vp:
                        x = x * torch.exp2(spread * torch.rand(m, Hkv, 1, 1, generator=g,
                                                               device=dev) - spread / 2)
                    s = scale_of(x.abs().amax((2, 3))).float()
                    y = (x / s[..., None, None]).to(E4M3).view(torch.uint8)
                    if T % B:
                        y[-1, :, T % B:] = 0x7f
                    pool[blocks], scale[blocks] = y, s
                pools.append(pool.view(E4M3))
                scales.append(scale)
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
                        max_requests=kw.get("max_requests", max(self.tables.shape[0], 1)),
                        max_blocks_per_req=max(2, self.tables.shape[1]), k_scales=self.ks,
                        v_scales=self.vs)

    def attn(self, cache, **kw):
        return cache.chunk_attn(self.layer, self.q, self.starts, self.tables, self.lengths,
                                self.scale, self.out, req_idx=self.req_idx, **kw)

    def decode(self, cache, **kw):
        return cache.decode(self.layer, self.q.contiguous(), self.tables, self.lengths, self.scale,
                            self.out, req_idx=self.req_idx, **kw)

    def append(self, cache, **kw):
        return cache.append_kv_chunk(self.layer, self.k_new, self.v_new, self.starts, self.tables,
                                     self.lengths, req_idx=self.req_idx, **kw)

    def rows_of(self, i):
        """K and V of request i in token order, [T, Hkv, d], in 64 bits."""
        T = self.spans[i][1]
        blocks = self.tables[self.order[i], :-(-T // B)].long()
        return (values(p[self.layer], s[self.layer], blocks)[:T]
                for p, s in ((self.kp, self.ks), (self.vp, self.vs)))

    def check_attn(self, skip=(), split=2.0 ** -17):
        """The output against 64 bits, within the bound of `attn_ref` (split: of the chunk
        call; 0 for single tokens); the rows of no chunk (and of the requests in `skip`)
        still hold 7."""
        seen = torch.zeros(self.total, dtype=torch.bool, device=self.dev)
        worst = 0.0
        for i, (n, T) in enumerate(self.spans):
            if n == 0 or i in skip:
                continue
            a = int(self.starts_np[i])
            k, v = self.rows_of(i)
            wide = split > 0 and n * (self.Hq // self.Hkv) >= WIDE_ROWS
            want, tol = attn_ref(self.q[a:a + n], k, v, self.scale, split,
                                 2.0 ** -8 if wide else 2.0 ** -11)
            err = (self.out[a:a + n].double() - want).abs()
            assert bool((err <= tol).all()), (
                i, n, T, float((err / tol).nan_to_num(math.inf).max()))
            worst = max(worst, float((err / tol).max()))
            seen[a:a + n] = True
        assert bool((self.out[~seen] == 7.0).all()), "rows of no chunk were written"
        return worst

    def expected_append(self):
        """[(bytes of K, scales of K), (of V)] of the layer after the append."""
        done = []
        for pools, scales, new in ((self.kp, self.ks, self.k_new), (self.vp, self.vs, self.v_new)):
            pool = pools[self.layer].clone().view(torch.uint8).cpu()
            scale = scales[self.layer].clone().cpu()
            new = new.cpu()
            tables = self.tables.cpu()
            for i, (n, T) in enumerate(self.spans):
                t, at = T - n, int(self.starts_np[i])
                while t < T:
                    m = min(T, (t // B + 1) * B) - t
                    b = int(tables[self.order[i], t // B])
                    for h in range(self.Hkv):
                        held = pool[b, h].view(E4M3).double()
                        num, s = put(held, scale[b, h], t % B, new[at:at + m, h])
                        upto = t % B + m
                        pool[b, h, :upto] = num[:upto].float().to(E4M3).view(torch.uint8)
                        scale[b, h] = float(s)
                    t, at = t + m, at + m
            done.append((pool, scale))
        return done

    def check_append(self, want):
        """Numbers and scales as expected, to the byte (a NaN's sign apart), every other byte
        as it was."""
        for (pool, scale), p, s in zip(want, (self.kp, self.vp), (self.ks, self.vs)):
            got = p[self.layer].view(torch.uint8).cpu()
            same = (got == pool) | (((got & 0x7f) == 0x7f) & ((pool & 0x7f) == 0x7f))
            assert bool(same.all()), int((~same).sum())
            got_s = s[self.layer].cpu()
            assert torch.equal(got_s.view(torch.int32), scale.view(torch.int32))


def values(pool, scale, blocks):
    """[tokens, Hkv, d] in 64 bits of blocks of an 8-bit pool."""
    x = pool[blocks].double() * scale[blocks].double()[..., None, None]
    return x.permute(0, 2, 1, 3).flatten(0, 1)


def attn_ref(q, k, v, scale, split=0.0, weight=2.0 ** -11):
    """(out, bound) of one chunk in 64 bits: q [n, Hq, d], k and v [T, Hkv, d] (values).

    The bound counts: the result's rounding to bf16 (half a step, 2^-8 of the value);
    each probability's weight rounded to fp16 for the product with V (`weight`: 2^-11 of
    sum p |v|, or 2^-8 where it is bf16, of long chunks; that while it is at least 2^-14, else half of 2^-24, where the largest is at least 2^5:
    2^-30 of the largest p |v| a key; twice that is taken); the fp32 logit in base 2, a
    sum of d products (d + 2 roundings of 2^-23 -- the matrix unit may truncate -- of scale
    |q| . |k|), times the two scales (4 more) and plus log2 of V's scale, of at
    most 32 (a rounding of 2^-23 of both), which enters a probability and the sum it is
    divided by (twice); with `split` (2^-17: q as two e4m3 numbers, whose steps of 2^-9
    leave half a step of error where the largest element is above 2^7) that part of the
    largest |q| times the sum of |k| in the logit; and 2^-11 of sum p |v| for the exponential (2^-22), the T-term
    fp32 sums and the joining of partial results."""
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
        mag = mag.masked_fill(hidden, 0).amax(1, keepdim=True)
        lost = split * abs(scale) * q[:, hq].abs().amax(1, keepdim=True) * k[:, h].abs().sum(1).max()
        spread = 2 * ((d + 7) * 2.0 ** -23 * mag + 33 * 2.0 ** -23 + lost)
        out[:, hq] = p @ v[:, h]
        pv = p @ v[:, h].abs()
        # the largest weight of a number in the product, a row's
        most = (p * v[:, h].abs().amax(1)[None]).amax(1, keepdim=True)
        tol[:, hq] = (2.0 ** -8 * out[:, hq].abs() + (weight + 2.0 ** -11 + spread) * pv +
                      T * 2.0 ** -29 * most)
    return out, tol


def filter_ref(x, t=1.0, k=0, p=1.0, m=0.0):
    """Kept weights of one row of logits (numpy, 64 bits), in index order."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    by = np.argsort(-x, kind="stable")
    top = x[by[0]]
    if t == 0.0:
        by, t = by[:1], 1.0
    if 0 < k < len(x):
        by = by[:int(k)]
    with np.errstate(invalid="ignore"):
        w = np.where(x[by] == top, 1.0, np.exp((x[by] - top) / t))
    w = np.nan_to_num(w)
    if p < 1.0:
        c = np.cumsum(w)
        n = max(1, int(np.searchsorted(c, p * c[-1], side="left")) + 1)
        by, w = by[:n], w[:n]
    keep = w >= min(m, 1.0)
    out = np.zeros(len(x))
    out[by[keep]] = w[keep]
    return out


def draw_ref(w, u):
    """The lowest index whose running sum exceeds u times all."""
    c = np.cumsum(w)
    return int(np.argmax(c > u * c[-1]))


def border(w, u):
    """How near u times all lies to a border between tokens, relative to all."""
    c = np.cumsum(w)
    return float(np.abs(c - u * c[-1]).min() / c[-1])
