"""The operators of a decode step over an 8-bit cache as measured workloads: new
keys and values rounded into it, the attention that reads it, and the next
token drawn from logits, or their filtered probabilities for the verification
of drafted tokens.

``run`` makes the calls a user of the library makes when ``own`` is true and
computes the same operators from elementary torch operations when it is false.

The 8-bit cache holds e4m3 numbers (3 bits of mantissa, up to 448) and one scale
for each block of 16 tokens and kv head, K and V apart: value = scale * number.
Request i brings n_i new tokens, packed one request after the other (rows
starts[i] .. starts[i+1]-1), and afterwards holds T_i = lengths[i] cached
tokens, the new ones being the last n_i of them.

  append  a block's scale is the least power of two (2^-32 .. 2^32) that takes its
          new rows into +-448; a block that holds tokens already keeps its scale if
          that one is larger, else they are rounded again to the new one
  attn    out = sum_t softmax_t(scale q . k_t) v_t over t <= the token's own
          position, query head hq reading kv head hq / (Hq / Hkv)
  sample  weights exp((l - max l) / temperature), the largest logit alone for a
          temperature of 0; kept are the top_k largest logits (0: all), of these the
          shortest run of the largest whose sum reaches top_p of theirs, of these the
          weights of at least min_p; equal logits count from the lowest index on.  The
          token is the lowest kept index whose running sum exceeds u times all
  probs   the kept weights over their sum, 0 elsewhere
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16
MAX_TOKENS = 32768      # longest request the admission path takes
E4M3_MAX = 448.0


# ------------------------------------------------------------------- the cases

def _cached(op, name, R, n, ctx, heads, d):
    return {"name": name, "op": op, "R": R, "n_lo": n[0], "n_hi": n[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "Hkv": heads[0], "Hq": heads[1], "d": d}


def _logits(op, name, R, rows, V, dtype, filters, pad=0):
    return {"name": name, "op": op, "R": R, "rows": rows, "V": V, "dtype": dtype,
            "filters": filters, "pad": pad}


def listed():
    return [
        # the lowest latency: a single stream's next token at the 2048-token budget
        _cached("attn", "decode_one", 1, (1, 1), (2000, 2000), (8, 32), 128),
        # a full batch of single tokens
        _cached("attn", "decode_256", 256, (1, 1), (1024, 2039), (8, 32), 128),
        # a full batch's speculative step
        _cached("attn", "drafts_256", 256, (2, 9), (1024, 2038), (8, 32), 128),
        # admission: whole prompts of ragged lengths, seven query heads on a kv head
        _cached("attn", "prompts", 16, (331, 4007), (0, 0), (4, 28), 64),
        # one piece of a long prompt over what is already cached
        _cached("attn", "long_chunk", 1, (2048, 2048), (30001, 30001), (8, 32), 128),
        # new rows of a decode step: blocks that hold tokens already
        _cached("append", "append_256", 256, (1, 1), (1024, 2039), (8, 32), 128),
        # new rows of admitted prompts: whole blocks
        _cached("append", "append_prompts", 16, (331, 4007), (0, 0), (8, 32), 128),
        # a single stream with a small vocabulary: the smallest call
        _logits("sample", "sample_one", 1, 1, 32000, "f32", "p"),
        # a full batch without filters: every weight counts
        _logits("sample", "sample_all_256", 256, 1, 151936, "f32", "none"),
        # requests with filters of their own, an odd vocabulary, 16-bit logits
        _logits("sample", "sample_mixed_96", 96, 1, 50257, "bf16", "mixed"),
        # a small batch's speculative step, 16-bit logits in padded rows
        _logits("probs", "probs_8", 8, 5, 128000, "bf16", "mixed", 64),
        # the largest: a full batch's speculative step, a large vocabulary
        _logits("probs", "probs_256", 256, 5, 151936, "f32", "mixed"),
    ]


def _spans(case):
    """(n_i, T_i) of every request: spread over their ranges, the same for every seed."""
    out = []
    for i in range(case["R"]):
        f = (i + 1) * 0.6180339887498949 % 1.0
        g = (i + 1) * 0.7548776662466927 % 1.0
        n = case["n_lo"] + int(f * (case["n_hi"] - case["n_lo"] + 1))
        out.append((n, n + case["ctx_lo"] + int(g * (case["ctx_hi"] - case["ctx_lo"] + 1))))
    return out


def work(case):
    if case["op"] in ("sample", "probs"):
        total = case["R"] * case["rows"]
        b = total * case["V"] * (4 if case["dtype"] == "f32" else 2) + case["R"] * 16
        if case["op"] == "probs":
            return {"bytes": b + 4 * total * case["V"], "flops": 3.0 * total * case["V"]}
        return {"bytes": b + 8 * total, "flops": 3.0 * total * case["V"]}
    spans = _spans(case)
    new = sum(n for n, _ in spans)
    Hkv, Hq, d = case["Hkv"], case["Hq"], case["d"]
    if case["op"] == "append":
        # the new rows in 16 bits, the blocks they touch in 8; of blocks that hold
        # tokens already those are not read where the scale stays
        blocks = sum((T - 1) // BLOCK - (T - n) // BLOCK + 1 for n, T in spans)
        return {"bytes": 2 * Hkv * (new * d * (2 + 1) + 4 * blocks) + 8 * case["R"], "flops": 0}
    seen = sum(n * T - n * (n - 1) // 2 for n, T in spans)
    blocks = sum(-(-T // BLOCK) for _, T in spans)
    return {"bytes": 2 * Hkv * (sum(T for _, T in spans) * d + 4 * blocks) + 4 * new * Hq * d,
            "flops": 4 * d * Hq * seen}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = {}
    for c in listed():
        for k, v in work(c).items():
            top[c["op"], k] = max(top.get((c["op"], k), 0), v)
    op = rng.choice(["attn", "attn", "attn", "append", "sample", "sample", "probs"])
    while True:
        if op in ("sample", "probs"):
            c = _logits(op, "", _log(rng, 1, 256), 1 if op == "sample" else rng.randint(1, 8),
                        _log(rng, 1000, 152000), rng.choice(["f32", "bf16"]),
                        rng.choice(["none", "k", "p", "mixed", "mixed"]),
                        rng.choice([0, 0, 1, 64]))
        else:
            hkv, g = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16])
            n_lo = rng.choice([1, _log(rng, 1, 4096)])
            n_hi = n_lo + (0 if n_lo == 1 and rng.random() < 0.7 else rng.randint(0, n_lo))
            ctx = rng.choice([0, _log(rng, 1, 30000)])
            c = _cached(op, "", _log(rng, 1, 256), (n_lo, n_hi), (ctx // 2, ctx), (hkv, hkv * g),
                        rng.choice([64, 128]))
            if c["n_hi"] + c["ctx_hi"] > MAX_TOKENS or sum(n for n, _ in _spans(c)) > 65536:
                continue
        w = work(c)
        if all(w[k] <= top[op, k] for k in w):
            del c["name"]
            return c


# ------------------------------------------------------------------- the inputs

def _scale_of(most):
    """The least power of two, 2^-32 .. 2^32, that takes `most` into 448."""
    m, e = torch.frexp(most)
    return torch.ldexp(torch.ones_like(most), (e - 9 + (m > 0.875).int()).clamp(-32, 32))


def _rounded(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 29)
    rnd = random.Random(seed * 7919 + 5)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    if case["op"] in ("sample", "probs"):
        R, V = case["R"], case["V"]
        total = R * case["rows"]
        dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        logits = torch.zeros(total, V + case["pad"], device="cuda", dtype=dtype)
        for a in range(0, total, 64):
            b = min(total, a + 64)
            # from flat rows to peaked ones; a few tokens far ahead in half of them
            x = randn(b - a, V) * (1.0 + 3.0 * rand(b - a, 1))
            ahead = (rand(b - a, V) < 8.0 / V) & (rand(b - a, 1) < 0.5)
            logits[a:b, :V] = torch.where(ahead, x + 10.0, x).to(dtype)
        # filters of each request: temperature, top_k (0: off), top_p (1: off), min_p (0: off)
        kind = case["filters"]
        t, k, p, m = [], [], [], []
        for i in range(R):
            t.append(rnd.choice([0.6, 0.8, 1.0, 1.0, 1.3]))
            k.append(rnd.choice([1, 20, 50, 50, 200]) if kind in ("k", "mixed") else 0)
            p.append(rnd.choice([0.5, 0.8, 0.9, 0.95]) if kind in ("p", "mixed") else 1.0)
            m.append(rnd.choice([0.0, 0.02, 0.1]) if kind == "mixed" else 0.0)
            if kind == "mixed":  # some requests use only a part of them, or are greedy
                off = rnd.randint(0, 9)
                k[i], p[i] = (0 if off < 5 else k[i]), (1.0 if off in (0, 5, 6) else p[i])
                t[i] = 0.0 if off == 9 else t[i]
        rows = torch.arange(R, device="cuda").repeat_interleave(case["rows"])
        return {"case": case, "logits": logits[:, :V], "req_idx": rows.to(torch.int32),
                "temperature": torch.tensor(t, device="cuda"),
                "top_k": torch.tensor(k, device="cuda", dtype=torch.int32),
                "top_p": torch.tensor(p, device="cuda"), "min_p": torch.tensor(m, device="cuda"),
                "u": rand(total)}

    spans = _spans(case)
    R, Hkv, Hq, d = case["R"], case["Hkv"], case["Hq"], case["d"]
    total = sum(n for n, _ in spans)
    need = [-(-T // BLOCK) for _, T in spans]
    num_blocks = sum(need) + 8
    ids = list(range(num_blocks))
    rnd.shuffle(ids)
    tables = np.full((R, max(need) + 1), -1, np.int32)
    at = 0
    for i, m in enumerate(need):
        tables[i, :m] = ids[at:at + m]
        at += m
    # keys with 1 % heavy hitters (8 times the norm), a common offset a head
    k = randn(num_blocks, Hkv, BLOCK, d)
    heavy = rand(num_blocks, Hkv, BLOCK, 1) < 0.01
    k = torch.where(heavy, k * 8, k) + 0.5 * randn(1, Hkv, 1, d)
    v = randn(num_blocks, Hkv, BLOCK, d)
    scales = [_scale_of(x.abs().amax((2, 3))) for x in (k, v)]
    pools = [_rounded(x / s[..., None, None]) for x, s in zip((k, v), scales)]
    starts = np.concatenate([[0], np.cumsum([n for n, _ in spans])]).astype(np.int32)
    qkv = randn(total, Hq + 2 * Hkv, d, dtype=torch.bfloat16)
    if case["n_hi"] == 1:  # a decode step's are contiguous
        q, k_new, v_new = (x.contiguous() for x in qkv.split([Hq, Hkv, Hkv], 1))
    else:                  # slices of the projection's packed output
        q, k_new, v_new = qkv.split([Hq, Hkv, Hkv], 1)
    return {"case": case, "spans": spans, "k_pool": pools[0], "v_pool": pools[1],
            "k_scale": scales[0], "v_scale": scales[1], "tables": torch.from_numpy(tables).cuda(),
            "lengths": torch.tensor([T for _, T in spans], dtype=torch.int32, device="cuda"),
            "starts": torch.from_numpy(starts).cuda(), "q": q, "k": k_new, "v": v_new,
            "scale": d ** -0.5}


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "sample":
        s["tokens"] = torch.zeros(case["R"], dtype=torch.int32, device="cuda")
    elif case["op"] == "probs":
        s["probs"] = torch.zeros(s["logits"].shape, device="cuda")
    elif case["op"] == "attn":
        s["out"] = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    if own:
        from compressed_paged_kv_gb300 import zp
        if case["op"] in ("sample", "probs"):  # the decoding cache's handle; its pools play no part
            pool = torch.zeros(1, 1, BLOCK, 64, dtype=torch.bfloat16, device="cuda")
            s["cache"] = zp.Cache([pool], [pool.clone()], 1, max_requests=case["R"],
                                  max_blocks_per_req=2)
        else:
            s["cache"] = zp.Cache([s["k_pool"]], [s["v_pool"]], case["Hq"],
                                  max_requests=case["R"],
                                  max_blocks_per_req=max(2, s["tables"].shape[1]),
                                  k_scales=[s["k_scale"]], v_scales=[s["v_scale"]])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        cache = s["cache"]
        if op == "sample":
            cache.sample(s["logits"], s["u"], s["tokens"], s["temperature"], top_k=s["top_k"],
                         top_p=s["top_p"], min_p=s["min_p"])
            return s["tokens"]
        if op == "probs":
            cache.token_probs(s["logits"], s["probs"], s["temperature"], top_k=s["top_k"],
                              top_p=s["top_p"], min_p=s["min_p"], req_idx=s["req_idx"])
            return s["probs"]
        if op == "append":
            if case["n_hi"] == 1:
                cache.append_kv(0, s["k"], s["v"], s["tables"], s["lengths"])
            else:
                cache.append_kv_chunk(0, s["k"], s["v"], s["starts"], s["tables"], s["lengths"])
            return [s["k_pool"], s["k_scale"], s["v_pool"], s["v_scale"]]
        if case["n_hi"] == 1:
            cache.decode(0, s["q"], s["tables"], s["lengths"], s["scale"], s["out"])
        else:
            cache.chunk_attn(0, s["q"], s["starts"], s["tables"], s["lengths"], s["scale"],
                             s["out"])
        return s["out"]
    return {"sample": _plain_sample, "probs": _plain_probs, "append": _plain_append,
            "attn": _plain_attn}[op](s)


def _plain_append(s):
    # touched block by touched block: the request, the block of it, the slots that are new
    ends, n = s["lengths"].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    lo = (ends - n) // BLOCK
    touched = torch.where(n > 0, (ends - 1) // BLOCK - lo + 1, 0)
    req = torch.repeat_interleave(torch.arange(len(n), device="cuda"), touched)
    nth = torch.arange(len(req), device="cuda") - (touched.cumsum(0) - touched)[req]
    index = lo[req] + nth
    block = s["tables"][req, index].long()
    pos = index[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    first = (ends - n)[req][:, None]
    new = (pos >= first) & (pos < ends[req][:, None])
    src = (s["starts"][:-1].long()[req][:, None] + pos - first).clamp(0, len(s["k"]) - 1)
    for pool, scale, x in ((s["k_pool"], s["k_scale"], s["k"]), (s["v_pool"], s["v_scale"], s["v"])):
        x = x[src].float().transpose(1, 2)                       # [touched, Hkv, 16, d]
        is_new = new[:, None, :, None]
        held, before = pool[block].float(), scale[block]
        begun = (first > index[:, None] * BLOCK)                 # holds tokens already
        want = _scale_of((x * is_new).abs().amax((2, 3)))
        want = torch.where(begun, torch.maximum(want, before), want)
        old = (pos < first)[:, None, :, None]
        held = torch.where(old, held * (before / want)[..., None, None], held)
        pool[block] = _rounded(torch.where(is_new, x / want[..., None, None], held))
        scale[block] = want
    return [s["k_pool"], s["k_scale"], s["v_pool"], s["v_scale"]]


def _plain_attn(s):
    c = s["case"]
    Hkv, G, d = c["Hkv"], c["Hq"] // c["Hkv"], c["d"]
    n, T = max(n for n, _ in s["spans"]), max(T for _, T in s["spans"])
    # requests whose padded scores and rows are held at once, and kv heads of them
    step = max(1, (1 << 29) // (Hkv * T * max(G * n, 2 * d)))
    heads = Hkv if step > 1 else max(1, min(Hkv, (1 << 29) // (T * max(G * n, 2 * d))))
    for a in range(0, c["R"], step):
        spans = s["spans"][a:a + step]
        n, T = max(n for n, _ in spans), max(T for _, T in spans)
        starts, ends = s["starts"][a:a + len(spans) + 1].long(), s["lengths"][a:a + len(spans)]
        count = starts[1:] - starts[:-1]
        at = torch.arange(n, device="cuda")
        live = at < count[:, None]
        rows = (starts[:-1, None] + at).clamp_(max=len(s["q"]) - 1)
        q = s["q"][rows].float().reshape(len(spans), n, Hkv, G, d).permute(0, 2, 3, 1, 4)
        blocks = s["tables"][a:a + len(spans), :-(-T // BLOCK)].long().clamp_(min=0)
        t = torch.arange(T, device="cuda")
        pos = (ends - count)[:, None] + at
        hidden = (t > pos[..., None]) & live[..., None]          # [requests, n, T]
        gone = (t >= ends[:, None])[:, None, :, None]
        for h in range(0, Hkv, heads):
            k, v = ((pool[blocks, h:h + heads].float() * scale[blocks, h:h + heads][..., None, None])
                    .transpose(1, 2).flatten(2, 3)[:, :, :T].masked_fill(gone, 0.0)
                    for pool, scale in ((s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"])))
            w = torch.matmul(q[:, h:h + heads].flatten(2, 3), k.transpose(-1, -2)) * s["scale"]
            w = w.unflatten(2, (G, n)).masked_fill_(hidden[:, None, None], -math.inf)
            w = torch.exp(w - w.amax(-1, keepdim=True))
            o = torch.matmul(w.flatten(2, 3), v).unflatten(2, (G, n)) / w.sum(-1, keepdim=True)
            o = o.permute(0, 3, 1, 2, 4)[live].flatten(1, 2)
            s["out"][rows[live], h * G:(h + heads) * G] = o.to(torch.bfloat16)
    return s["out"]


def _plain_weights(s, a, b):
    """The kept weights of logit rows a .. b-1, 0 elsewhere."""
    at = s["req_idx"][a:b].long()
    t, k, p, m = (s[x][at][:, None] for x in ("temperature", "top_k", "top_p", "min_p"))
    x, index = torch.sort(s["logits"][a:b].float(), dim=1, descending=True, stable=True)
    w = torch.exp((x.double() - x[:, :1].double()) / torch.where(t > 0, t, 1.0).double())
    rank = torch.arange(x.shape[1], device="cuda")
    w *= (rank < torch.where(k > 0, k, x.shape[1])) & ((t > 0) | (rank == 0))
    total = w.cumsum(1)
    # kept while the sum before it is short of top_p of all
    w[:, 1:] *= (total[:, :-1] < p.double() * total[:, -1:]) | (p >= 1)
    w *= w >= m.double()
    return torch.zeros_like(w).scatter_(1, index, w)


def _plain_sample(s):
    for a in range(0, s["case"]["R"], 256):
        b = min(s["case"]["R"], a + 256)
        total = _plain_weights(s, a, b).cumsum(1)
        level = s["u"][a:b, None].double() * total[:, -1:]
        s["tokens"][a:b] = torch.searchsorted(total, level, right=True)[:, 0].int()
    return s["tokens"]


def _plain_probs(s):
    for a in range(0, len(s["logits"]), 256):
        w = _plain_weights(s, a, a + 256)
        s["probs"][a:a + 256] = (w / w.sum(1, keepdim=True)).float()
    return s["probs"]


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("sample", "probs"):
        out = []
        for i in range(len(s["logits"])):
            r = int(s["req_idx"][i])
            x = s["logits"][i].double()
            t, k = float(s["temperature"][r]), int(s["top_k"][r])
            p, m = float(s["top_p"][r]), float(s["min_p"][r])
            # falling, equal ones by index
            by = torch.argsort(-x, stable=True)
            if t == 0.0:
                by = by[:1]
                w = torch.ones(1, dtype=torch.float64, device="cuda")
            else:
                by = by[:k] if k > 0 else by
                w = ((x[by] - x[by[0]]) / t).exp()
                if p < 1.0:
                    run_sum = torch.cumsum(w, 0)
                    # the first place where the sum reaches its part
                    n = int((run_sum < p * run_sum[-1]).sum()) + 1
                    by, w = by[:n], w[:n]
                by, w = by[w >= m], w[w >= m]
            whole = torch.zeros_like(x)
            whole[by] = w
            if case["op"] == "probs":
                out.append(whole / whole.sum())
                continue
            run_sum = whole.cumsum(0)
            out.append((run_sum > float(s["u"][i]) * run_sum[-1]).int().argmax())
        return torch.stack(out) if case["op"] == "probs" else torch.stack(out).int()
    Hkv, G, d = case["Hkv"], case["Hq"] // case["Hkv"], case["d"]
    if case["op"] == "append":
        tables = s["tables"].cpu().numpy()
        done = []
        for name, x in (("k", s["k"]), ("v", s["v"])):
            pool, scale = s[name + "_pool"].double(), s[name + "_scale"].double()
            at = 0
            for i, (n, T) in enumerate(s["spans"]):
                t = T - n
                while t < T:  # block after block
                    m = min(T, (t // BLOCK + 1) * BLOCK) - t
                    b, o = int(tables[i, t // BLOCK]), t % BLOCK
                    rows = x[at:at + m].transpose(0, 1).double()  # [Hkv, m, d]
                    most = rows.abs().amax((1, 2)).clamp(min=2.0 ** -60)
                    e = torch.log2(most / E4M3_MAX).ceil().clamp(-32, 32)
                    want = torch.exp2(e)
                    if o:
                        want = torch.maximum(want, scale[b])
                        pool[b, :, :o] = _e4m3(pool[b, :, :o] * (scale[b] / want)[:, None, None])
                    pool[b, :, o:o + m] = _e4m3(rows / want[:, None, None])
                    scale[b] = want
                    t, at = t + m, at + m
            done += [pool, scale]
        return done
    # attention, one kv head of one request at a time
    if work(case)["flops"] > 4e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    a = 0
    for i, (n, T) in enumerate(s["spans"]):
        blocks = s["tables"][i].long()[:(T + BLOCK - 1) // BLOCK]
        for h in range(Hkv):
            k, v = ((s[x + "_pool"][blocks, h].double() *
                     s[x + "_scale"][blocks, h].double()[:, None, None]).reshape(-1, d)[:T]
                    for x in ("k", "v"))
            for part in range(0, n, 4096):
                m = min(n - part, 4096)
                q = s["q"][a + part:a + part + m, h * G:(h + 1) * G].double()
                x = torch.einsum("ngd,td->ngt", q, k) * s["scale"]
                first = T - n + part + 1  # keys the part's first token sees
                sees = torch.arange(first, first + m, device="cuda")
                x = torch.where(torch.arange(T, device="cuda") < sees[:, None, None], x,
                                -torch.inf)
                out[a + part:a + part + m, h * G:(h + 1) * G] = torch.einsum(
                    "ngt,td->ngd", torch.softmax(x, -1), v)
        a += n
    return out


def _e4m3(x):
    """x rounded to an e4m3 number: ties to even, steps of 2^-9 below 2^-6."""
    e = torch.frexp(x)[1].clamp(min=-5) - 4  # of the last bit that is kept
    step = torch.exp2(e.double())
    return ((x / step).round() * step).clamp(-E4M3_MAX, E4M3_MAX)
