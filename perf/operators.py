"""The chunked-serving operators as measured workloads: a ragged chunk of new
tokens written into the paged cache, its attention over the cache, and the
verification of drafted tokens against the target's probabilities.

``run`` makes the calls a user of the library makes when ``own`` is true and
computes the same operators from elementary torch operations when it is false.

A batch holds R requests; request i brings a chunk of n_i new tokens, packed
one request after the other (chunk i is rows starts[i] .. starts[i+1]-1 of
every packed tensor), and afterwards holds T_i = lengths[i] cached tokens, the
chunk being the last n_i of them.

  append  K/V rows of the chunk into the slots the block tables name
  attn    out = sum_t softmax_t(scale q . k_t) v_t over t <= the token's own
          position, query head hq reading kv head hq / (Hq / Hkv)
  verify  chunk token j+1 (a drafted one) is accepted when all before it are
          and u q(x) < p(x); the first rejected position (or the one after the
          last token) is sampled from max(p - q, 0) (or from p)
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16
MAX_TOKENS = 32768      # longest request the admission path takes


# ------------------------------------------------------------------- the cases

def _attn(name, R, chunks, n, ctx, heads, d, packed=True):
    return {"name": name, "op": "attn", "R": R, "chunks": chunks, "n_lo": n[0], "n_hi": n[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "Hkv": heads[0], "Hq": heads[1], "d": d,
            "packed": packed}


def _append(name, R, chunks, n, ctx, heads, d, packed=True):
    return dict(_attn(name, R, chunks, n, ctx, heads, d, packed), op="append")


def _verify(name, R, drafts, V, dtype, draft, pad):
    return {"name": name, "op": "verify", "R": R, "k_lo": drafts[0], "k_hi": drafts[1], "V": V,
            "dtype": dtype, "draft": draft, "pad": pad}


def listed():
    return [
        # the lowest latency: one short request, its last token and four drafted ones
        _attn("attn_one_short", 1, 1, (5, 5), (100, 100), (2, 4), 64),
        # a speculative step of a small batch at the 2048-token budget
        _attn("attn_drafts_8", 8, 8, (5, 5), (1024, 2040), (8, 32), 128),
        # the same for a full batch, ragged draft lengths: every cached row is read once
        _attn("attn_drafts_256", 256, 256, (2, 9), (1024, 2038), (8, 32), 128),
        # admission: whole prompts of ragged lengths, nothing cached before them
        _attn("attn_prompts", 16, 16, (331, 4007), (0, 0), (8, 32), 128),
        # one piece of a long prompt over what is already cached
        _attn("attn_long_chunk", 1, 1, (2048, 2048), (30001, 30001), (8, 32), 128),
        # a continuous batch: two prompt pieces beside sixty single tokens, seven
        # query heads on a kv head
        _attn("attn_mixed_64", 62, 2, (700, 1100), (333, 1900), (4, 28), 64, packed=False),
        # new rows of a speculative step
        _append("append_drafts_8", 8, 8, (5, 5), (1024, 2040), (8, 32), 128),
        # new rows of admitted prompts
        _append("append_prompts", 16, 16, (331, 4007), (0, 0), (8, 32), 128),
        # a single stream with a small vocabulary
        _verify("verify_one", 1, (4, 4), 32000, "f32", True, 0),
        # a batch with an odd vocabulary: rows that start at any 4-byte address
        _verify("verify_odd_48", 48, (1, 7), 50257, "f32", True, 0),
        # the largest: a full batch, a large vocabulary
        _verify("verify_256", 256, (4, 4), 151936, "f32", True, 0),
        # tokens proposed without probabilities (looked up), 16-bit target rows padded
        _verify("verify_lookup_128", 128, (2, 6), 128000, "bf16", False, 64),
    ]


def _spans(case):
    """(n_i, T_i) of every request: spread over their ranges, the same for every seed."""
    out = []
    for i in range(case["R"]):
        f = (i + 1) * 0.6180339887498949 % 1.0
        g = (i + 1) * 0.7548776662466927 % 1.0
        n = case["n_lo"] + int(f * (case["n_hi"] - case["n_lo"] + 1))
        if i >= case["chunks"]:
            n = 1
        out.append((n, n + case["ctx_lo"] + int(g * (case["ctx_hi"] - case["ctx_lo"] + 1))))
    return out


def _counts(case):
    """Chunk tokens of every request of a verification: the last accepted one and its drafts."""
    return [1 + case["k_lo"] + int((i + 1) * 0.6180339887498949 % 1.0 *
                                   (case["k_hi"] - case["k_lo"] + 1)) for i in range(case["R"])]


def work(case):
    if case["op"] == "verify":
        # only the row that decides the next token is needed whole; an eighth of the
        # drafted tokens or so is rejected, then the draft's row is needed as well
        esz = 4 if case["dtype"] == "f32" else 2
        total = sum(_counts(case))
        rows = 0.0
        for n in _counts(case):
            rows += 1.0 + ((1.0 - 0.88 ** (n - 1)) if case["draft"] else 0.0)
        return {"bytes": rows * case["V"] * esz + total * (8 + 2 * esz) + case["R"] * 16,
                "flops": 2.0 * rows * case["V"]}
    spans = _spans(case)
    new = sum(n for n, _ in spans)
    row = case["d"] * 2
    if case["op"] == "append":
        return {"bytes": 4 * new * case["Hkv"] * row + 8 * case["R"], "flops": 0}
    seen = sum(n * T - n * (n - 1) // 2 for n, T in spans)
    return {"bytes": 2 * sum(T for _, T in spans) * case["Hkv"] * row + 2 * new * case["Hq"] * row,
            "flops": 4 * case["d"] * case["Hq"] * seen}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = {}
    for c in listed():
        for k, v in work(c).items():
            top[c["op"], k] = max(top.get((c["op"], k), 0), v)
    op = rng.choice(["attn", "attn", "attn", "append", "verify", "verify"])
    while True:
        if op == "verify":
            k_lo = rng.randint(0, 6)
            c = _verify("", _log(rng, 1, 256), (k_lo, k_lo + rng.randint(0, 6)),
                        _log(rng, 1000, 152000), rng.choice(["f32", "bf16"]),
                        rng.random() < 0.7, rng.choice([0, 0, 1, 64]))
        else:
            hkv, g = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16])
            n_lo = _log(rng, 1, 4096)
            ctx = rng.choice([0, _log(rng, 1, 30000)])
            R = _log(rng, 1, 256)
            c = _attn("", R, R if rng.random() < 0.7 else rng.randint(0, R),
                      (n_lo, n_lo + rng.randint(0, n_lo)), (ctx // 2, ctx), (hkv, hkv * g),
                      rng.choice([64, 128]), rng.random() < 0.5)
            if op == "append":
                c["op"] = "append"
            if c["n_hi"] + c["ctx_hi"] > MAX_TOKENS or sum(n for n, _ in _spans(c)) > 65536:
                continue
        w = work(c)
        if all(w[k] <= top[op, k] for k in w):
            del c["name"]
            return c


# ------------------------------------------------------------------- the inputs

def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 17)
    rnd = random.Random(seed * 7919 + 3)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    if case["op"] == "verify":
        counts = _counts(case)
        total, R, V = sum(counts), case["R"], case["V"]
        stride = V + case["pad"]
        dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        starts = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
        # peaked target rows; the draft's logits are the target's with some noise
        target = torch.zeros(total, stride, device="cuda", dtype=dtype)
        draft = torch.zeros(total, stride, device="cuda", dtype=dtype) if case["draft"] else None
        picked = torch.empty(total, device="cuda", dtype=torch.int64)
        for a in range(0, total, 64):
            b = min(total, a + 64)
            logits = 3.0 * randn(b - a, V)
            noisy = logits + 0.4 * randn(b - a, V)
            target[a:b, :V] = torch.softmax(logits, 1).to(dtype)
            q = torch.softmax(noisy, 1)
            if draft is not None:
                draft[a:b, :V] = q.to(dtype)
                picked[a:b] = torch.multinomial(draft[a:b, :V].float(), 1, generator=gen)[:, 0]
            else:  # the likeliest token of a sharpened row: accepted fairly often
                target[a:b, :V] = torch.softmax(1.7 * logits, 1).to(dtype)
                picked[a:b] = noisy.argmax(1)
        # the token drafted at row j is the chunk's token j + 1
        tokens = torch.randint(0, V, (total,), generator=gen, device="cuda")
        inner = torch.ones(total, dtype=torch.bool)
        inner[starts[:-1].long()] = False
        inner = inner.nonzero()[:, 0].cuda()
        tokens[inner] = picked[inner - 1]
        return {"case": case, "starts": starts.cuda(), "tokens": tokens.to(torch.int32),
                "target": target[:, :V], "draft": None if draft is None else draft[:, :V],
                "accept_u": torch.rand(total, generator=gen, device="cuda"),
                "sample_u": torch.rand(R, generator=gen, device="cuda"),
                "counts": counts}

    spans = _spans(case)
    R, Hkv, Hq, d = case["R"], case["Hkv"], case["Hq"], case["d"]
    total = sum(n for n, _ in spans)
    need = [-(-T // BLOCK) for _, T in spans]
    width = max(need) + 1
    num_blocks = sum(need) + 8
    ids = list(range(num_blocks))
    rnd.shuffle(ids)
    tables = np.full((R, width), -1, np.int32)
    at = 0
    for i, m in enumerate(need):
        tables[i, :m] = ids[at:at + m]
        at += m
    # keys with 1 % heavy hitters (8 times the norm), a common offset a head
    k_pool = randn(num_blocks, Hkv, BLOCK, d, dtype=torch.bfloat16)
    heavy = torch.rand(num_blocks, Hkv, BLOCK, 1, generator=gen, device="cuda") < 0.01
    k_pool = torch.where(heavy, k_pool * 8, k_pool)
    k_pool += 0.5 * randn(1, Hkv, 1, d, dtype=torch.bfloat16)
    v_pool = randn(num_blocks, Hkv, BLOCK, d, dtype=torch.bfloat16)
    starts = np.concatenate([[0], np.cumsum([n for n, _ in spans])]).astype(np.int32)
    # the projection's packed output [token][Hq + 2 Hkv][d], or separate tensors
    if case["packed"]:
        qkv = randn(total, Hq + 2 * Hkv, d, dtype=torch.bfloat16)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = (randn(total, h, d, dtype=torch.bfloat16) for h in (Hq, Hkv, Hkv))
    return {"case": case, "spans": spans, "k_pool": k_pool, "v_pool": v_pool,
            "tables": torch.from_numpy(tables).cuda(),
            "lengths": torch.tensor([T for _, T in spans], dtype=torch.int32, device="cuda"),
            "starts": torch.from_numpy(starts).cuda(), "q": q, "k": k, "v": v,
            "scale": d ** -0.5}


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "verify":
        R = case["R"]
        s["accepted"] = torch.zeros(R, dtype=torch.int32, device="cuda")
        s["next"] = torch.zeros(R, dtype=torch.int32, device="cuda")
    elif case["op"] == "attn":
        s["out"] = torch.zeros(s["q"].shape[0], case["Hq"], case["d"], dtype=torch.bfloat16,
                               device="cuda")
    if own:
        from compressed_paged_kv_gb300 import zp
        if case["op"] == "verify":  # the decoding cache's handle; its pools play no part
            pool = torch.zeros(1, 1, BLOCK, 64, dtype=torch.bfloat16, device="cuda")
            s["cache"] = zp.Cache([pool], [pool.clone()], 1, max_requests=case["R"],
                                  max_blocks_per_req=2)
        else:
            s["cache"] = zp.Cache([s["k_pool"]], [s["v_pool"]], case["Hq"],
                                  max_requests=case["R"],
                                  max_blocks_per_req=max(2, s["tables"].shape[1]))
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        cache = s["cache"]
        if op == "verify":
            cache.verify_draft(s["tokens"], s["starts"], s["target"], s["accept_u"],
                               s["sample_u"], s["accepted"], s["next"], draft_probs=s["draft"])
            return [s["accepted"], s["next"]]
        if op == "append":
            cache.append_kv_chunk(0, s["k"], s["v"], s["starts"], s["tables"], s["lengths"])
            return [s["k_pool"], s["v_pool"]]
        cache.chunk_attn(0, s["q"], s["starts"], s["tables"], s["lengths"], s["scale"], s["out"])
        return s["out"]
    return {"verify": _plain_verify, "append": _plain_append, "attn": _plain_attn}[op](s)


def _plain_append(s):
    total = s["k"].shape[0]
    at = torch.arange(total, device="cuda", dtype=torch.int32)
    req = torch.searchsorted(s["starts"], at, right=True) - 1
    pos = s["lengths"][req] - s["starts"][req + 1] + at
    block = s["tables"][req, pos // BLOCK].long()
    s["k_pool"][block, :, pos.long() % BLOCK] = s["k"]
    s["v_pool"][block, :, pos.long() % BLOCK] = s["v"]
    return [s["k_pool"], s["v_pool"]]


def _plain_attn(s):
    c = s["case"]
    Hkv, G, d = c["Hkv"], c["Hq"] // c["Hkv"], c["d"]
    a = 0
    for i, (n, T) in enumerate(s["spans"]):
        blocks = s["tables"][i, :-(-T // BLOCK)].long()
        k = s["k_pool"][blocks].permute(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :T].float()
        v = s["v_pool"][blocks].permute(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :T].float()
        q = s["q"][a:a + n].reshape(n, Hkv, G, d).permute(1, 2, 0, 3).float()
        hidden = None
        if n > 1:
            t = torch.arange(T, device="cuda")
            hidden = t[None, :] > t[T - n:, None]
        step = max(1, (1 << 29) // (G * n * T))  # kv heads whose scores are held at once
        for h in range(0, Hkv, step):
            w = torch.matmul(q[h:h + step], k[h:h + step, None].transpose(-1, -2)) * s["scale"]
            if hidden is not None:
                w.masked_fill_(hidden, -math.inf)
            w = torch.exp(w - w.amax(-1, keepdim=True))
            o = torch.matmul(w, v[h:h + step, None]) / w.sum(-1, keepdim=True)
            o = o.permute(2, 0, 1, 3).reshape(n, -1, d)
            s["out"][a:a + n, h * G:h * G + o.shape[1]] = o.to(torch.bfloat16)
        a += n
    return s["out"]


def _plain_verify(s):
    starts, R = s["starts"].long(), s["case"]["R"]
    n = max(s["counts"])
    # row starts[i] + j judges the chunk's token j + 1; all chunks padded to the longest
    j = torch.arange(n - 1, device="cuda")
    row = (starts[:-1, None] + j).clamp_(max=s["tokens"].numel() - 2) if n > 1 else None
    accepted = torch.zeros(R, dtype=torch.int64, device="cuda")
    drafts = starts[1:] - starts[:-1] - 1
    if n > 1:
        x = s["tokens"].long()[row + 1]
        u = s["accept_u"][row].double()
        p = s["target"][row, x].double()
        q = s["draft"][row, x].double() if s["draft"] is not None else torch.ones_like(p)
        ok = (u * q < p) & (j < drafts[:, None])
        accepted = torch.cumprod(ok.long(), 1).sum(1)
    last = starts[:-1] + accepted
    rejected = accepted < drafts
    p = s["target"][last].double()
    if s["draft"] is not None:
        w = (p - s["draft"][last].double() * rejected[:, None]).clamp_(min=0)
    else:
        x = s["tokens"].long()[torch.where(rejected, last + 1, last)]
        w = p
        w[torch.arange(R, device="cuda"), x] *= (~rejected).double()
    total = w.cumsum(1)
    level = s["sample_u"].double() * total[:, -1]
    s["accepted"].copy_(accepted)
    s["next"].copy_(torch.searchsorted(total, level[:, None], right=True)[:, 0])
    return [s["accepted"], s["next"]]


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "append":
        k, v = s["k_pool"].double(), s["v_pool"].double()
        tables = s["tables"].cpu().numpy()
        at = 0
        for i, (n, T) in enumerate(s["spans"]):
            t = T - n
            while t < T:  # block after block
                m = min(T, (t // BLOCK + 1) * BLOCK) - t
                b, o = int(tables[i, t // BLOCK]), t % BLOCK
                k[b, :, o:o + m] = s["k"][at:at + m].transpose(0, 1).double()
                v[b, :, o:o + m] = s["v"][at:at + m].transpose(0, 1).double()
                t, at = t + m, at + m
        return [k, v]
    if case["op"] == "verify":
        tokens = s["tokens"].cpu().numpy()
        u, r = s["accept_u"].cpu().numpy(), s["sample_u"].cpu().numpy()
        accepted, following = [], []
        a = 0
        for i, n in enumerate(s["counts"]):
            p = s["target"][a:a + n].cpu().double().numpy()
            q = s["draft"][a:a + n].cpu().double().numpy() if s["draft"] is not None else None
            j = 0
            while j < n - 1:
                x = int(tokens[a + j + 1])
                if not float(u[a + j]) * (1.0 if q is None else q[j, x]) < p[j, x]:
                    break
                j += 1
            w = p[j].copy()
            if j < n - 1:
                if q is None:
                    w[int(tokens[a + j + 1])] = 0.0
                else:
                    w = np.maximum(w - q[j], 0.0)
            run_sum = np.cumsum(w)
            accepted.append(j)
            following.append(int(np.argmax(run_sum > float(r[i]) * run_sum[-1])))
            a += n
        return [torch.tensor(accepted, dtype=torch.int64), torch.tensor(following)]
    # attention, one query head of one request at a time, from the largest exponent down
    if work(case)["flops"] > 4e12:
        return None
    out = torch.zeros(s["q"].shape[0], case["Hq"], case["d"], dtype=torch.float64, device="cuda")
    G = case["Hq"] // case["Hkv"]
    a = 0
    for i, (n, T) in enumerate(s["spans"]):
        blocks = s["tables"][i].long()[:(T + BLOCK - 1) // BLOCK]
        for h in range(case["Hkv"]):
            k = s["k_pool"][blocks, h].reshape(-1, case["d"])[:T].double()
            v = s["v_pool"][blocks, h].reshape(-1, case["d"])[:T].double()
            for part in range(0, n, 4096):
                m = min(n - part, 4096)
                q = s["q"][a + part:a + part + m, h * G:(h + 1) * G].double()
                x = torch.einsum("ngd,td->ngt", q, k) * s["scale"]
                first = T - n + part + 1  # keys the part's first token sees
                for_each = torch.arange(first, first + m, device="cuda")
                x = torch.where(torch.arange(T, device="cuda") < for_each[:, None, None], x,
                                -torch.inf)
                x = torch.softmax(x, -1)
                out[a + part:a + part + m, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", x, v)
        a += n
    return out
