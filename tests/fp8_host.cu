// Host checks of the calls on an 8-bit cache and of the draws from logits, without a GPU: the
// work shares with kv heads two at a time and with chunks that are another kernel's; which
// kernels a batch goes to; refusals; the weights.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>
#include <tuple>
#include <vector>

static std::string g_calls;
static cudaError_t fake_get_device(int *d)
{
    *d = 0;
    return cudaSuccess;
}
#define cudaGetDevice fake_get_device
#include "zp_api.cu"
#include "zp_chunk_attn.cuh"
#include "zp_sample.cuh"

namespace zp {
static ChunkAttnArgs g_attn;
static SampleArgs g_sample;
static int g_few;
cudaError_t launch_fp8_append(const Fp8KvArgs &a, cudaStream_t)
{
    g_calls += a.starts ? "A" : "a";
    return cudaSuccess;
}
cudaError_t launch_fp8_decode(const Fp8AttnArgs &, int, cudaStream_t)
{
    g_calls += "d";
    return cudaSuccess;
}
cudaError_t launch_fp8_few_rows(const Fp8AttnArgs &a, int rows, int, cudaStream_t)
{
    const bool first = a.over == 0, behind = !g_calls.empty();
    const bool ok = a.groups == 1 && a.splits >= 1 && a.splits <= 8 && a.follows == behind;
    g_calls += !ok ? "?" : first ? "f" : "g";
    g_few = first ? rows : g_few * 100 + rows;
    return cudaSuccess;
}
cudaError_t launch_fp8_widen(const Fp8WidenArgs &, int, cudaStream_t)
{
    g_calls += "w";
    return cudaSuccess;
}
cudaError_t launch_fp8_chunk_attn(const ChunkAttnArgs &a, int, int, cudaStream_t)
{
    g_calls += "c";
    g_attn = a;
    return cudaSuccess;
}
cudaError_t launch_chunk_attn(const ChunkAttnArgs &a, int, int, cudaStream_t)
{
    g_calls += a.widened ? "b" : "?";
    return cudaSuccess;
}
cudaError_t launch_sample(const SampleArgs &a, bool bf16, int, cudaStream_t)
{
    g_calls += a.tokens ? (bf16 ? "T" : "t") : (bf16 ? "P" : "p");
    g_sample = a;
    return cudaSuccess;
}
bool encode_chunk_q_map(CUtensorMap *, const void *, int, int64_t, int, int, int) { return true; }
}  // namespace zp

using namespace zp;

static unsigned long long g_state = 1;
static int rnd(int n)  // the same numbers on every machine
{
    g_state = g_state * 6364136223846793005ull + 1442695040888963407ull;
    return static_cast<int>((g_state >> 33) % static_cast<unsigned>(n));
}

#define CHECK(x)                                                        \
    do {                                                                \
        if (!(x)) {                                                     \
            std::printf("batch %d: line %d: %s\n", batch, __LINE__, #x); \
            return 1;                                                   \
        }                                                               \
    } while (0)

struct Part {
    int cta, ka, kb, kt, w;
    long long x;
    bool single;
};

static int walk()
{
    long long items = 0;
    for (int batch = 0; batch < 700; ++batch) {
        const int groups[] = {1, 2, 3, 4, 5, 7, 8, 16};
        const int G = groups[rnd(8)], Hkv = 1 + rnd(8), R = 1 + (rnd(3) == 0 ? rnd(300) : rnd(8));
        const int grid = rnd(4) ? 152 : 1 + rnd(8), mode = rnd(5);
        std::vector<int> starts{0}, lengths;
        for (int i = 0; i < R; ++i) {
            int n = mode == 0   ? 1
                    : mode == 1 ? rnd(9)
                    : mode == 2 ? rnd(700)
                    : mode == 3 ? (rnd(10) ? 1 : rnd(3000))
                                : rnd(200);
            int T = n + rnd(rnd(2) ? 3000 : 40);
            if (rnd(50) == 0)
                T += rnd(30000);
            starts.push_back(starts.back() + n);
            lengths.push_back(T);
        }
        ChunkAttnArgs a{};
        a.starts = starts.data();
        a.total = starts.back();
        a.stride = 1 << 20;
        a.num_rows = a.R = R;
        a.lengths = lengths.data();
        a.Hkv = Hkv;
        a.Hq = Hkv * G;
        const int tpt = tile_tokens(G);
        const bool duos = rnd(4) != 0;
        a.few = rnd(3) ? 0 : rnd(6);  // shorter chunks are another kernel's
        auto ours = [&](int i) { return starts[i + 1] - starts[i] > a.few; };
        long long cost = 0;
        int longest = 0;
        for (int i = 0; i < R; ++i) {
            ChunkReq c;
            bool bad;
            if (attn_request(a, i, c, &bad)) {
                cost += request_cost(c, tpt, Hkv, duos);
                longest = std::max(longest, heads_by_two(c.n, tpt, Hkv, duos)
                                                ? item_cost(c.len, false)
                                                : longest_item(c, tpt));
            }
            CHECK(!bad);
        }
        CaPlan plan{};
        make_shares(plan, cost, longest, grid);
        CHECK(plan.ctas >= 1 && plan.ctas <= grid);
        std::map<std::tuple<int, int, int>, std::vector<Part>> seen;
        for (int b = 0; b < grid; ++b) {
            CaPlan p = plan;
            p.lo = share_border(p, b);
            p.hi = share_border(p, b + 1);
            CHECK(b < plan.ctas || p.lo >= p.hi);
            long long before = 0;
            for (int i = 0; i < R && p.lo < p.hi; ++i) {
                bool bad;
                if (!attn_request(a, i, p.c0, &bad))
                    continue;
                p.i0 = i;
                const long long w = request_cost(p.c0, tpt, Hkv, duos);
                if (p.lo < before + w)
                    break;
                before += w;
            }
            p.x0 = before;
            CaWalk walk{a, p, tpt, {}, duos};
            int heads = 0, tails = 0;  // partial results that begin, or do not begin, their item
            for (bool more = walk.begin(); more; more = walk.next()) {
                const CaItem &t = walk.it;
                CHECK(t.ka < t.kb);
                CHECK(t.duo == heads_by_two(t.c.n, tpt, Hkv, duos));
                CHECK(t.single == (t.ntok <= tpt && !t.duo));
                CHECK(t.ntok >= 1 && t.ntok <= (t.duo ? tpt : 2 * tpt));
                seen[{t.i, t.h, t.p}].push_back({b, t.ka, t.kb, t.kt, t.w, t.x, t.single});
                if (t.ka != 0 || t.kb != t.kt)
                    ++(t.ka == 0 ? heads : tails);
            }
            CHECK(heads <= 1 && tails <= 1);
        }
        long long expected = 0;
        for (int i = 0; i < R; ++i) {
            const int n = starts[i + 1] - starts[i];
            const int pairs = n && ours(i) ? pair_count(n, tpt) : 0;
            const bool two = n && heads_by_two(n, tpt, Hkv, duos);
            for (int h = 0; h < (two ? Hkv / 2 : Hkv); ++h)
                for (int p = 0; p < pairs; ++p) {
                    ++expected;
                    const auto f = seen.find({i, h, p});
                    CHECK(f != seen.end());
                    const std::vector<Part> &v = f->second;
                    const int vis = lengths[i] - n + std::min(n, (p + 1) * 2 * tpt);
                    CHECK(v[0].kt == (vis + kTile - 1) / kTile);
                    int at = 0;
                    for (const Part &e : v) {
                        CHECK(e.ka == at);
                        at = e.kb;
                    }
                    CHECK(at == v[0].kt);
                    // the shares as the joining CTA sees them: a lane a share
                    const int bs = static_cast<int>(quotient(v[0].x, plan.share));
                    size_t k = 0;
                    for (int b = bs; b < std::min(bs + 32, plan.ctas); ++b) {
                        const long long lo = share_border(plan, b), hi = share_border(plan, b + 1);
                        const long long x = v[0].x, end = x + v[0].w;
                        if (lo >= end)
                            break;
                        const int k0 = lo > x ? cut_tile(lo - x, v[0].kt, v[0].single) : 0;
                        const int k1 =
                            hi < end ? cut_tile(hi - x, v[0].kt, v[0].single) : v[0].kt;
                        if (k0 >= k1)
                            continue;
                        CHECK(k < v.size() && v[k].cta == b);
                        ++k;
                    }
                    CHECK(k == v.size());
                }
        }
        CHECK(expected == static_cast<long long>(seen.size()));
        items += expected;
    }
    return items > 0 ? 0 : 1;
}

// Memory is a line of addresses that nothing reads.
struct Line {
    uintptr_t at = 1 << 20;
    template <class T>
    T *take(size_t bytes)
    {
        T *p = reinterpret_cast<T *>(at);
        at += (bytes + 31) / 32 * 32;
        return p;
    }
};

static zp_cache handle(Line &m, int max_requests)
{
    zp_cache c;
    c.L = 1;
    c.Hkv = 8;
    c.Hq = 32;
    c.d = 128;
    c.b = 16;
    c.num_blocks = 8;
    c.num_sms = 152;
    c.max_requests = max_requests;
    c.fp8 = true;
    c.kpools.push_back(m.take<void>(8 * 8 * 16 * 128));
    c.vpools.push_back(m.take<void>(8 * 8 * 16 * 128));
    c.kscales.push_back(m.take<float>(8 * 8 * 4));
    c.vscales.push_back(m.take<float>(8 * 8 * 4));
    return c;
}

static int calls()
{
    const int batch = 0;
    Line m;
    zp_cache c = handle(m, 512);
    const size_t most = 8193;
    int32_t *starts = m.take<int32_t>(4 * 513), *tables = m.take<int32_t>(4 * 512 * 2048);
    int32_t *lengths = m.take<int32_t>(4 * 512), *req_idx = m.take<int32_t>(4 * 512);
    uint8_t *q = m.take<uint8_t>(most * 8192), *out = m.take<uint8_t>(most * 8192);
    uint8_t *kv = m.take<uint8_t>(most * 2048);
    zp_status st;
    auto attn = [&](int R, int total, int stride, void *o = nullptr, int64_t qs = 4096,
                    float scale = 1.f) {
        g_calls.clear();
        st = zp_paged_chunk_attn(&c, 0, q, qs, starts, total, tables, stride, 512, lengths, req_idx,
                                 R, scale, o ? o : out, nullptr);
        return g_calls;
    };
    // a large batch by the mean of the rows (four heads a group): up to 8, up to 24, up to 128,
    // above; the longer ones first, the others behind them and each other
    CHECK(attn(256, 2 * 256, 128) == "cfg" && g_few == 824 && g_attn.few == 6);
    CHECK(attn(256, 2 * 256 + 1, 128) == "cfg" && g_few == 1624 && g_attn.few == 6);
    CHECK(attn(256, 6 * 256, 128) == "cfg" && g_few == 1624 && g_attn.few == 6);
    CHECK(attn(256, 6 * 256 + 1, 128) == "cf" && g_few == 16 && g_attn.few == 4);
    CHECK(attn(256, 32 * 256, 128) == "cf" && g_few == 16 && g_attn.few == 4);
    CHECK(attn(256, 32 * 256 + 1, 128) == "c" && g_attn.few == 0 && g_attn.duos == 1);
    // no more rows in all than the first launch's, or the second's: nothing for the others
    CHECK(attn(256, 2, 128) == "f" && attn(256, 6, 128) == "fg" && attn(256, 7, 128) == "cfg");
    // a smaller one: up to 20, the launch of its mean
    CHECK(attn(38, 38 * 2, 128) == "cf" && g_few == 8 && g_attn.few == 2);
    CHECK(attn(38, 38 * 4, 128) == "cf" && g_few == 16 && g_attn.few == 4);
    CHECK(attn(38, 38 * 5, 128) == "cf" && g_few == 24 && g_attn.few == 6);
    CHECK(attn(38, 38 * 5 + 1, 128) == "c" && g_attn.few == 0);
    CHECK(attn(37, 37 * 30, 128) == "c" && g_attn.duos == 0);
    CHECK(attn(4, 4 * 191, 128) == "c" && attn(4, 4 * 192, 128) == "wbc");
    // all of them few: no other kernel
    CHECK(attn(1, 4, 128) == "f" && attn(1, 5, 128) == "f" && g_few == 24);
    // few units and a wide table
    CHECK(attn(1, 4, 512) == "f" && attn(1, 4, 513) == "c" && attn(1, 5, 342) == "c");
    CHECK(attn(38, 38 * 4, 2000) == "cf");
    CHECK(attn(0, 0, 128).empty() && st == ZP_OK && attn(3, 0, 128).empty() && st == ZP_OK);
    // refusals
    auto refused = [&](const std::string &x) { return x.empty() && st == ZP_ERR_INVALID_ARG; };
    for (void *p : {c.kpools[0], c.vpools[0], static_cast<void *>(c.kscales[0]),
                    static_cast<void *>(c.vscales[0]), static_cast<void *>(q),
                    static_cast<void *>(starts), static_cast<void *>(tables),
                    static_cast<void *>(lengths), static_cast<void *>(req_idx),
                    static_cast<void *>(out + 16)})
        CHECK(refused(attn(4, 16, 128, p)));
    CHECK(refused(attn(513, 600, 128)) && refused(attn(4, 16, 0)) && refused(attn(4, -1, 128)));
    CHECK(refused(attn(4, 16, 128, out, 4100)) && refused(attn(4, 16, 128, out, 2048)));
    CHECK(refused(attn(4, 16, 128, out, 4096, INFINITY)) &&
          refused(attn(4, 16, 128, out, 4096, NAN)));
    auto append = [&](const void *k, const void *v, int total) {
        g_calls.clear();
        st = zp_append_kv_chunk(&c, 0, k, 1024, v, 1024, starts, total, tables, 128, 512, lengths,
                                req_idx, 4, nullptr);
        return g_calls;
    };
    CHECK(append(kv, kv, 16) == "A");
    for (void *p : {c.kpools[0], c.vpools[0], static_cast<void *>(c.kscales[0]),
                    static_cast<void *>(c.vscales[0])})
        CHECK(refused(append(p, kv, 16)) && refused(append(kv, p, 16)));
    return 0;
}

constexpr int R = 8, V = 1000, S = 1024;

static int draws()
{
    const int batch = 0;
    Line m;
    zp_cache c = handle(m, 8);
    float *logits = m.take<float>(4 * R * S), *probs = m.take<float>(4 * R * S);
    float *t = m.take<float>(4 * 8), *p = m.take<float>(4 * 8), *mp = m.take<float>(4 * 8);
    float *u = m.take<float>(4 * R);
    int32_t *k = m.take<int32_t>(4 * 8), *idx = m.take<int32_t>(4 * R), *tok = m.take<int32_t>(4 * R);
    zp_status st;
    struct Call {
        const void *logits;
        int type, vocab;
        int64_t stride;
        int rows, R;
        const int32_t *idx;
    };
    const Call good{logits, ZP_DTYPE_F32, V, S, 8, R, idx};
    auto sample = [&](const Call &x, int32_t *to) {
        g_calls.clear();
        st = zp_sample(&c, x.logits, x.type, x.vocab, x.stride, t, k, p, mp, x.rows, x.idx, u, x.R,
                       to, nullptr);
        return g_calls;
    };
    auto token_probs = [&](const Call &x, void *to, int type = ZP_DTYPE_F32, int64_t stride = S) {
        g_calls.clear();
        st = zp_token_probs(&c, x.logits, x.type, x.vocab, x.stride, t, k, p, mp, x.rows, x.idx, x.R,
                            to, type, stride, nullptr);
        return g_calls;
    };
    auto refused = [&](const std::string &x, zp_status by = ZP_ERR_INVALID_ARG) {
        return x.empty() && st == by;
    };
    CHECK(sample(good, tok) == "t" && g_sample.R == R && g_sample.vocab == V);
    CHECK(token_probs(good, probs) == "p" && token_probs(good, probs, ZP_DTYPE_BF16) == "p");
    Call x = good;
    x.type = ZP_DTYPE_BF16;
    CHECK(sample(x, tok) == "T" && token_probs(x, probs) == "P");
    x.type = 7;
    CHECK(refused(sample(x, tok), ZP_ERR_UNSUPPORTED) &&
          refused(token_probs(good, probs, 7), ZP_ERR_UNSUPPORTED));
    for (int vocab : {0, -1, S + 1}) {  // none; more than the stride
        x = good;
        x.vocab = vocab;
        CHECK(refused(sample(x, tok)) && refused(token_probs(x, probs)));
    }
    x = good;
    x.vocab = kSampleMaxVocab;
    x.stride = x.vocab;
    x.R = 1;
    CHECK(sample(x, tok) == "t" || st == ZP_ERR_INVALID_ARG);  // (the line is shorter)
    x.stride = ++x.vocab;
    CHECK(refused(sample(x, tok), ZP_ERR_UNSUPPORTED));
    x = good;
    x.R = 9;
    CHECK(refused(sample(x, tok)));
    x.R = -1;
    CHECK(refused(sample(x, tok)) && refused(token_probs(x, probs)));
    x.R = 0;
    CHECK(refused(sample(x, tok), ZP_OK) && refused(token_probs(x, probs), ZP_OK));
    x = good;
    x.rows = 0;
    CHECK(refused(sample(x, tok)) && refused(token_probs(x, probs)));
    x.rows = 7;
    CHECK(sample(x, tok) == "t");
    x.idx = nullptr;  // eight rows for seven entries
    CHECK(refused(sample(x, tok)) && refused(token_probs(x, probs)));
    x = good;
    x.logits = nullptr;
    CHECK(refused(sample(x, tok)) && refused(sample(good, nullptr)));
    x.logits = reinterpret_cast<const char *>(logits) + 2;
    CHECK(refused(sample(x, tok)) && refused(token_probs(good, probs, ZP_DTYPE_F32, V - 1)));
    for (void *in : {static_cast<void *>(logits), static_cast<void *>(t), static_cast<void *>(k),
                     static_cast<void *>(p), static_cast<void *>(mp), static_cast<void *>(idx)}) {
        CHECK(refused(sample(good, static_cast<int32_t *>(in))));
        CHECK(refused(token_probs(good, in)));
    }
    CHECK(refused(sample(good, reinterpret_cast<int32_t *>(u) + R - 1)));
    return 0;
}

// 2^-y within 2^-40 (of which 5.6 units of 2^-44 are the table's number cut to 30 bits times
// |z| < 2^-11.5, 4 two roundings of z to 2^-42, 2.5 the shift, the lowest bit and the table; the pair
// y is known to less than 1), odd, and none past 2^-48.
static int weights_()
{
    const int batch = 0;
    static const WeightTable table;
    double worst = 0;
    for (int n = 0; n < 2000000; ++n) {
        const float T = std::exp2(static_cast<float>(rnd(1 << 20)) / (1 << 16) - 8.f);
        const float M = static_cast<float>(rnd(1 << 24) - (1 << 23)) / (1 << (rnd(20) + 3));
        const double d = 1.4426950408889634 / static_cast<double>(T);
        WeightScale c;
        c.ch = static_cast<float>(d);
        c.cl = static_cast<float>(d - static_cast<double>(c.ch));
        const float l = M - T * static_cast<float>(rnd(1 << 24)) / (1 << (19 + rnd(5)));
        float h, lo;
        gap(M, l, h, lo);
        const uint64_t w = weight(table.v, c, h, lo);
        const long double y = (static_cast<long double>(M) - l) / T / std::log(2.0L);
        const double want = static_cast<double>(std::exp2(-y));
        worst = std::max(worst, std::fabs(static_cast<double>(w) * 0x1p-44 - want));
        CHECK(y > 47.999 || (w & 1));
        CHECK(y < 48.001 || w == 0);
    }
    CHECK(worst < 0x1p-40);
    return 0;
}

int main(int argc, char **argv)
{
    const char *what = argc > 1 ? argv[1] : "";
    int bad = 2;
    if (!std::strcmp(what, "walk"))
        bad = walk();
    else if (!std::strcmp(what, "calls"))
        bad = calls();
    else if (!std::strcmp(what, "draws"))
        bad = draws();
    else if (!std::strcmp(what, "weights"))
        bad = weights_();
    if (!bad)
        std::printf("ok\n");
    return bad;
}
