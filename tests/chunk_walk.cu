// Host check of the chunk attention's work shares: over random batches, every
// key tile of every work item belongs to exactly one CTA, in order; a CTA leaves
// at most one partial result of each kind; and what the joining CTA works out
// about an item's shares is what the CTAs did.  Runs without a GPU.
#include "zp_chunk_attn.cu"

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>
#include <vector>

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

int main()
{
    long long items = 0;
    for (int batch = 0; batch < 1500; ++batch) {
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
        long long cost = 0;
        int longest = 0;
        for (int i = 0; i < R; ++i) {
            ChunkReq c;
            bool bad;
            if (chunk_request(a, i, c, &bad)) {
                cost += Hkv * head_cost(c, tpt);
                longest = std::max(longest, longest_item(c, tpt));
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
                if (!chunk_request(a, i, p.c0, &bad))
                    continue;
                p.i0 = i;
                const long long w = Hkv * head_cost(p.c0, tpt);
                if (p.lo < before + w)
                    break;
                before += w;
            }
            p.x0 = before;
            CaWalk walk{a, p, tpt, {}};
            int heads = 0, tails = 0;  // partial results that begin, or do not begin, their item
            for (bool more = walk.begin(); more; more = walk.next()) {
                const CaItem &t = walk.it;
                CHECK(t.ka < t.kb);
                CHECK(t.single == (t.ntok <= tpt) && t.ntok >= 1 && t.ntok <= 2 * tpt);
                seen[{t.i, t.h, t.p}].push_back({b, t.ka, t.kb, t.kt, t.w, t.x, t.single});
                if (t.ka != 0 || t.kb != t.kt)
                    ++(t.ka == 0 ? heads : tails);
            }
            CHECK(heads <= 1 && tails <= 1);
        }
        long long expected = 0;
        for (int i = 0; i < R; ++i) {
            const int n = starts[i + 1] - starts[i];
            const int pairs = n ? pair_count(n, tpt) : 0;
            for (int h = 0; h < Hkv; ++h)
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
    std::printf("ok %lld\n", items);
    return 0;
}
