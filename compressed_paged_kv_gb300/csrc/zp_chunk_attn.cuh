// zp_chunk_attn.cuh -- attention of a ragged chunk of new tokens over the paged
// cache: the many-query form of the decode attention, on the 5th-generation
// tensor cores.
//
// Query j of a chunk of n tokens sits at position p = T - n + j of its
// request's T tokens and sees the keys t <= p.  The G query heads of a kv head
// share its keys, so a query ROW is (token, head of the group), token-major:
// floor(128/G) tokens make one 128-row tile.  Keys go by 128 (eight cache
// blocks).  Per (request, kv head) there are two forms of work item:
//   pair    two query tiles A and B, both over the item's key tiles;
//   single  one query tile (a chunk, or the rest of one, of at most 128
//           rows): A takes the even key tiles and B the odd ones, and the two
//           halves are joined at the end.
// Either way two streams S = Q K^T -> softmax -> O += P V run at once, so that
// the tensor cores work for one while the other is in its softmax, and each
// K/V tile is staged once for up to 256 rows.
//
// Twenty warps:
//   warps 0-7, 8-15  softmax of A and of B, a row of S a pair of threads (64
//           columns each, out of tensor memory; they exchange their maxima): a
//           running maximum and sum (fp32, base 2), P rounded to bf16 over S in
//           tensor memory.  O is rescaled only when a maximum grows by more
//           than 2^20 over the one it is held against, in place in tensor memory,
//           between the products: S's arrival says that the product before it is
//           done.  p is taken against 2^50 over that maximum: it stays below
//           2^-30, so over the 2^30 keys of the longest row no sum of p v exceeds
//           the largest |v|, and what gets lost below 2^-126 are values below
//           2^-75.  (By the item's own length, 2^(20 + log2), the key loop took 0.6
//           to 1 % longer.)  Then the epilogue.
//   warp 16 walks the items, describes each in shared memory for the others,
//           and loads Q once per item and the K tiles (TMA, a box a cache block
//           and 64 dims, 128-byte swizzle) into a ring of their own
//   warps 17, 18  the products of A and of B: tcgen05.mma (kind::f16, bf16 ->
//           fp32), S from shared memory, P V with P from tensor memory and V as
//           an MN-major operand
//   warp 19 loads the V tiles into theirs
//
// A key past the length or hidden from a row has probability 0, but 0 times an
// infinity or NaN is NaN.  The V rows past the length in the last block are
// cleared in shared memory.  Values hidden from some rows of an item and seen by
// others cannot be: a CTA whose share gave an O that is not finite to a row with
// keys hidden from it walks its whole share once more, "clean".  Then what is not
// finite in a V row hidden from the item's first token counts as 0 in the
// products, and the epilogue puts the infinities and NaNs back into the outputs of
// the rows that see them.  A share is walked at most twice, however long its rows
// are: with such values in every request, 160 chunks of 64 tokens over 2,000 (8
// heads of 128) take 250 to 570 us, 109 without any.
//
// The grid is one CTA an SM.  Every CTA adds up the cost of all items (the
// keys each reads, plus a fixed part) from the device arrays and takes an equal,
// contiguous share, cut at key tiles, so that few long rows and many short
// ones both fill the GPU.  An item cut by a border leaves partial results (m,
// l, O) in the handle's workspace, and the CTA that arrives last joins them in
// the fixed order of the shares: results do not depend on the timing.  The
// arrivals are counted in two sets of words that the calls use in turn.  A CTA
// takes a number when it enters: with g CTAs a call, numbers 0 .. g - 1 (modulo
// 2 g) belong to a call of the first set and the others to one of the second,
// whatever the order in which they enter.  Each clears its words of the other
// set, which no CTA of this call touches, for the next call: whatever a call
// that gave up a wait has left uncounted is gone, with no help from the host.
//
// P is bf16 because the product takes two operands of one type and V is bf16;
// it makes the error of a result, relative to 64 bits, 0.0020 where the result's
// own rounding to bf16 is 0.0015.
//
// Measured, calls in a row, 32 heads of 128 over 8 kv heads: 2,048 tokens over
// 32,049, 1.04 TFLOP in 0.715 ms = 1.46 PFLOP/s, 0.84 of the library products'
// sustained rate; 16 prompts of 331 to 4,007 tokens in 0.667 ms = 1.15 PFLOP/s; 256
// speculative chunks over 1,024 to 2,040 tokens, 1.64 GB in 0.271 ms = 6.0 TB/s,
// 0.89 of the copy peak.  What bounds it: in the first the power limit and, as in
// the second, the chain of a stream (product -> softmax -> product; tensor pipe 60 %
// busy, issue slots 48 %), in the second also 2.5 us between two items of a CTA; in
// the last one HBM; in batches of a few chunks the chain of the start (8 chunks of
// 5 tokens, from a cold cache, on the device: offsets -> plan 2.0 us -> block ids ->
// first tile 7.3, in the slowest CTA 9.2) and of the join (the slowest 5 us).
//
// Over an 8-bit cache (F8), with a key ks k8 and a value vs v8, one ks and one vs a block:
//     t = scale (q . k8) ks + log2 vs,  p = 2^t,  out = sum p v8 / sum (p / vs),
// so no value is multiplied out, and the running maximum is that of t.
//   S   e4m3 products (kind::f8f6f4) of k8 as it lies there with q as two e4m3 numbers, f q =
//       upper + lower, whose eight bits hold bf16's: two passes at twice fp16's rate, and no K
//       is converted
//   V   to fp16 (exact) by the softmax warps while they wait for S, raw tiles in a ring of their
//       own; P in fp16, 2^5 to 2^15 at the maximum, with 2^-11 of rounding instead of bf16's
//       2^-8.  In e4m3 P would lose all but four bits.  Conversion by four warps of
//       their own left the others too few registers (24 warps: 1 KB of spills a thread).
//   The blocks' scales come to shared memory by the loader's lanes, beside the K tiles.
// A request of many query rows has its V tiles converted once for every 256 of them: those are
// widened to bf16 first (zp_fp8_widen.cu).  Chunks of few rows are zp_fp8_decode.cu's.
//
// Measured, 256 chunks of 8 tokens over 1,536 keys, 32 heads of 128 over 8, 0.81 GB in 295 us, 2.7
// TB/s (a bf16 cache, of twice the bytes: 260); 19 chunks of 64 over 8,192 159 us (116).
// What bounds it: with few rows a tile, the two warps of a stream that have them (a row's 64 columns
// take one warp 1.4 to 2.2 us of the 2.8 us between key tiles) and 13 us of Q, joins and output
// between items; with many, the chain of a stream, longer by V's conversion.
#pragma once

#include "zp_fp8.cuh"

namespace zp {

namespace {

constexpr int kTile = 128;             // query rows a tile, keys a tile
constexpr int kSmWarps = 8;            // softmax warps a query tile
constexpr int kCaThreads = (2 * kSmWarps + 4) * 32;
constexpr int kSmRegs = 104, kOtherRegs = 64;  // registers a thread after the split
static_assert(kSmRegs * 2 * kSmWarps + kOtherRegs * 4 <= 96 * (2 * kSmWarps + 4),
              "the split draws on the registers of the launch");
// Costs, in keys of a pair (measured: 1.4 us for 128 of them, 0.6 for 128 of a
// single item, whose streams take half the tiles each, and 2.7 to 2.9 us between
// the last tile of an item and the first of the next).  With a single item's
// keys at full cost 60 single tokens beside two prompt pieces take 69 us, not 61.
constexpr int kItemCost = 320;         // an item's fixed cost
constexpr int kSingle = 8;             // 16ths of a pair's cost that a single item's key takes
constexpr int kMinShare = 2 * kTile;   // least cost given to a CTA
constexpr int kMaxSpan = 30;           // CTAs an item is cut over, about (a lane each joins them)
constexpr int kLoadWarp = 2 * kSmWarps;       // then the products' warps of A and of B, V's loader
constexpr int kMmaWarp = kLoadWarp + 1;
constexpr int kLoadVWarp = kLoadWarp + 3;
constexpr int kDescs = 4;              // item descriptions in flight
constexpr int kTmemCols = 512;         // S/P of A, of B; O of A, of B
constexpr float kRescale = 20.f;       // log2 of the growth that rescales O
constexpr float kAbove = kRescale + 30.f;  // of what p is taken against, over the maximum
// The same of an 8-bit cache, where p is fp16: from 2^5 to 2^15 at the maximum
constexpr float kRescale8 = 10.f;
constexpr float kAbove8 = -5.f;
constexpr int kScales = 16;            // key tiles whose scales are kept
constexpr int kQTiles = 2 * kDescs;    // query tiles whose rows' factors are kept

// What every CTA works out at its start.
struct CaPlan {
    long long cost;   // of all items
    long long share;  // of a CTA
    long long lo, hi; // this CTA's share
    long long x0;     // cost before request i0
    ChunkReq c0;      // the request `lo` falls into
    int i0;
    int ctas;         // CTAs with a share
};

// A work item as the other warps need it.
struct CaDesc {
    int row0;    // packed row of its first token
    int ntok;    // its tokens; 0: no more items
    int h;       // kv head
    int pos0;    // position of its first token
    int len;     // cached tokens of the request
    int row;     // the request's table row
    int ka, kb;  // this CTA's key tiles
    int kt;      // all its key tiles
    int w;       // cost
    int clean;   // of the second walk
    int duo;     // one query tile of h for A, one of h + 1 for B
    long long x; // cost before it
};

template <int D, bool F8>
struct CaSmem {
    static constexpr int PANELS = D / 64;
    static constexpr int PANEL = kTile * 128;            // bytes of 128 rows of 64 dims
    static constexpr int TILE = PANELS * PANEL;          // of 16-bit elements
    static constexpr int TILE8 = kTile * D;              // of 8-bit ones
    static constexpr int KTILE = F8 ? TILE8 : TILE;
    // stages of K, of V and of 8-bit V
    static constexpr int NK = D == 128 ? (F8 ? 3 : 2) : 5;
    static constexpr int NV = D == 128 ? (F8 ? 2 : 3) : F8 ? 4 : 5;
    static constexpr int NR = F8 ? (D == 128 ? 2 : 4) : 0;
    static_assert(NR <= NV, "a V tile that has come implies the release before last of its place");
    static constexpr int XC = 16;  // columns of O a step of the epilogue
    static constexpr int off_q = 0;                      // Q of A, Q of B
    // with 64 dims a row's numbers lie elsewhere than the row did: two more tiles for them
    static constexpr bool SPLIT = F8 && D == 64;
    static constexpr int off_k = off_q + (SPLIT ? 4 : 2) * TILE;
    static constexpr int off_v = off_k + NK * KTILE;
    static constexpr int off_raw = off_v + NV * TILE;
    static constexpr int off_scale = off_raw + NR * TILE8;  // float4 [kScales][8]: of key tiles
    // float [kQTiles][128] of Q's rows; float [2][2][128], the maxima of row halves
    static constexpr int off_qf = off_scale + (F8 ? kScales * 8 * 16 : 0);
    static constexpr int off_max = off_qf + (F8 ? kQTiles * kTile * 4 : 0);
    static constexpr int off_desc = off_max + 4 * kTile * 4;  // CaDesc [kDescs]
    static constexpr int off_plan = off_desc + kDescs * static_cast<int>(sizeof(CaDesc));
    static constexpr int off_scan = off_plan + static_cast<int>(sizeof(CaPlan));  // int64 [warps]
    static constexpr int off_bar = off_scan + kCaThreads / 32 * 8;
    // K full, empty; V full, empty; Sfull[2], Pready[2], Ofull[2], Oempty[2], Qfull[2],
    // Qempty[2], turn[2]; described, read [kDescs]; half, taken, done; 8-bit V full for A, for B,
    // empty; Qready[2]
    static constexpr int NBAR = 2 * NK + 2 * NV + 14 + 2 * kDescs + 3 + (F8 ? 3 * NR + 2 : 0);
    static constexpr int off_tmem = off_bar + NBAR * 8;
    // int: last arrived [2]; the call's set of arrivals; what the walk met (1: rows to
    // walk for again, 2: a wait given up); partial results left to the second walk [2]
    static constexpr int off_last = off_tmem + 8;
    static constexpr int BYTES = off_last + 24;
    static_assert(BYTES <= 232448 && off_desc % 8 == 0 && off_bar % 8 == 0, "shared memory");
};

struct CaItem {
    ChunkReq c;
    int i, h, p;            // request, kv head, pair
    int pairs;              // of the request
    long long x;            // cost before the item
    long long span;         // cost of the request's items of one kv head
    int tok0, ntok;         // tokens of the item
    int kt;                 // key tiles
    int w;                  // cost
    int ka, kb;             // this CTA's key tiles
    bool single;
    bool duo;               // h and span of two kv heads
    int units;              // heads, or pairs of them, of the request
};

__host__ __device__ __forceinline__ int tile_tokens(int G) { return kTile / G; }

// Cost of an item whose last token sees `vis` keys.
__host__ __device__ __forceinline__ int item_cost(int vis, bool single)
{
    return kItemCost + (single ? vis / 16 * kSingle : vis);
}

// Cost of the first p pairs of one kv head, p < pairs (all but the last are whole).
__host__ __device__ __forceinline__ long long pair_prefix(const ChunkReq &c, int w2, int p)
{
    return static_cast<long long>(p) * (c.len - c.n + kItemCost) +
           static_cast<long long>(w2) * (static_cast<long long>(p) * (p + 1) / 2);
}

__host__ __device__ __forceinline__ int pair_count(int n, int tpt)
{
    return n <= tpt ? 1 : (n + 2 * tpt - 1) / (2 * tpt);
}

// Tokens of a request's last item.
__host__ __device__ __forceinline__ int last_tokens(int n, int tpt)
{
    return n - (pair_count(n, tpt) - 1) * 2 * tpt;
}

__host__ __device__ __forceinline__ long long head_cost(const ChunkReq &c, int tpt)
{
    return pair_prefix(c, 2 * tpt, pair_count(c.n, tpt) - 1) +
           item_cost(c.len, last_tokens(c.n, tpt) <= tpt);
}

// Whether the request's kv heads go by two (of an 8-bit cache): its one query tile of one
// head to A and of the next to B, each with its own key tiles, instead of one after the
// other with A and B sharing the key tiles.  Half as many ends of items, and no half to wait
// for there: 256 chunks of 2..9 over 1,030..2,040, 8 kv heads of 128: 340 -> 304 us.  Only a
// batch of two heads an SM or more (`duos`): 19 chunks over 1,500 took 25.7 us the one way
// and 33.5 the other, 38 of them 48.6 and 46.3.
__host__ __device__ __forceinline__ bool heads_by_two(int n, int tpt, int Hkv, bool duos)
{
    return duos && n <= tpt && Hkv % 2 == 0;
}

__host__ __device__ __forceinline__ long long request_cost(const ChunkReq &c, int tpt, int Hkv,
                                                           bool duos)
{
    return heads_by_two(c.n, tpt, Hkv, duos)
               ? static_cast<long long>(Hkv / 2) * item_cost(c.len, false)
               : Hkv * head_cost(c, tpt);
}

// The cost of the request's longest item.
__host__ __device__ __forceinline__ int longest_item(const ChunkReq &c, int tpt)
{
    const int last = last_tokens(c.n, tpt);
    return max(item_cost(c.len, last <= tpt), last < c.n ? item_cost(c.len - last, false) : 0);
}

// Key tile at which a border `x` of cost into an item of `kt` tiles cuts it.
__host__ __device__ __forceinline__ int cut_tile(long long x, int kt, bool single)
{
    if (x <= kItemCost)
        return 0;
    const long long keys = single ? (x - kItemCost) * 16 / kSingle : x - kItemCost;
    const long long k = (keys + kTile / 2) / kTile;
    return k < kt ? static_cast<int>(k) : kt;
}

// n / d for n >= 0, d > 0: 32-bit where it can be (a 64-bit division is slow).
__host__ __device__ __forceinline__ long long quotient(long long n, long long d)
{
    if (((n | d) >> 32) == 0)
        return static_cast<uint32_t>(n) / static_cast<uint32_t>(d);
    return n / d;
}

__host__ __device__ __forceinline__ long long share_border(const CaPlan &pl, int b)
{
    const long long x = pl.share * b;
    return x < pl.cost ? x : pl.cost;
}

// Shares over at most `grid` CTAs: none below kMinShare (about), and no item
// over more than kMaxSpan + 2 of them.
__host__ __device__ __forceinline__ void make_shares(CaPlan &pl, long long cost, int longest,
                                                     int grid)
{
    const float span = kMaxSpan * (static_cast<float>(cost) / max(longest, 1));
    const long long most = cost / kMinShare;
    int ctas = most < grid ? static_cast<int>(most) : grid;
    if (span < ctas)
        ctas = static_cast<int>(span);
    pl.cost = cost;
    pl.ctas = ctas < 1 ? 1 : ctas;
    pl.share = quotient(cost + pl.ctas - 1, pl.ctas);
}

// Request i, if it is this call's: of an 8-bit cache's batch the requests with a place
// among the widened blocks are the call's over those, with the place for a table row, and
// the others the call's over the cache, but for those of few query rows.
__host__ __device__ __forceinline__ bool attn_request(const ChunkAttnArgs &a, int i, ChunkReq &c,
                                                      bool *bad)
{
    if (!chunk_request(a, i, c, bad) || c.n <= a.few)
        return false;
    if (!a.places)
        return true;
    const int at = a.places[i];
    if (a.widened)
        c.row = at;
    return (at >= 0) == (a.widened != 0);
}

// Block q of the request with table row `row`.
__device__ __forceinline__ int block_at(const ChunkAttnArgs &a, int row, int q)
{
    return a.widened ? row + q : a.tables[static_cast<size_t>(row) * a.stride + q];
}

// Walks this CTA's items; every role walks the same ones on its own.
struct CaWalk {
    const ChunkAttnArgs &a;
    const CaPlan &pl;
    int tpt;
    CaItem it;
    bool duos = false;

    __host__ __device__ __forceinline__ void fill()
    {
        it.tok0 = it.p * 2 * tpt;
        it.ntok = min(it.c.n - it.tok0, 2 * tpt);
        it.single = it.ntok <= tpt && !it.duo;
        const int vis = it.c.len - it.c.n + it.tok0 + it.ntok;
        it.kt = (vis + kTile - 1) / kTile;
        it.w = item_cost(vis, it.single);
        it.ka = it.x < pl.lo ? cut_tile(pl.lo - it.x, it.kt, it.single) : 0;
        it.kb = it.x + it.w > pl.hi ? cut_tile(pl.hi - it.x, it.kt, it.single) : it.kt;
    }

    __host__ __device__ __forceinline__ void entered(int i)
    {
        it.i = i;
        it.pairs = pair_count(it.c.n, tpt);
        it.duo = heads_by_two(it.c.n, tpt, a.Hkv, duos);
        it.units = it.duo ? a.Hkv / 2 : a.Hkv;
        it.span = it.duo ? item_cost(it.c.len, false) : head_cost(it.c, tpt);
    }

    __host__ __device__ __forceinline__ bool request(int i)
    {
        bool bad;
        for (; i < a.R; ++i)
            if (attn_request(a, i, it.c, &bad))
                break;
        if (i >= a.R)
            return false;
        entered(i);
        return true;
    }

    // The first item of the share; false when there is none.
    __host__ __device__ __forceinline__ bool begin()
    {
        if (pl.lo >= pl.hi)
            return false;
        it.c = pl.c0;
        entered(pl.i0);
        const long long off = pl.lo - pl.x0;
        it.h = static_cast<int>(quotient(off, it.span));
        const long long rem = off - it.h * it.span;
        int p0 = 0, p1 = it.pairs - 1;
        while (p0 < p1) {  // the last pair that begins at or before the border
            const int m = (p0 + p1 + 1) / 2;
            if (pair_prefix(it.c, 2 * tpt, m) <= rem)
                p0 = m;
            else
                p1 = m - 1;
        }
        it.p = p0;
        it.x = pl.x0 + it.h * it.span + pair_prefix(it.c, 2 * tpt, p0);
        fill();
        return skip_empty();
    }

    __host__ __device__ __forceinline__ bool step()
    {
        it.x += it.w;
        if (it.x >= pl.hi)
            return false;
        if (++it.p == it.pairs) {
            it.p = 0;
            if (++it.h == it.units) {
                it.h = 0;
                if (!request(it.i + 1))
                    return false;
            }
        }
        fill();
        return true;
    }

    __host__ __device__ __forceinline__ bool skip_empty()
    {
        while (it.ka >= it.kb)
            if (!step())
                return false;
        return true;
    }

    __host__ __device__ __forceinline__ bool next() { return step() && skip_empty(); }
};

// tcgen05 ---------------------------------------------------------------------

// Shared-memory descriptor of an operand in 128-byte rows with the 128-byte
// swizzle.  K-major: 8-row groups 1024 bytes apart (the leading offset is not
// used).  MN-major: groups of 8 along K 1024 bytes apart, panels of 64 along
// N `lead` bytes apart.
// Only the low word differs between operands of one layout.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead)
{
    return ((saddr & 0x3ffffu) >> 4) | ((lead >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// Rows of 64 bytes with the 64-byte swizzle: 8-row groups 512 bytes apart.
constexpr uint32_t kDescHi64 = (512u >> 4) | (1u << 14) | (4u << 29);

// kind::f16, bf16 x bf16 (or fp16 x fp16) -> fp32, M = 128, N = n, A K-major, B K- or
// MN-major.
__host__ __device__ constexpr uint32_t ca_idesc(int n, bool b_mn, bool f16 = false)
{
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kTile >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}\n" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}

// kind::f8f6f4, e4m3 x e4m3 -> fp32, M = 128, N = n, both K-major.
__host__ __device__ constexpr uint32_t ca_idesc8(int n)
{
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(kTile >> 4) << 24);
}

template <uint32_t HI>
__device__ __forceinline__ void mma_ss8(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc,
                                        uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}\n" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "n"(HI)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t blo, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(blo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

#define ZP_R32(v, o)                                                                             \
    "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), \
        "=r"(v[o + 6]), "=r"(v[o + 7]), "=r"(v[o + 8]), "=r"(v[o + 9]), "=r"(v[o + 10]),        \
        "=r"(v[o + 11]), "=r"(v[o + 12]), "=r"(v[o + 13]), "=r"(v[o + 14]), "=r"(v[o + 15])
#define ZP_RW16(v, o)                                                                            \
    "+r"(v[o]), "+r"(v[o + 1]), "+r"(v[o + 2]), "+r"(v[o + 3]), "+r"(v[o + 4]), "+r"(v[o + 5]), \
        "+r"(v[o + 6]), "+r"(v[o + 7]), "+r"(v[o + 8]), "+r"(v[o + 9]), "+r"(v[o + 10]),        \
        "+r"(v[o + 11]), "+r"(v[o + 12]), "+r"(v[o + 13]), "+r"(v[o + 14]), "+r"(v[o + 15])
#define ZP_IN16(v, o)                                                                        \
    "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]),   \
        "r"(v[o + 6]), "r"(v[o + 7]), "r"(v[o + 8]), "r"(v[o + 9]), "r"(v[o + 10]),         \
        "r"(v[o + 11]), "r"(v[o + 12]), "r"(v[o + 13]), "r"(v[o + 14]), "r"(v[o + 15])

// Starts loading 16 columns of this thread's lane into v[o ..]; ld_wait makes
// them valid.
template <int N>
__device__ __forceinline__ void ld16(uint32_t t, uint32_t (&v)[N], int o)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : ZP_R32(v, o)
        : "r"(t));
}

template <int N>
__device__ __forceinline__ void ld_wait(uint32_t (&v)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int o = 0; o < N; o += 16)  // the values are used only after the wait
        asm volatile("" : ZP_RW16(v, o));
}

template <int N>
__device__ __forceinline__ void st16(uint32_t t, const uint32_t (&v)[N], int o)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(t),
        ZP_IN16(v, o)
        : "memory");
}

__device__ __forceinline__ void st8(uint32_t t, const uint32_t (&v)[8])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
        : "memory");
}

__device__ __forceinline__ void st_wait()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// True in one lane of a converged warp.  The instructions that take uniform
// registers (products, tensor copies) issue back to back only where the
// compiler knows that a single lane runs them.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}\n"
        : "=r"(p));
    return p != 0;
}

// Bounded waits, all for this CTA's own work: 32 M tries, which the hardware
// lets last 72 clocks (with 640 threads waiting) to 2,600 (with one): a second or
// more.  A wait ends within microseconds, in the second walk (see the head of the
// file) within a few hundred.  No sleeping in between: the 64 ns naps of
// mbar_wait cost 10 to 30 % of the kernel's time (256 speculative chunks 314 ->
// 295 us, 16 prompts 752 -> 687 us), and a look at the clock as much.
constexpr uint32_t kCaSpins = 1u << 25;

__device__ __forceinline__ bool ca_wait(uint64_t *bar, uint32_t parity)
{
    const uint32_t addr = smem_u32(bar);
    for (uint32_t i = 0; i < kCaSpins; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(done)
            : "r"(addr), "r"(parity)
            : "memory");
        if (done)
            return true;
    }
    return false;
}

// Whether the phase is over, without a wait; a converged warp's.
__device__ __forceinline__ bool warp_test(uint64_t *bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return __all_sync(0xffffffffu, done);
}

// A converged warp's wait.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, ca_wait(bar, parity));
}

__device__ __forceinline__ void bar_sync(uint32_t id, uint32_t threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The barrier of bar_sync; whether v holds for any of the threads.
__device__ __forceinline__ bool bar_any(uint32_t id, uint32_t threads, bool v)
{
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %3, 0;\n\t"
        "bar.red.or.pred q, %1, %2, p;\n\t"
        "selp.b32 %0, 1, 0, q;\n\t}\n"
        : "=r"(any)
        : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(v))
        : "memory");
    return any != 0;
}

// Two bf16 numbers, each 0 where it is not finite.
__device__ __forceinline__ uint32_t finite2(uint32_t v)
{
    if ((v & 0x7f80u) == 0x7f80u)
        v &= 0xffff0000u;
    if ((v & 0x7f800000u) == 0x7f800000u)
        v &= 0xffffu;
    return v;
}

__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v)
{
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Two fp32 operations at once.
__device__ __forceinline__ void fma2(float &x, float &y, float m, float c)
{
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmov.b64 d, {%3, %3};\n\t"
        "fma.rn.f32x2 a, a, b, d;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(m), "f"(c));
}

__device__ __forceinline__ void add2(float &x, float &y, float u, float v)
{
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(u), "f"(v));
}

__device__ __forceinline__ void st_global_v8(void *p, const uint32_t (&v)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Bytes that a barrier's copies will bring, the arrival left for later.
__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                 "r"(bytes)
                 : "memory");
}

// Four fp32 numbers from shared memory.
__device__ __forceinline__ float4 ld_shared_f32x4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

// Two fp16 numbers to e4m3.
__device__ __forceinline__ uint32_t e4m3x2_of_f16(uint32_t v)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
    return r;
}

// What a logit over an 8-bit cache is multiplied by: its row's factor times its block's scale.
// Never 0, so that a masked score, -infinity, stays that (a row of zeros has a factor of about
// 2^-138, a block of zeros a scale of 2^-32), and finite, so that a score of 0 does; NaN stays NaN.
__device__ __forceinline__ float logit_factor(float row, float scale)
{
    float f;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(row * scale), "f"(__uint_as_float(0x00800000u)));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(f), "f"(__uint_as_float(0x7f7fffffu)));
    return f;
}

// The workspace slot of a partial result: O [256][D], then (max, sum) [256].
template <int D>
__device__ __forceinline__ float *slot_ptr(float *part, int slot)
{
    return part + static_cast<size_t>(slot) * (2 * kTile * (D + 2));
}

// Rows 16 part .. + 15 of a tile of 8-bit V, as its map leaves it at `from`, to fp16 in
// the layout of a bf16 tile at `to`, by one warp.  Rows from `first` on are tidied: to 0, or
// with `clean` their NaN to 0.  All chunks of 16 bytes are on their way at once; each
// becomes two.  The lanes of a 16-byte access (eight at a time) lie in different banks
// on both sides: with 128 dims they are four chunks of rows r and r ^ 5, whose
// swizzles differ in the bit that parts the loads' chunks and in the one that parts the
// stores'; with 64 dims two whole rows.
template <int D>
__device__ __forceinline__ void convert_v(uint32_t from, uint32_t to, int part, int lane,
                                          int first, bool clean)
{
    constexpr int STEPS = kTile * D / 16 / (32 * kSmWarps);
    const int ch = D == 128 ? (lane & 3) | (lane >> 3 & 1) << 2 : lane & 3;
    // the rows of step i: row[i & 1] + 8 * (i / 2), or row[0] + 8 i
    int row[2];
    uint32_t src[2], dst[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        row[k] = kTile / kSmWarps * part +
                 (D == 128 ? (k << 1 | lane >> 4) ^ ((lane >> 2 & 1) * 5) : lane >> 2);
        src[k] = from + swz8<D>(row[k], ch);
        dst[k] = to + swz(row[k], 2 * ch, kTile);
    }
    uint4 v[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        v[i] = ld_shared_v4(src[D == 128 ? i & 1 : 0] + (D == 128 ? i / 2 * 1024 : i * 512));
    if (first < kTile) {  // the whole warp alike
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
            if ((D == 128 ? row[i & 1] + 8 * (i / 2) : row[0] + 8 * i) >= first)
                v[i] = clean ? make_uint4(numbers4(v[i].x), numbers4(v[i].y), numbers4(v[i].z),
                                          numbers4(v[i].w))
                             : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const uint32_t at = dst[D == 128 ? i & 1 : 0] + (D == 128 ? i / 2 : i) * 1024;
        st_shared_v4(at, make_uint4(f16x2_of_e4m3(v[i].x), f16x2_of_e4m3(v[i].x >> 16),
                                    f16x2_of_e4m3(v[i].y), f16x2_of_e4m3(v[i].y >> 16)));
        st_shared_v4(at ^ 16, make_uint4(f16x2_of_e4m3(v[i].z), f16x2_of_e4m3(v[i].z >> 16),
                                         f16x2_of_e4m3(v[i].w), f16x2_of_e4m3(v[i].w >> 16)));
    }
}

// Q of an 8-bit cache's chunk: row r of the tile at `from`, bf16 as its map leaves it, becomes
// two rows of e4m3 numbers, f q = upper + lower, `upper` in the first half of the tile at
// `to` and `lower` in its second (with 128 dims the same tile, where a row's numbers lie
// where the row did).  The power of two f takes the row's largest element
// into (224, 448]; four bits of mantissa and then four more hold the eight of a bf16
// number exactly down to a 2^-10 of that, and below it the error stays under a 2^-17 of
// the largest.  factor[r] becomes what a logit of the row is multiplied by, scale / f (NaN
// for a row that is not finite); a negative scale goes into the numbers.  By a stream's
// 256 threads, ct the number of one, two neighbours a row.
template <int D>
__device__ __forceinline__ void split_q(uint32_t from, uint32_t to, int ct, int rows,
                                        float logit_scale, float *factor)
{
    constexpr int CH = D / 16;     // 16-byte chunks of bf16 a thread
    constexpr int LO = kTile * D;  // from `upper` to `lower`
    const int r = ct >> 1, hf = ct & 1;
    if ((r & ~15) >= rows)  // none of the warp's 16 rows
        return;
    uint4 v[CH];
    uint32_t most = 0;
    // (with 128 dims in another order in the second half, for the banks' sake)
    const int flip = D == 128 ? hf * 4 : 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        v[c] = ld_shared_v4(from + swz(r, hf * CH + (c ^ flip), kTile));
        const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            most = __vmaxu2(most, w[e] & 0x7fff7fffu);
    }
    most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = max(most << 16, most & 0xffff0000u);
    __syncwarp();  // the row is read
    // f = 2^e; two factors, as it may not be an fp32 number
    const int e = 8 - (static_cast<int>(most >> 23) - 127) - ((most & 0x7fffffu) > 0x600000u);
    const int e1 = max(min(e, 100), -100), e2 = e - e1;
    const float f1 = __uint_as_float(exp2_bits(e1) | (__float_as_uint(logit_scale) & 0x80000000u));
    const float f2 = __uint_as_float(exp2_bits(e2));
    // a loop, as the code runs once an item and comes from memory (256 chunks of 2 to 9: in line
    // 304 us, so 299)
#pragma unroll 1
    for (int c = 0; c < CH; c += 2) {
        uint32_t up[4], lo[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            uint32_t u8[4], l8[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x = pack_f16x2(__uint_as_float(w[i] << 16) * f1 * f2,
                                              __uint_as_float(w[i] & 0xffff0000u) * f1 * f2);
                u8[i] = e4m3x2_of_f16(x);
                const uint32_t b = f16x2_of_e4m3(u8[i]);
                const __half2 rest = __hsub2(*reinterpret_cast<const __half2 *>(&x),
                                             *reinterpret_cast<const __half2 *>(&b));
                l8[i] = e4m3x2_of_f16(*reinterpret_cast<const uint32_t *>(&rest));
            }
            up[2 * k] = u8[0] | u8[1] << 16;
            up[2 * k + 1] = u8[2] | u8[3] << 16;
            lo[2 * k] = l8[0] | l8[1] << 16;
            lo[2 * k + 1] = l8[2] | l8[3] << 16;
        }
        const uint32_t at = to + swz8<D>(r, (hf * CH + (c ^ flip)) / 2);
        st_shared_v4(at, make_uint4(up[0], up[1], up[2], up[3]));
        st_shared_v4(at + LO, make_uint4(lo[0], lo[1], lo[2], lo[3]));
#pragma unroll
        for (int k = 0; k + 2 < CH; ++k)
            v[k] = v[k + 2];
    }
    const float back = fabsf(logit_scale) * __uint_as_float(exp2_bits(-e1)) *
                       __uint_as_float(exp2_bits(-e2));
    if (hf == 0)
        factor[r] = most < 0x7f800000u ? back : INFINITY - INFINITY;
}

}  // namespace

// F8: over an 8-bit cache.
template <int D, bool F8>
__global__ void __launch_bounds__(kCaThreads, 1)
    zp_chunk_attn_kernel(const __grid_constant__ ChunkAttnArgs a)
{
    using S = CaSmem<D, F8>;
    constexpr int PANELS = S::PANELS, NK = S::NK, NV = S::NV, NR = S::NR, XC = S::XC;
    extern __shared__ __align__(1024) uint8_t sm[];
    if (smem_u32(sm) & 1023u) {  // the swizzled tiles need it
        if (threadIdx.x == 0)
            set_error(a.sticky, ZP_ERR_UNSUPPORTED);
        return;
    }
    uint8_t *sQ = sm + S::off_q, *sK = sm + S::off_k, *sV = sm + S::off_v;
    float *sMax = reinterpret_cast<float *>(sm + S::off_max);
    CaDesc *sDesc = reinterpret_cast<CaDesc *>(sm + S::off_desc);
    CaPlan &plan = *reinterpret_cast<CaPlan *>(sm + S::off_plan);
    long long *scan = reinterpret_cast<long long *>(sm + S::off_scan);
    uint64_t *kfull = reinterpret_cast<uint64_t *>(sm + S::off_bar), *kempty = kfull + NK;
    uint64_t *vfull = kempty + NK, *vempty = vfull + NV, *sfull = vempty + NV, *pready = sfull + 2;
    uint64_t *ofull = pready + 2, *oempty = ofull + 2, *qfull = oempty + 2, *qempty = qfull + 2;
    uint64_t *turn = qempty + 2, *described = turn + 2, *read = described + kDescs;
    uint64_t *half = read + kDescs, *taken = half + 1, *done = taken + 1;
    uint64_t *rfull = done + 1, *rempty = rfull + 2 * NR, *qready = rempty + NR;  // F8 alone
    const uint32_t scales_at = smem_u32(sm + S::off_scale);
    float *sQf = reinterpret_cast<float *>(sm + S::off_qf);
    uint32_t *sTmem = reinterpret_cast<uint32_t *>(sm + S::off_tmem);
    int *sLast = reinterpret_cast<int *>(sm + S::off_last);

    const int tid = threadIdx.x, lane = tid & 31, wi = tid >> 5;
    const int G = a.Hq / a.Hkv, tpt = tile_tokens(G);
    const bool duos = F8 && a.duos;

    if (tid == 0) {
        for (int s = 0; s < NK; ++s) {
            mbar_init(&kfull[s], 1);
            mbar_init(&kempty[s], 2);  // both products' warps have passed it
        }
        for (int s = 0; s < NV; ++s) {
            mbar_init(&vfull[s], F8 ? kSmWarps : 1);
            mbar_init(&vempty[s], 2);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&sfull[x], 1);
            mbar_init(&pready[x], kSmWarps);
            mbar_init(&ofull[x], 1);
            mbar_init(&oempty[x], kSmWarps);
            mbar_init(&qfull[x], 1);
            mbar_init(&qempty[x], 2);
            mbar_init(&turn[x], 1);
            if constexpr (F8)
                mbar_init(&qready[x], kSmWarps);
        }
        for (int s = 0; s < NR; ++s) {
            mbar_init(&rfull[s], 1);
            mbar_init(&rfull[NR + s], 1);
            mbar_init(&rempty[s], kSmWarps);
        }
        for (int s = 0; s < kDescs; ++s) {
            mbar_init(&described[s], 1);
            mbar_init(&read[s], 2 * kSmWarps + 3);
        }
        mbar_init(half, kSmWarps);
        mbar_init(taken, kSmWarps);
        mbar_init(done, 2);
        mbar_arrive(&turn[0]);  // A begins
        fence_mbar_init();
    }
    if (wi == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(sTmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == kLoadWarp * 32) {  // the maps' first use waits for them else
        asm volatile("prefetch.tensormap [%0];" ::"l"(a.kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(a.vmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&a.qmap) : "memory");
    }
    pdl_wait();  // launched early: everything of the kernels before it is visible from here
    if (F8 && a.visible && blockIdx.x == 0 && tid == 0)
        say_visible(a.visible);
    pdl_launch_dependents();

    // the call's set of arrivals (a thread with no requests of its own in most batches)
    if (tid == kLoadVWarp * 32) {
        const unsigned set = 2 * gridDim.x;
        const bool second = atomicInc(a.entered, 2 * gridDim.x - 1) >= gridDim.x;
        uint32_t *other = a.arrived + (second ? 0 : set) + 2 * blockIdx.x;
        other[0] = other[1] = 0;
        sLast[2] = second ? set : 0;
        sLast[3] = sLast[4] = sLast[5] = 0;
    }

    // the shares: thread t adds up a contiguous run of requests
    {
        const int per = (a.R + kCaThreads - 1) / kCaThreads;
        const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
        long long mine = 0;
        int longest = 0;
        ChunkReq c;  // the last one
        for (int i = r0; i < r1; ++i) {
            bool bad;
            if (attn_request(a, i, c, &bad)) {
                mine += request_cost(c, tpt, a.Hkv, duos);
                longest = max(longest, heads_by_two(c.n, tpt, a.Hkv, duos) ? item_cost(c.len, false)
                                                                           : longest_item(c, tpt));
            }
            if (bad && blockIdx.x == 0)
                set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
        }
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += y;
        }
        longest = __reduce_max_sync(0xffffffffu, longest);
        if (tid == 0)
            sLast[0] = 0;
        __syncthreads();
        if (lane == 31) {
            scan[wi] = incl;
            atomicMax(&sLast[0], longest);
        }
        __syncthreads();
        long long before = incl - mine, cost;
        {
            long long v = lane < kCaThreads / 32 ? scan[lane] : 0;
            const long long own = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o)
                    v += y;
            }
            cost = __shfl_sync(0xffffffffu, v, 31);
            before += __shfl_sync(0xffffffffu, v - own, wi);
        }
        CaPlan p;
        make_shares(p, cost, sLast[0], static_cast<int>(gridDim.x));
        p.lo = share_border(p, blockIdx.x);
        p.hi = share_border(p, blockIdx.x + 1);
        if (tid == 0 && p.lo >= p.hi)
            plan = p;
        if (before <= p.lo && p.lo < before + mine) {
            p.i0 = r0;
            p.c0 = c;
            for (int i = r0; i < r1 && per > 1; ++i) {  // the request the share begins in
                bool bad;
                if (!attn_request(a, i, p.c0, &bad))
                    continue;
                p.i0 = i;
                const long long w = request_cost(p.c0, tpt, a.Hkv, duos);
                if (p.lo < before + w)
                    break;
                before += w;
            }
            p.x0 = before;
            plan = p;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *sTmem;
    bool bad = false;
    uint32_t nd = 0;  // items this warp has gone through

    // The next item's description, or null at the end; a warp lets it go with
    // `leave` once it no longer reads it.  (A warp that gave up still follows
    // the descriptions: the barriers of its group count on it.)
    auto enter = [&]() -> const CaDesc * {
        const int j = nd % kDescs;
        if (!warp_wait(&described[j], (nd / kDescs) & 1)) {
            bad = true;
            return nullptr;
        }
        return sDesc[j].ntok ? &sDesc[j] : nullptr;
    };
    auto leave = [&] {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&read[nd % kDescs]);
        ++nd;
    };

    // At the end of a walk, every warp of the CTA: whether a second one follows.
    auto walk_again = [&](bool clean) {
        if (bad && lane == 0)
            atomicOr(&sLast[3], 2);
        fence_before();
        bar_sync(0, kCaThreads);
        return !clean && *static_cast<volatile int *>(&sLast[3]) == 1;
    };
    auto ended_clean = [&] { return sDesc[nd % kDescs].clean != 0; };  // at an end's description

    if (wi >= 2 * kSmWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        // The tiles of a ring: eight cache blocks of 16 keys, PANELS boxes each.
        // A lane holds the pool row of a block of this kv head (negative past the
        // request's blocks: the load then fills zeros), four tiles at a time and
        // the next four ahead.
        auto block_y = [&](const CaDesc &d, int q) {
            if (q * kBlk >= d.len)
                return -kBlk;
            const int blk = block_at(a, d.row, q);
            if (blk < 0 || blk >= a.num_blocks) {
                set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
                return -kBlk;
            }
            return (blk * a.Hkv + d.h) * kBlk;
        };
        auto load_tile = [&](const CUtensorMap *map, uint8_t *dst, uint64_t *bar, int ids, int t) {
            int y[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                y[q] = __shfl_sync(0xffffffffu, ids, (t & 3) * 8 + q);
            if (elect_one()) {
                if constexpr (F8) {  // a box a block; the arrival is the caller's
                    mbar_expect_tx(bar, S::TILE8);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        tma_load_2d(dst + q * kBlk * D, map, 0, y[q], bar);
                } else {
                    mbar_arrive_expect_tx(bar, S::TILE);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
#pragma unroll
                        for (int p = 0; p < PANELS; ++p)
                            tma_load_2d(dst + p * S::PANEL + q * kBlk * 128, map, p * 64, y[q],
                                        bar);
                }
            }
            __syncwarp();
        };
        // The same pool rows of the next kv head.
        auto next_head = [&](int ids) { return ids < 0 ? ids : ids + kBlk; };
        // The scales of the block whose pool row is y: K's and V's.
        auto scales_of = [&](int y) {
            const int at = y < 0 ? 0 : y / kBlk;
            const float ks = y < 0 ? 1.f : a.kscale[at], vs = y < 0 ? 1.f : a.vscale[at];
            return make_float2(ks, vs);
        };
        if (wi == kLoadWarp) {
            // ------------------------------------------- the items, Q and K
            uint32_t loaded = 0, cur = 0, par = 0, qs = 0;  // ring cursor and parity, query tiles
            auto load_q = [&](const CaDesc &d, int tiles) {
                for (int x = 0; x < tiles; ++x, ++qs) {
                    const int k = qs & 1;
                    if (qs >= 2 && !warp_wait(&qempty[k], ((qs >> 1) - 1) & 1)) {
                        bad = true;
                        break;
                    }
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&qfull[k], PANELS * G * tpt * 128);
#pragma unroll
                        for (int p = 0; p < PANELS; ++p)
                            asm volatile(
                                "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier"
                                "::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                                    smem_u32(sQ + k * S::TILE + p * S::PANEL)),
                                "l"(&a.qmap), "r"(p * 64), "r"((d.h + (F8 && d.duo ? x : 0)) * G),
                                "r"(d.row0 + (F8 && d.duo ? 0 : x * tpt)), "r"(smem_u32(&qfull[k]))
                                : "memory");
                    }
                    __syncwarp();
                }
            };
            for (bool clean = false;; clean = true) {
                CaWalk wk{a, plan, tpt, {}, duos};
                bool more = wk.begin();
                for (; !bad; more = wk.next()) {
                    const CaItem &it = wk.it;
                    const int j = nd % kDescs;
                    if (nd >= kDescs && !warp_wait(&read[j], (nd / kDescs - 1) & 1)) {
                        bad = true;
                        break;
                    }
                    CaDesc d;
                    d.row0 = it.c.first + it.tok0;
                    d.ntok = more ? it.ntok : 0;
                    d.h = it.duo ? 2 * it.h : it.h;
                    d.pos0 = it.c.len - it.c.n + it.tok0;
                    d.len = it.c.len;
                    d.row = it.c.row;
                    d.ka = it.ka;
                    d.kb = it.kb;
                    d.kt = it.kt;
                    d.w = it.w;
                    d.clean = clean;
                    d.duo = it.duo;
                    d.x = it.x;
                    if (lane == 0) {
                        sDesc[j] = d;
                        mbar_arrive(&described[j]);
                    }
                    __syncwarp();
                    ++nd;
                    if (!more)
                        break;
                    const int len = d.kb - d.ka;
                    int ids = block_y(d, d.ka * 8 + lane);
                    int ids_next = len > 4 ? block_y(d, (d.ka + 4) * 8 + lane) : 0;
                    // F8: scales, of a duo's second head too; its key tiles come in turn
                    const bool duo = F8 && d.duo;
                    [[maybe_unused]] float2 sc[2] = {}, sc_next[2] = {};
                    if constexpr (F8) {
                        sc[0] = scales_of(ids);
                        sc[1] = duo ? scales_of(next_head(ids)) : sc[0];
                    }
                    const int tiles = it.single ? 1 : 2;
                    const bool q_early = qs == 0;  // the first item's: while the block ids come
                    if (q_early)
                        load_q(d, tiles);
                    for (int i = 0; i < (duo ? 2 * len : len); ++i) {
                        const int t = duo ? i >> 1 : i, second = duo ? i & 1 : 0;
                        if (t > 0 && (t & 3) == 0 && !second) {
                            ids = ids_next;
                            ids_next = t + 4 < len ? block_y(d, (d.ka + t + 4) * 8 + lane) : 0;
                        }
                        if (loaded >= NK && !warp_wait(&kempty[cur], par ^ 1)) {
                            bad = true;
                            break;
                        }
                        load_tile(a.kmap, sK + cur * S::KTILE, &kfull[cur],
                                  second ? next_head(ids) : ids, t);
                        if constexpr (F8) {
                            // the tile's scales, which the softmax reads once S has arrived
                            if (t > 0 && (t & 3) == 0 && !second) {
                                sc[0] = sc_next[0];
                                sc[1] = sc_next[1];
                            }
                            if ((t & 3) == 2 && t + 2 < len && !second) {
                                sc_next[0] = scales_of(ids_next);
                                sc_next[1] = duo ? scales_of(next_head(ids_next)) : sc_next[0];
                            }
                            const float2 now = second ? sc[1] : sc[0];
                            if ((lane >> 3) == (t & 3))
                                st_shared_v4(
                                    scales_at + ((loaded % kScales) * 8 + (lane & 7)) * 16,
                                    make_uint4(__float_as_uint(now.x),
                                               __float_as_uint(log2f(now.y)),
                                               __float_as_uint(1.f / now.y), 0u));
                            __syncwarp();
                            if (elect_one())
                                mbar_arrive(&kfull[cur]);
                            __syncwarp();
                        }
                        ++loaded;
                        if (++cur == NK) {
                            cur = 0;
                            par ^= 1;
                        }
                        // Q behind the first K tile, which does not wait for the item before
                        if (i > 0)
                            continue;
                        if (!q_early)
                            load_q(d, tiles);
                        if (bad)
                            break;
                    }
                }
                // every copy issued has landed before the CTA may exit
                for (uint32_t k = qs > 2 ? qs - 2 : 0; k < qs; ++k)
                    bad |= !warp_wait(&qfull[k & 1], (k >> 1) & 1);
                for (uint32_t k = loaded > NK ? loaded - NK : 0; k < loaded; ++k)
                    bad |= !warp_wait(&kfull[k % NK], (k / NK) & 1);
                if (!walk_again(clean))
                    break;
            }
        } else if (wi == kLoadVWarp) {
            // ------------------------------------------------------------- V
            uint32_t loaded = 0, cur = 0, par = 0;
            constexpr uint32_t N = F8 ? NR : NV;  // 8-bit tiles go into a ring of their own
            uint64_t *empty = F8 ? rempty : vempty;
            // 8-bit: the tiles that A converts have barriers of their own, and so do B's, as a
            // stream does not wait for the other's: it could take the phase before last, of a
            // tile that it did not wait for, for the one that it waits for
            [[maybe_unused]] uint32_t owned[2] = {0, 0};
            for (;;) {
                while (const CaDesc *dp = bad ? nullptr : enter()) {
                    const CaDesc d = *dp;
                    leave();
                    const int len = d.kb - d.ka;
                    int ids = block_y(d, d.ka * 8 + lane);
                    int ids_next = len > 4 ? block_y(d, (d.ka + 4) * 8 + lane) : 0;
                    const bool duo = F8 && d.duo;
                    for (int i = 0; i < (duo ? 2 * len : len); ++i) {
                        const int t = duo ? i >> 1 : i, second = duo ? i & 1 : 0;
                        if (t > 0 && (t & 3) == 0 && !second) {
                            ids = ids_next;
                            ids_next = t + 4 < len ? block_y(d, (d.ka + t + 4) * 8 + lane) : 0;
                        }
                        if (loaded >= N && !warp_wait(&empty[cur], par ^ 1)) {
                            bad = true;
                            break;
                        }
                        uint64_t *full = &vfull[cur];
                        if constexpr (F8) {
                            const bool b = d.ntok <= tpt && (i & 1);  // in turn, and B's
                            full = &rfull[(b ? NR : 0) + (b ? owned[1] : owned[0]) % N];
                            ++(b ? owned[1] : owned[0]);
                        }
                        load_tile(a.vmap,
                                  F8 ? sm + S::off_raw + cur * S::TILE8 : sV + cur * S::TILE, full,
                                  second ? next_head(ids) : ids, t);
                        if constexpr (F8) {
                            if (elect_one())
                                mbar_arrive(full);
                            __syncwarp();
                        }
                        ++loaded;
                        if (++cur == N) {
                            cur = 0;
                            par ^= 1;
                        }
                    }
                }
                auto landed = [&](uint64_t *full, uint32_t n) {
                    for (uint32_t k = n > N ? n - N : 0; k < n; ++k)
                        bad |= !warp_wait(&full[k % N], (k / N) & 1);
                };
                if constexpr (F8) {
                    landed(rfull, owned[0]);
                    landed(rfull + NR, owned[1]);
                } else {
                    landed(vfull, loaded);
                }
                if (!walk_again(ended_clean()))
                    break;
                leave();
            }
        } else {
            // ----------------------------------------------------- products
            // One warp a stream, so that the waits of one lie beside the products of
            // the other (the issue of a product waits for a place in a short queue).
            // They take turns at P V and the next S: products of both in the queue
            // at once would end at the same time, and so would the two softmaxes,
            // with nothing left to run beside them.  Both pass every stage of the
            // rings, used or not: a stage's parity then never runs ahead of a warp.
            // The whole warp waits; one lane issues.
            // (a negative scale negates Q in the product: bit 13)
            const uint32_t ID_S =
                F8 ? ca_idesc8(kTile)
                   : ca_idesc(kTile, false) | (a.logit_scale < 0.f ? 1u << 13 : 0u);
            constexpr uint32_t ID_O = ca_idesc(D, true, F8);
            constexpr uint32_t STEP = S::TILE >> 4, KSTEP = S::KTILE >> 4;
            const int x = wi - kMmaWarp;
            const uint32_t qdesc = desc_lo(smem_u32(sQ) + (S::SPLIT ? 2 * S::TILE : 0), 16);
            const uint32_t kdesc = desc_lo(smem_u32(sK), 16);
            const uint32_t vdesc = desc_lo(smem_u32(sV), S::PANEL);
            const uint32_t tS = tmem + x * kTile, tO = tmem + 256 + x * kTile;
            uint32_t kc = 0, kpar = 0, vc = 0, vpar = 0;  // ring cursors and parities
            uint32_t qs = 0, np = 0, no = 0, turns = 0;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (!bad && !warp_wait(bar, parity))
                    bad = true;
            };
            auto k_on = [&] {
                if (++kc == NK) {
                    kc = 0;
                    kpar ^= 1;
                }
            };
            auto v_on = [&] {
                if (++vc == NV) {
                    vc = 0;
                    vpar ^= 1;
                }
            };
            auto tell = [&](uint64_t *bar) {
                if (elect_one())
                    mbar_arrive(bar);
                __syncwarp();
            };
            uint32_t walks = 0;
            for (;;) {
                while (const CaDesc *dp = bad ? nullptr : enter()) {
                    const bool duo = F8 && dp->duo;
                    const int ka = dp->ka, kb = dp->kb, len = duo ? 2 * (kb - ka) : kb - ka;
                    const bool single = dp->ntok <= tpt && !duo;
                    const bool in_turn = single || duo;  // the key tiles are A's and B's in turn
                    // the key from which on V is tidied, negative in the second walk
                    const int tidy = dp->clean ? -(dp->pos0 + 1) : dp->len;
                    // the stream's key tiles: t with t % 2 == x of a single item or a duo; of
                    // a pair all for B, the ones its last token sees for A
                    const int na =
                        x == 0 ? (dp->pos0 + min(dp->ntok, tpt) + kTile - 1) / kTile : kb;
                    leave();
                    const int cnt = in_turn ? (len + 1 - x) / 2 : max(0, min(kb, na) - ka);
                    const int last = in_turn ? 2 * (cnt - 1) + x : cnt - 1;  // the last one
                    const uint32_t slot = single ? qs : qs + x;
                    const uint32_t qd = __shfl_sync(0xffffffffu, qdesc + (slot & 1) * STEP, 0);
                    auto skip_k = [&] {  // a tile of the other stream's
                        wait(&kfull[kc], kpar);
                        if (bad)
                            return;
                        tell(&kempty[kc]);
                        k_on();
                    };
                    auto skip_v = [&] {
                        wait(&vfull[vc], vpar);
                        if (bad)
                            return;
                        tell(&vempty[vc]);
                        v_on();
                    };
                    auto issue_s = [&](uint32_t kd, int from, int to) {
#pragma unroll
                        for (int ks = from; ks < to; ++ks) {
                            if constexpr (F8) {  // Q's upper parts, then its lower ones
                                constexpr int N = D / 32;
                                const uint32_t o = (ks % N * 32) >> 4;
                                mma_ss8<D == 128 ? kDescHi : kDescHi64>(
                                    tS, qd + (ks / N * S::TILE8 >> 4) + o, kd + o, ID_S, ks > 0);
                            } else {
                                const uint32_t o = ((ks >> 2) * S::PANEL + (ks & 3) * 32) >> 4;
                                mma_ss(tS, qd + o, kd + o, ID_S, ks > 0);
                            }
                        }
                    };
                    auto done_s = [&](int t) {
                        mma_commit(&sfull[x]);
                        mma_commit(&kempty[kc]);
                        if (t == last)
                            mma_commit(&qempty[slot & 1]);
                    };
                    auto first_s = [&](bool mine, int t) {
                        if (!mine) {
                            skip_k();
                            return;
                        }
                        wait(&kfull[kc], kpar);
                        if (bad)
                            return;
                        fence_after();
                        const uint32_t kd = __shfl_sync(0xffffffffu, kdesc + kc * KSTEP, 0);
                        if (elect_one()) {
                            issue_s(kd, 0, D / 16);
                            done_s(t);
                        }
                        __syncwarp();
                        k_on();
                    };
                    // P V with V tile t, then S with K tile `next`
                    auto burst = [&](int t, int next) {
                        wait(&vfull[vc], vpar);
                        // rows that may hold what is not finite and counts as 0: the rest of the
                        // last cached block, or in the second walk all but the first token's keys
                        // (both streams may tidy a tile at once: each writes zeros alone)
                        const int from = max(abs(tidy) - (ka + t) * kTile, 0);
                        if (!F8 && from < kTile && (tidy < 0 || (from & (kBlk - 1))) && !bad) {
                            const int end = tidy < 0 ? kTile : (from + kBlk - 1) / kBlk * kBlk;
                            for (int c = from * (D / 8) + lane; c < end * (D / 8); c += 32) {
                                const uint32_t at = smem_u32(sV + vc * S::TILE) +
                                                    swz(c / (D / 8), c % (D / 8), kTile);
                                const uint4 v = ld_shared_v4(at);
                                const uint4 f = make_uint4(finite2(v.x), finite2(v.y), finite2(v.z),
                                                           finite2(v.w));
                                if (((v.x ^ f.x) | (v.y ^ f.y) | (v.z ^ f.z) | (v.w ^ f.w)) != 0)
                                    st_shared_v4(at, f);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        if (next < len)
                            wait(&kfull[kc], kpar);
                        const bool first = t == (in_turn ? x : 0);
                        if (first) {  // the epilogue of O's last use has read it
                            if (no > 0)
                                wait(&oempty[x], (no - 1) & 1);
                            ++no;
                        }
                        const uint32_t vd = __shfl_sync(0xffffffffu, vdesc + vc * STEP, 0);
                        const uint32_t kd = __shfl_sync(0xffffffffu, kdesc + kc * KSTEP, 0);
                        const bool more_s = next <= last;
                        wait(&turn[x], turns++ & 1);
                        wait(&pready[x], np++ & 1);
                        if (bad)
                            return;
                        fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int ks = 0; ks < kTile / 16; ++ks)
                                mma_ts(tO, tS + ks * 8, vd + ks * (2048 >> 4), ID_O,
                                       !first || ks > 0);
                            mma_commit(&vempty[vc]);
                            if (t == last)
                                mma_commit(&ofull[x]);
                            // the other stream wakes up while the rest is queued
                            if (more_s) {
                                issue_s(kd, 0, D / 32);
                                mbar_arrive(&turn[1 - x]);
                                issue_s(kd, D / 32, D / 16);
                                done_s(next);
                            } else {
                                mbar_arrive(&turn[1 - x]);
                            }
                        }
                        __syncwarp();
                        v_on();
                        if (more_s)
                            k_on();
                        if (next < len && next > last) {
                            tell(&kempty[kc]);
                            k_on();
                        }
                    };
                    auto no_burst = [&] {
                        wait(&turn[x], turns++ & 1);
                        if (!bad)
                            tell(&turn[1 - x]);
                    };
                    uint64_t *q_there = F8 ? qready : qfull;
                    wait(&q_there[qs & 1], (qs >> 1) & 1);
                    if (!single)
                        wait(&q_there[(qs + 1) & 1], ((qs + 1) >> 1) & 1);
                    if (bad)
                        break;
                    if (!single)
                        tell(&qempty[(qs + 1 - x) & 1]);  // the other stream's queries
                    if (cnt == 0)
                        tell(&qempty[slot & 1]);
                    if (in_turn) {  // K0 K1, then V0 K2 | V1 K3 | ..: in turn A's and B's
                        first_s(x == 0, 0);
                        if (len > 1)
                            first_s(x == 1, 1);
                        for (int t = 0; t < len && !bad; t += 2) {
                            if (x == 1) {
                                skip_v();
                                if (t + 2 < len)
                                    skip_k();
                            }
                            if (t + x < len)
                                burst(t + x, t + x + 2);
                            else
                                no_burst();
                            if (x == 0 && t + 1 < len) {
                                skip_v();
                                if (t + 3 < len)
                                    skip_k();
                            }
                        }
                    } else {  // K0, then V0 K1 | V1 K2 | ..
                        first_s(cnt > 0, 0);
                        for (int t = 0; t < len && !bad; ++t) {
                            if (t < cnt) {
                                burst(t, t + 1);
                            } else {
                                skip_v();
                                if (t + 1 < len)
                                    skip_k();
                                no_burst();
                            }
                        }
                    }
                    qs += single ? 1 : 2;
                }
                // every product issued is done before the tensor memory is freed
                if (elect_one())
                    mma_commit(done);
                __syncwarp();
                bad |= !warp_wait(done, walks++ & 1);
                if (!walk_again(ended_clean()))
                    break;
                leave();
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSmRegs));
        // ------------------------------------------------------- softmax
        // A row belongs to two threads, of warps w (columns 0 .. 63 of S and the
        // first half of O's) and w + 4 (the others), which exchange its maximum.
        constexpr int HK = kTile / 2, HD = D / 2;
        // columns of P a store: the widest that the registers allow (16 prompts of 128
        // dims 679 us with 16, 667 with 32; with 64 dims 32 spill)
        constexpr int PC = D == 128 ? 32 : 16;
        const int x = wi / kSmWarps;           // tile A or B
        const int wq = wi & 3;                 // tensor-memory lanes 32 wq ..
        const int hf = (wi >> 2) & 1;          // the row's half
        const int r = wq * 32 + lane;          // row of the tile
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tS = tmem + x * kTile + lane_off;
        const uint32_t tH = tS + hf * HK, tP = tS + hf * (HK / 2);  // this half of S and of P
        const uint32_t tO = (D == 128 ? tH : tP) + 256;             // and of O
        static_assert(HD == (D == 128 ? HK : HK / 2), "O's half lies behind S's or P's");
        const uint32_t max_at = smem_u32(sMax + (x * 2 + hf) * kTile + r);
        constexpr uint32_t kOther = kTile * 4;  // max_at ^ kOther: the other half's
        static_assert(S::off_max % (2 * kOther) == 0, "the halves differ in one bit");
        const uint32_t pair_bar = 1 + x * 4 + wq;  // the barrier of this warp and its other half
        // (above 0, for scores of -infinity; 2^-149 times any finite one is nothing)
        const float ls = fmaxf(fabsf(a.logit_scale), __uint_as_float(1u));
        uint32_t ns = 0, no = 0, halves = 0;
        // F8: query tiles, key tiles and, of these, the stream's V tiles so far
        [[maybe_unused]] uint32_t qs = 0, tiles = 0, raws = 0;
        [[maybe_unused]] bool ahead = false;          // F8: the item's Q is split already
        bool lent = false;  // B: its (max, sum) of a join lie in sMax
        // F8: the item's Q to e4m3, before any of its S: two tiles by their streams, a single
        // one by B, for which A's epilogue has no work
        [[maybe_unused]] auto split = [&](const CaDesc &d) {
            const bool single = d.ntok <= tpt && !d.duo;
            if (single && x == 0)
                return;
            const uint32_t t = single ? qs : qs + x, k = t & 1;
            if (!bad && !ca_wait(&qfull[k], (t >> 1) & 1))
                bad = true;
            bad = __any_sync(0xffffffffu, bad);
            const int toks = min(single || d.duo || x == 0 ? d.ntok : d.ntok - tpt, tpt);
            split_q<D>(smem_u32(sQ) + k * S::TILE, smem_u32(sQ) + (S::SPLIT ? 2 + k : k) * S::TILE,
                       tid & (32 * kSmWarps - 1), toks * G, a.logit_scale,
                       sQf + t % kQTiles * kTile);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&qready[k]);
        };
        for (;;) {
            while (const CaDesc *dp = enter()) {
                const bool duo = F8 && dp->duo, single = dp->ntok <= tpt && !duo;
                const int len = dp->kb - dp->ka, pos0 = dp->pos0;
                // its first token in the item
                const int tile_tok = single || duo || x == 0 ? 0 : tpt;
                const int toks = min(dp->ntok - tile_tok, tpt);   // its tokens
                const int tok = min(r / G, toks - 1);             // rows past the last follow it
                const int lim = pos0 + tile_tok + tok + 1;        // keys the row sees
                const bool live = wq * 32 < toks * G;
                int cnt = single ? (len + 1 - x) / 2 : len;            // key tiles
                if (!single && !duo && x == 0)
                    cnt = max(0, min(dp->kb, (pos0 + tpt + kTile - 1) / kTile) - dp->ka);
                if (lent && cnt > 0) {  // A has taken what B left in place of its maxima
                    if (!bad && !ca_wait(taken, halves++ & 1))
                        bad = true;
                    bad = __any_sync(0xffffffffu, bad);
                    lent = false;
                }
                // keys the thread's half of the next tile still holds for the row: fewer
                // than all for any row of the warp, and the tile is masked
                // F8: what a logit is multiplied by but for K's scale
                [[maybe_unused]] float lr = 0.f;
                [[maybe_unused]] const uint32_t qt = single ? qs : qs + x;
                if constexpr (F8) {
                    if (!ahead)
                        split(*dp);
                    qs += single ? 1 : 2;
                }
                // F8: where the stream's key tile i lies among the item's
                auto nth = [&](int i) { return single || duo ? x + 2 * i : i; };
                // F8: V of the stream's key tile i to fp16, by this stream's warps: a pair's tiles
                // by A, which is ahead of B, others by the stream that uses them
                [[maybe_unused]] auto to_fp16 = [&](int i) {
                    constexpr uint32_t N = F8 ? NR : 1;
                    const uint32_t k = tiles + nth(i), st = k % NV, rs = k % N;
                    const int t = single ? nth(i) : i;
                    if (!bad && (!ca_wait(&rfull[x * NR + raws % N], (raws / N) & 1) ||
                                 (k >= NV && !ca_wait(&vempty[st], (k / NV - 1) & 1))))
                        bad = true;
                    ++raws;
                    bad = __any_sync(0xffffffffu, bad);
                    if (bad)
                        return;
                    // the key from which on rows are tidied: past the length all of them are 0,
                    // in the second walk NaN counts as 0
                    const int tidy = dp->clean ? dp->pos0 + 1 : dp->len;
                    convert_v<D>(smem_u32(sm + S::off_raw + rs * S::TILE8),
                                 smem_u32(sV + st * S::TILE), wi & (kSmWarps - 1), lane,
                                 tidy - (dp->ka + t) * kTile, dp->clean != 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&rempty[rs]);
                        mbar_arrive(&vfull[st]);
                    }
                };
                int m_lim = lim - (dp->ka + (single ? x : 0)) * kTile - hf * HK;
                const int m_step = single ? 2 * kTile : kTile;
                float mref = -INFINITY, negm = 0.f;
                float l0 = 0.f, l1 = 0.f;
                for (int t = cnt; t > 0; --t, m_lim -= m_step) {
                    if constexpr (F8) {
                        if (single || duo || x == 0)
                            to_fp16(cnt - t);
                    }
                    if (!bad && !ca_wait(&sfull[x], ns & 1))
                        bad = true;
                    ++ns;
                    bad = __any_sync(0xffffffffu, bad);
                    if (bad) {
                        if (live)
                            bar_sync(pair_bar, 64);
                        continue;
                    }
                    fence_after();
                    if (live) {
                        uint32_t sr[HK];
#pragma unroll
                        for (int o = 0; o < HK; o += 16)
                            ld16(tH + o, sr, o);
                        ld_wait(sr);
                        float *s = reinterpret_cast<float *>(sr);
                        if (__any_sync(0xffffffffu, m_lim < HK)) {
#pragma unroll
                            for (int c = 0; c < HK; ++c)
                                s[c] = c < m_lim ? s[c] : -INFINITY;
                        }
                        float m_new;
                        // F8: the scales of this half's four blocks
                        [[maybe_unused]] const uint32_t sc_at =
                            scales_at + ((tiles + nth(cnt - t)) % kScales * 8 + hf * 4) * 16;
                        if constexpr (F8) {
                            if (t == cnt)
                                lr = sQf[qt % kQTiles * kTile + r];
                            m_new = -INFINITY;
#pragma unroll
                            for (int b = 0; b < HK; b += kBlk) {
                                float mx[2] = {s[b], s[b + 1]};
#pragma unroll
                                for (int c = 2; c < kBlk; c += 2) {
                                    mx[0] = fmaxf(mx[0], s[b + c]);
                                    mx[1] = fmaxf(mx[1], s[b + c + 1]);
                                }
                                const float4 sc = ld_shared_f32x4(sc_at + b / kBlk * 16);
                                m_new = fmaxf(
                                    m_new, fmaf(fmaxf(mx[0], mx[1]), logit_factor(lr, sc.x), sc.y));
                            }
                        } else {
                            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                            for (int c = 4; c < HK; c += 8) {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    mx[e] = c + 4 + e < HK
                                                ? fmaxf(fmaxf(mx[e], s[c + e]), s[c + 4 + e])
                                                : fmaxf(mx[e], s[c + e]);
                            }
                            m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        }
                        st_shared_f32(max_at, m_new);
                        bar_sync(pair_bar, 64);  // also: both halves of S are in registers
                        m_new = fmaxf(m_new, ld_shared_f32(max_at ^ kOther));
                        const bool up = F8 ? m_new - mref > kRescale8  // or the first: infinite
                                           : (m_new - mref) * ls > kRescale;
                        float f = 1.f;
                        bool rescale = false;
                        if (up) {
                            const float old = negm;
                            const bool fresh = mref == -INFINITY;  // (O holds nothing yet)
                            rescale = !fresh;
                            mref = m_new;
                            negm = F8 ? -kAbove8 - m_new : fmaf(-m_new, ls, -kAbove);
                            f = fresh ? 0.f : ex2_approx(negm - old);
                            l0 *= f;
                            l1 *= f;
                        }
#pragma unroll
                        for (int c = 0; c < HK; c += PC) {
                            uint32_t pk[PC / 2];
                            if constexpr (F8) {
#pragma unroll
                                for (int b = 0; b < PC; b += kBlk) {
                                    const float4 sc = ld_shared_f32x4(sc_at + (c + b) / kBlk * 16);
                                    const float mul = logit_factor(lr, sc.x), add = sc.y + negm;
                                    float g0 = 0.f, g1 = 0.f;
#pragma unroll
                                    for (int e = b; e < b + kBlk; e += 2) {
                                        fma2(s[c + e], s[c + e + 1], mul, add);
                                        s[c + e] = ex2_approx(s[c + e]);
                                        s[c + e + 1] = ex2_approx(s[c + e + 1]);
                                        add2(g0, g1, s[c + e], s[c + e + 1]);
                                        pk[e / 2] = pack_f16x2(s[c + e], s[c + e + 1]);
                                    }
                                    l0 = fmaf(g0 + g1, sc.z, l0);
                                }
                            } else {
#pragma unroll
                                for (int e = 0; e < PC; e += 2) {
                                    fma2(s[c + e], s[c + e + 1], ls, negm);
                                    s[c + e] = ex2_approx(s[c + e]);
                                    s[c + e + 1] = ex2_approx(s[c + e + 1]);
                                    add2(l0, l1, s[c + e], s[c + e + 1]);
                                    pk[e / 2] = pack_bf16x2(s[c + e], s[c + e + 1]);
                                }
                            }
                            if constexpr (PC == 32)
                                st16(tP + c / 2, pk, 0);
                            else
                                st8(tP + c / 2, pk);
                        }
                        // O by the factor, this half of the row in flight at once
                        if (__any_sync(0xffffffffu, rescale)) {
                            uint32_t ov[HD];
#pragma unroll
                            for (int o = 0; o < HD; o += 16)
                                ld16(tO + o, ov, o);
                            ld_wait(ov);
#pragma unroll
                            for (int o = 0; o < HD; o += 16) {
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    ov[o + e] = __float_as_uint(__uint_as_float(ov[o + e]) * f);
                                st16(tO + o, ov, o);
                            }
                        }
                        st_wait();
                    }
                    fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&pready[x]);
                }
                // ----------------------------------------------------- epilogue
                if constexpr (F8) {
                    if (!single && !duo && x == 0)  // the tiles that B alone sees
                        for (int t = cnt; t < len; ++t)
                            to_fp16(t);
                    tiles += duo ? 2 * len : len;
                    // a next pair's Q if it is there, so that its S comes during the epilogue
                    // (16 prompts of 64 dims 802 -> 770 us; with a single item's, whose B
                    // A's epilogue waits for, 256 speculative chunks take 381 us, not 350)
                    const uint32_t j = (nd + 1) % kDescs;
                    ahead = warp_test(&described[j], ((nd + 1) / kDescs) & 1) &&
                            (sDesc[j].ntok > tpt || (sDesc[j].duo && sDesc[j].ntok)) &&
                            warp_test(&qfull[(qs + x) & 1], ((qs + x) >> 1) & 1);
                    if (ahead)
                        split(sDesc[j]);
                }
                const CaDesc &d = *dp;
                const int head = d.h + (duo ? x : 0);
                // (what follows from G stays out of the key loop's registers)
                int G = a.Hq / a.Hkv;
                asm volatile("" : "+r"(G));
                float l = l0 + l1;
                float m = mref == -INFINITY ? -INFINITY : -negm;  // base 2, scaled
                if (cnt > 0) {
                    if (!bad && !ca_wait(&ofull[x], no & 1))
                        bad = true;
                    ++no;
                    fence_after();
                    bad = __any_sync(0xffffffffu, bad);
                    st_shared_f32(max_at, l);  // for the other half
                    bar_sync(pair_bar, 64);
                    const float other = ld_shared_f32(max_at ^ kOther);
                    l = hf == 0 ? l + other : other + l;
                    bar_sync(pair_bar, 64);  // read before the next maximum is written
                }
                const bool whole = d.ka == 0 && d.kb == d.kt;
                // a partial result that the first walk has left already
                const bool skip = d.clean && !whole && !(sLast[4 + x] >> (d.ka == 0) & 1);
                const bool join = single && len > 1;  // B holds the odd key tiles
                if (single && x == 1) {
                    if (join) {  // A reads both halves of O: the lanes are the same
                        st_shared_f32(max_at, hf == 0 ? m : l);
                        lent = true;
                        fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(half);
                    }
                    leave();
                    continue;
                }
                float fa = 1.f, fb = 0.f;
                if (join) {
                    if (!bad && !ca_wait(half, halves & 1))
                        bad = true;
                    ++halves;
                    bad = __any_sync(0xffffffffu, bad);
                    fence_after();
                    const float mb = sMax[2 * kTile + r], lb = sMax[3 * kTile + r];
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(taken);
                    const float mm = fmaxf(m, mb);
                    fa = m == -INFINITY ? 0.f : ex2_approx(m - mm);
                    fb = mb == -INFINITY ? 0.f : ex2_approx(mb - mm);
                    m = mm;
                    l = l * fa + lb * fb;
                }
                const bool read_o = cnt > 0 && live && !bad;
                // XC columns of O, the halves joined
                auto load_o = [&](int c, uint32_t (&v)[XC]) {
                    if (read_o) {
                        ld16(tO + c, v, 0);
                        if (join) {
                            uint32_t w[XC];
                            ld16(tO + kTile + c, w, 0);
                            ld_wait(v);
                            ld_wait(w);
#pragma unroll
                            for (int e = 0; e < XC; ++e)
                                v[e] = __float_as_uint(__uint_as_float(v[e]) * fa +
                                                       __uint_as_float(w[e]) * fb);
                        } else {
                            ld_wait(v);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < XC; ++e)
                            v[e] = 0u;
                    }
                };
                auto o_done = [&] {  // this warp no longer reads O
                    if (cnt > 0) {
                        fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&oempty[x]);
                            if (join)
                                mbar_arrive(&oempty[1]);
                        }
                    }
                };
                int bs = 0;
                unsigned parts = 1;
                float *slot = nullptr;
                if (!whole) {
                    // the shares the item is cut over: lane k looks at share bs + k
                    bs = static_cast<int>(quotient(d.x, plan.share));
                    const int b = bs + lane;
                    bool some = false;
                    if (b < plan.ctas) {
                        const long long lo = share_border(plan, b), hi = share_border(plan, b + 1);
                        if (lo < d.x + d.w) {
                            const int k0 = lo > d.x ? cut_tile(lo - d.x, d.kt, single) : 0;
                            const int k1 =
                                hi < d.x + d.w ? cut_tile(hi - d.x, d.kt, single) : d.kt;
                            some = k0 < k1;
                        }
                    }
                    parts = __ballot_sync(0xffffffffu, some);
                    slot = slot_ptr<D>(a.part, 2 * blockIdx.x + (d.ka == 0));
                }
                const bool mine = r < toks * G;
                const int row = x * kTile + r;  // within a slot
                __nv_bfloat16 *dst =
                    a.out +
                    (static_cast<size_t>(d.row0 + tile_tok + r / G) * a.Hq + head * G + r % G) * D +
                    hf * HD;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                float odd = 0.f;  // becomes NaN with any element of O
#pragma unroll 1
                for (int c = 0; c < HD; c += XC) {
                    uint32_t v[XC];
                    load_o(c, v);
                    if (c + XC >= HD)
                        o_done();
#pragma unroll
                    for (int e = 0; e < XC; ++e)
                        odd += __uint_as_float(v[e]) * 0.f;
                    if (mine && !bad && !skip) {
                        if (whole) {
                            uint32_t o[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                o[k] = pack_bf16x2(__uint_as_float(v[2 * k]) * inv,
                                                   __uint_as_float(v[2 * k + 1]) * inv);
                            st_global_v8(dst + c, o);
                        } else {
                            float *to = slot + static_cast<size_t>(row) * D + hf * HD + c;
#pragma unroll
                            for (int e = 0; e < XC; e += 8) {
                                uint32_t o[8];
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    o[k] = v[e + k];
                                st_global_v8(to + e, o);
                            }
                        }
                    }
                }
                // Not finite, and keys of the share hidden from the row: once more
                bool spoiled = false;
                if (!d.clean) {
                    spoiled = __any_sync(0xffffffffu, mine && !bad && odd != odd &&
                                                          lim < min(d.len, d.kb * kTile));
                    if (spoiled && lane == 0)
                        atomicOr(&sLast[3], 1);
                } else if (!skip) {
                    // the values that counted as 0 though the row sees them: which of the half
                    // row's dims hold one above 0 (or NaN), and which one below (or NaN)
                    constexpr int OE = HD / 32;  // dims a lane
                    uint32_t pos[OE], neg[OE];
#pragma unroll
                    for (int e = 0; e < OE; ++e)
                        pos[e] = neg[e] = 0u;
                    const int from = max(d.pos0 + 1, d.ka * kTile);
                    const int to = min(d.pos0 + d.ntok, d.kb * kTile);
                    for (int b = from / kBlk; b * kBlk < to; ++b) {
                        const int blk = block_at(a, d.row, b);
                        if (blk < 0 || blk >= a.num_blocks)
                            continue;
                        const size_t at =
                            (static_cast<size_t>(blk) * a.Hkv + head) * kBlk * D + hf * HD;
                        const __nv_bfloat16 *v = a.vpool + at;
                        [[maybe_unused]] const uint8_t *v8 =
                            reinterpret_cast<const uint8_t *>(a.vpool) + at;
#pragma unroll 4
                        for (int j = 0; j < kBlk; ++j) {
                            const int key = b * kBlk + j;
                            if (key < from || key >= to)
                                continue;
#pragma unroll
                            for (int e = 0; e < OE; ++e) {
                                float y;
                                if constexpr (F8)  // NaN, or any number
                                    y = (v8[j * D + e * 32 + lane] & 0x7f) == 0x7f
                                            ? INFINITY - INFINITY
                                            : 0.f;
                                else
                                    y = __bfloat162float(v[j * D + e * 32 + lane]);
                                const uint32_t up = __ballot_sync(0xffffffffu, !(y < INFINITY));
                                const uint32_t down = __ballot_sync(0xffffffffu, !(y > -INFINITY));
                                pos[e] |= key < lim ? up : 0u;
                                neg[e] |= key < lim ? down : 0u;
                            }
                        }
                    }
                    if (mine && !bad) {
#pragma unroll
                        for (int e = 0; e < OE; ++e)
                            for (uint32_t q = pos[e] | neg[e]; q; q &= q - 1) {
                                const int c = e * 32 + __ffs(q) - 1;
                                const float y = !(neg[e] & q & -q)   ? INFINITY
                                                : !(pos[e] & q & -q) ? -INFINITY
                                                                     : INFINITY - INFINITY;
                                if (whole) {
                                    dst[c] = __float2bfloat16_rn(__bfloat162float(dst[c]) + y);
                                } else {
                                    float *to = slot + static_cast<size_t>(row) * D + hf * HD + c;
                                    *to += y;
                                }
                            }
                    }
                }
                if (whole || skip) {
                    leave();
                    continue;
                }
                // a partial result: the last of the item's shares to arrive joins them
                if (mine && hf == 0)
                    reinterpret_cast<float2 *>(slot + 2 * kTile * D)[row] = make_float2(m, l);
                __threadfence();
                if (bar_any(9 + x, 32 * kSmWarps, spoiled)) {  // not this one: the second walk's
                    if (r == 0 && hf == 0)
                        sLast[4 + x] |= 1 << (d.ka == 0);
                    leave();
                    continue;
                }
                if (r == 0 && hf == 0) {
                    const unsigned n = __popc(parts);
                    sLast[x] = atomicAdd(&a.arrived[sLast[2] + 2 * bs + x], 1) == n - 1;
                }
                bar_sync(9 + x, 32 * kSmWarps);
                if (sLast[x]) {
                    __threadfence();
                    if constexpr (D == 64) {
                        // A warp joins every eighth row, lane k weighs the k-th of them; then RW
                        // rows at once, RB times, two shares in flight (60 single tokens beside
                        // two prompt pieces 61 us, 69 with the join below).  With 128 dims the
                        // key loop loses registers to it (16 prompts 667 us with the join below,
                        // 712 with this one; 256 speculative chunks 271, 284).
                        constexpr int RW = 128 / D, RB = 4, ROWS = kTile / kSmWarps;
                        const int first = __ffs(parts) - 1, rows = toks * G;
                        const int w0 = hf * 4 + wq;
                        // this lane's row
                        const int row = min(w0 + (lane % ROWS) * kSmWarps, rows - 1);
                        auto part_at = [&](int k) {
                            return slot_ptr<D>(a.part, 2 * (bs + k) + (k == first)) +
                                   static_cast<size_t>(x * kTile) * D;
                        };
                        auto ml_at = [&](int k) {
                            const float *p = slot_ptr<D>(a.part, 2 * (bs + k) + (k == first));
                            return __ldcg(reinterpret_cast<const float2 *>(p + 2 * kTile * D) +
                                          x * kTile + row);
                        };
                        float M = -INFINITY, L = 0.f;
                        for (unsigned q = parts; q; q &= q - 1) {
                            const float2 ml = ml_at(__ffs(q) - 1);
                            const float up = fmaxf(M, ml.x);
                            if (up > -INFINITY)
                                L = L * ex2_approx(M - up) + ml.y * ex2_approx(ml.x - up);
                            M = up;
                        }
                        const float iv = L == 0.f ? 0.f : 1.f / L;
                        auto weight = [&](float m) {
                            return m == -INFINITY ? 0.f : ex2_approx(m - M) * iv;
                        };
                        const size_t to =
                            (static_cast<size_t>(d.row0 + tile_tok + row / G) * a.Hq + head * G +
                             row % G) * D;
                        const int col = lane % (D / 4) * 4, sub = lane / (D / 4);
#pragma unroll 1
                        for (int u0 = 0; u0 < ROWS; u0 += RB * RW) {
                            if (w0 + u0 * kSmWarps >= rows)
                                break;
                            float4 o[RB];
#pragma unroll
                            for (int u = 0; u < RB; ++u)
                                o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                            for (unsigned q = parts; q;) {
                                const int k0 = __ffs(q) - 1;
                                q &= q - 1;
                                const int k1 = q ? __ffs(q) - 1 : k0;
                                const bool two = q != 0;
                                q &= q - 1;
                                const float *p0 = part_at(k0) + col, *p1 = part_at(k1) + col;
                                float4 v0[RB], v1[RB];
#pragma unroll
                                for (int u = 0; u < RB; ++u) {
                                    const int at = (w0 + (u0 + u * RW + sub) * kSmWarps) * D;
                                    v0[u] = __ldcg(reinterpret_cast<const float4 *>(p0 + at));
                                    v1[u] = __ldcg(reinterpret_cast<const float4 *>(p1 + at));
                                }
                                const float f0 = weight(ml_at(k0).x);
                                const float f1 = two ? weight(ml_at(k1).x) : 0.f;
#pragma unroll
                                for (int u = 0; u < RB; ++u) {
                                    const float g0 =
                                        __shfl_sync(0xffffffffu, f0, u0 + u * RW + sub);
                                    const float g1 =
                                        __shfl_sync(0xffffffffu, f1, u0 + u * RW + sub);
                                    o[u].x += v0[u].x * g0;
                                    o[u].y += v0[u].y * g0;
                                    o[u].z += v0[u].z * g0;
                                    o[u].w += v0[u].w * g0;
                                    if (two) {  // of the only one, it would be added twice
                                        o[u].x += v1[u].x * g1;
                                        o[u].y += v1[u].y * g1;
                                        o[u].z += v1[u].z * g1;
                                        o[u].w += v1[u].w * g1;
                                    }
                                }
                            }
#pragma unroll
                            for (int u = 0; u < RB; ++u) {
                                const int k = u0 + u * RW + sub;
                                const unsigned long long t = __shfl_sync(0xffffffffu, to, k);
                                if (w0 + k * kSmWarps < rows)
                                    *reinterpret_cast<uint2 *>(a.out + t + col) =
                                        make_uint2(pack_bf16x2(o[u].x, o[u].y),
                                                   pack_bf16x2(o[u].z, o[u].w));
                            }
                        }
                    } else {
                        // RB rows a warp at a time: lane k weighs share bs + k, then every lane
                        // adds up EL columns over the shares, two of them in flight
                        constexpr int EL = 4, RB = 4;
                        const int first = __ffs(parts) - 1;
                        const bool in = parts >> lane & 1;
                        const float2 *ml_p =
                            reinterpret_cast<const float2 *>(
                                slot_ptr<D>(a.part, 2 * (bs + lane) + (lane == first)) +
                                2 * kTile * D) + x * kTile;
                        const int r_begin = (hf * 4 + wq) * RB;
                        float2 ml[RB];
                        auto load_ml = [&](int r0) {
#pragma unroll
                            for (int u = 0; u < RB; ++u)
                                ml[u] = in ? __ldcg(ml_p + r0 + u) : make_float2(-INFINITY, 0.f);
                        };
                        if (r_begin < toks * G)
                            load_ml(r_begin);
                        for (int r0 = r_begin; r0 < toks * G; r0 += kSmWarps * RB) {
                            float f[RB], o[RB][EL];
#pragma unroll
                            for (int u = 0; u < RB; ++u) {
                                float M = ml[u].x;
#pragma unroll
                                for (int w = 16; w; w >>= 1)
                                    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
                                f[u] = ml[u].x == -INFINITY ? 0.f : ex2_approx(ml[u].x - M);
                                float L = ml[u].y * f[u];
#pragma unroll
                                for (int w = 16; w; w >>= 1)
                                    L += __shfl_xor_sync(0xffffffffu, L, w);
                                f[u] *= L == 0.f ? 0.f : 1.f / L;
#pragma unroll
                                for (int e = 0; e < EL; ++e)
                                    o[u][e] = 0.f;
                            }
                            if (r0 + kSmWarps * RB < toks * G)
                                load_ml(r0 + kSmWarps * RB);
                            for (unsigned q = parts; q;) {
                                const int k0 = __ffs(q) - 1;
                                q &= q - 1;
                                const int k1 = q ? __ffs(q) - 1 : -1;
                                q &= q - 1;
                                float w[2][RB][EL];
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const int k = h ? k1 : k0;
                                    const float *o_p =
                                        slot_ptr<D>(a.part, 2 * (bs + k) + (k == first)) +
                                        static_cast<size_t>(x * kTile + r0) * D + lane * EL;
#pragma unroll
                                    for (int u = 0; u < RB; ++u) {
#pragma unroll
                                        for (int e = 0; e < EL; ++e)
                                            w[h][u][e] = 0.f;
                                        if (k < 0)
                                            continue;
                                        const float4 v =
                                            __ldcg(reinterpret_cast<const float4 *>(o_p + u * D));
                                        w[h][u][0] = v.x;
                                        w[h][u][1] = v.y;
                                        w[h][u][2] = v.z;
                                        w[h][u][3] = v.w;
                                    }
                                }
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const int k = h ? k1 : k0;
                                    if (k < 0)
                                        continue;
#pragma unroll
                                    for (int u = 0; u < RB; ++u) {
                                        const float fk = __shfl_sync(0xffffffffu, f[u], k);
#pragma unroll
                                        for (int e = 0; e < EL; ++e)
                                            o[u][e] += w[h][u][e] * fk;
                                    }
                                }
                            }
#pragma unroll
                            for (int u = 0; u < RB; ++u) {
                                const int rr = r0 + u;
                                if (rr >= toks * G)
                                    continue;
                                __nv_bfloat16 *d2 =
                                    a.out +
                                    (static_cast<size_t>(d.row0 + tile_tok + rr / G) * a.Hq +
                                     head * G + rr % G) * D + lane * EL;
#pragma unroll
                                for (int e = 0; e < EL; e += 2)
                                    *reinterpret_cast<uint32_t *>(d2 + e) =
                                        pack_bf16x2(o[u][e], o[u][e + 1]);
                            }
                        }
                    }
                }
                leave();
            }
            if (!walk_again(ended_clean()))
                break;
            leave();
        }
    }
    if (bad)
        set_error(a.sticky, ZP_ERR_TIMEOUT);
    if (wi == kMmaWarp) {  // (the walk's end: no other warp uses tensor memory any more)
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols)
                     : "memory");
    }
}

template <int D, bool F8>
static cudaError_t launch_chunk_attn_t(const ChunkAttnArgs &a, int sms, cudaStream_t s)
{
    using S = CaSmem<D, F8>;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms), 1, 1);
    cfg.blockDim = dim3(kCaThreads, 1, 1);
    cfg.dynamicSmemBytes = S::BYTES;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, zp_chunk_attn_kernel<D, F8>, a);
}

template <int D, bool F8>
static cudaError_t prepare_chunk_attn_t()
{
    return cudaFuncSetAttribute(zp_chunk_attn_kernel<D, F8>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, CaSmem<D, F8>::BYTES);
}

}  // namespace zp
