// zp_chunk_attn.cu -- attention of a ragged chunk of new tokens over the paged
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
// Twelve warps:
//   warps 0-3, 4-7  softmax of A and of B, a thread a row: the row of S from
//           tensor memory, a running maximum and sum (fp32, base 2), P
//           rounded to bf16 over S in tensor memory.  O is rescaled only when
//           a maximum grows by more than 2^8 (p stays below 2^8, which
//           changes no relative error), in place in tensor memory, between
//           the products: S's arrival says that the product before it is
//           done.  Then the epilogue.
//   warp 8  TMA producer: Q once per item, K and V through one ring of 128-key
//           stages (a box a cache block and 64 dims, 128-byte swizzle).
//   warp 9  one lane issues tcgen05.mma (kind::f16, bf16 -> fp32): S from
//           shared memory, P V with P from tensor memory and V as an
//           MN-major operand.
//   warps 10, 11  clean the V tiles that hold keys hidden from some row: a
//           probability of 0 times an infinity or NaN would be NaN.  Rows past
//           the length become 0; elements that are not finite at positions
//           past the item's first become 0, their lowest position is kept a
//           column, and the epilogue gives NaN to the rows that see it.
//
// The grid is one CTA an SM.  Every CTA adds up the cost of all items (the
// keys each reads, plus kItemCost) from the device arrays and takes an equal,
// contiguous share, cut at key tiles, so that few long rows and many short
// ones both fill the GPU.  An item cut by a border leaves partial results (m,
// l, O) in the handle's workspace, and the CTA that arrives last joins them in
// the fixed order of the shares: results do not depend on the timing.
#include <cudaTypedefs.h>

#include "zp_chunk.cuh"

namespace zp {

namespace {

constexpr int kTile = 128;             // query rows a tile, keys a tile
constexpr int kCaThreads = 384;
constexpr int kItemCost = 128;         // an item's fixed cost, in keys
constexpr int kMinShare = 2 * kTile;   // least cost given to a CTA
constexpr int kMaxSpan = 30;           // CTAs an item is cut over, about (a lane each joins them)
constexpr int kTmemCols = 512;         // S/P of A, of B; O of A, of B
constexpr float kRescale = 8.f;        // log2 of the growth that rescales O

template <int D>
struct CaSmem {
    static constexpr int PANELS = D / 64;
    static constexpr int PANEL = kTile * 128;            // bytes of 128 rows of 64 dims
    static constexpr int TILE = PANELS * PANEL;
    static constexpr int NS = D == 128 ? 5 : 10;         // K/V ring stages
    static constexpr int XC = D / 4;                     // columns a round of the halves' join
    static constexpr int off_q = 0;                      // Q of A, Q of B
    static constexpr int off_ring = off_q + 2 * TILE;
    static constexpr int off_bad = off_ring + NS * TILE;  // int [3][D]: cleared positions
    static constexpr int off_flag = off_bad + 3 * D * 4;  // int [3]; [3]: unused
    static constexpr int off_plan = off_flag + 16;        // CaPlan
    static constexpr int off_scan = off_plan + 64;        // int64 [12]
    static constexpr int off_bar = off_scan + 96;
    // full[NS], empty[NS], dirty[NS], clean[NS], Sfull[2], Pready[2], Ofull[2], Oempty[2], Qfull,
    // Qempty, done
    static constexpr int NBAR = 4 * NS + 8 + 3;
    static constexpr int off_tmem = off_bar + NBAR * 8;
    static constexpr int off_last = off_tmem + 8;         // int [2]
    static constexpr int BYTES = off_last + 8;
    static constexpr int ALLOC = BYTES + 1024;
    static_assert(ALLOC <= 232448, "shared memory of a CTA");
};

// What every CTA works out at its start.
struct CaPlan {
    long long cost;   // of all items
    long long lo, hi; // this CTA's share
    long long x0;     // cost before request i0
    int ctas;         // CTAs with a share
    int i0;           // the request `lo` falls into
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
};

__host__ __device__ __forceinline__ int tile_tokens(int G) { return kTile / G; }

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

__host__ __device__ __forceinline__ long long head_cost(const ChunkReq &c, int tpt)
{
    return pair_prefix(c, 2 * tpt, pair_count(c.n, tpt) - 1) + c.len + kItemCost;
}

// Key tile at which a border `x` of cost into an item of `kt` tiles cuts it.
__host__ __device__ __forceinline__ int cut_tile(long long x, int kt)
{
    if (x <= kItemCost)
        return 0;
    const long long k = (x - kItemCost + kTile / 2) / kTile;
    return k < kt ? static_cast<int>(k) : kt;
}

__host__ __device__ __forceinline__ long long share_border(const CaPlan &pl, int b)
{
    return pl.cost * b / pl.ctas;
}

// Walks this CTA's items; every role walks the same ones on its own.
struct CaWalk {
    const ChunkAttnArgs &a;
    const CaPlan &pl;
    int tpt;
    CaItem it;

    __host__ __device__ __forceinline__ void fill()
    {
        it.tok0 = it.p * 2 * tpt;
        it.ntok = min(it.c.n - it.tok0, 2 * tpt);
        it.single = it.ntok <= tpt;
        const int vis = it.c.len - it.c.n + it.tok0 + it.ntok;
        it.kt = (vis + kTile - 1) / kTile;
        it.w = vis + kItemCost;
        it.ka = it.x < pl.lo ? cut_tile(pl.lo - it.x, it.kt) : 0;
        it.kb = it.x + it.w > pl.hi ? cut_tile(pl.hi - it.x, it.kt) : it.kt;
    }

    __host__ __device__ __forceinline__ bool request(int i)
    {
        bool bad;
        for (; i < a.R; ++i)
            if (chunk_request(a, i, it.c, &bad))
                break;
        it.i = i;
        if (i >= a.R)
            return false;
        it.pairs = pair_count(it.c.n, tpt);
        it.span = head_cost(it.c, tpt);
        return true;
    }

    // The first item of the share; false when there is none.
    __host__ __device__ __forceinline__ bool begin()
    {
        if (pl.lo >= pl.hi || !request(pl.i0))
            return false;
        const long long off = pl.lo - pl.x0;
        it.h = static_cast<int>(off / it.span);
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
            if (++it.h == a.Hkv) {
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
__device__ __forceinline__ uint64_t ca_desc(uint32_t saddr, uint32_t lead)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3ffffu) >> 4);
    d |= static_cast<uint64_t>(lead >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// kind::f16, bf16 x bf16 -> fp32, M = 128, N = n, A K-major, B K- or MN-major.
__host__ __device__ constexpr uint32_t ca_idesc(int n, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kTile >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
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

__device__ __forceinline__ void st_wait()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void bar_sync(uint32_t id, uint32_t threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
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

// The workspace slot of a partial result: O [256][D], then (max, sum) [256].
template <int D>
__device__ __forceinline__ float *slot_ptr(float *part, int slot)
{
    return part + static_cast<size_t>(slot) * (2 * kTile * (D + 2));
}

}  // namespace

size_t chunk_attn_part_floats(int d, int sms)
{
    return static_cast<size_t>(2 * sms) * 2 * kTile * (d + 2);
}

template <int D>
__global__ void __launch_bounds__(kCaThreads, 1)
    zp_chunk_attn_kernel(const __grid_constant__ ChunkAttnArgs a)
{
    using S = CaSmem<D>;
    constexpr int PANELS = S::PANELS, NS = S::NS, XC = S::XC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *sQ = sm + S::off_q, *ring = sm + S::off_ring;
    int *sBad = reinterpret_cast<int *>(sm + S::off_bad);
    int *sFlag = reinterpret_cast<int *>(sm + S::off_flag);
    CaPlan &plan = *reinterpret_cast<CaPlan *>(sm + S::off_plan);
    long long *scan = reinterpret_cast<long long *>(sm + S::off_scan);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + S::off_bar);
    uint64_t *empty = full + NS, *dirty = empty + NS, *clean = dirty + NS;
    uint64_t *sfull = clean + NS, *pready = sfull + 2, *ofull = pready + 2, *oempty = ofull + 2;
    uint64_t *qfull = oempty + 2, *qempty = qfull + 1, *done = qempty + 1;
    uint32_t *sTmem = reinterpret_cast<uint32_t *>(sm + S::off_tmem);
    int *sLast = reinterpret_cast<int *>(sm + S::off_last);

    const int tid = threadIdx.x, lane = tid & 31, wi = tid >> 5;
    const int G = a.Hq / a.Hkv, tpt = tile_tokens(G);

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&dirty[s], 1);
            mbar_init(&clean[s], 2);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&sfull[x], 1);
            mbar_init(&pready[x], 4);
            mbar_init(&ofull[x], 1);
            mbar_init(&oempty[x], 4);
        }
        mbar_init(qfull, 1);
        // the item's last S, the join of a single item's halves, the two cleaners
        mbar_init(qempty, 4);
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (wi == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(sTmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();  // launched early: everything of the kernels before it is visible from here
    pdl_launch_dependents();

    // the shares: thread t adds up a contiguous run of requests
    {
        const int per = (a.R + kCaThreads - 1) / kCaThreads;
        const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
        long long mine = 0;
        int longest = 0;
        for (int i = r0; i < r1; ++i) {
            ChunkReq c;
            bool bad;
            if (chunk_request(a, i, c, &bad)) {
                mine += a.Hkv * head_cost(c, tpt);
                longest = max(longest, c.len);
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
        long long before = incl - mine, cost = 0;
        for (int w = 0; w < kCaThreads / 32; ++w) {
            if (w < wi)
                before += scan[w];
            cost += scan[w];
        }
        const long long wmax = sLast[0] + kItemCost;
        int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), cost / kMinShare));
        if (cost > 0)
            ctas = static_cast<int>(min(static_cast<long long>(ctas), kMaxSpan * cost / wmax));
        ctas = max(ctas, 1);
        CaPlan p;
        p.cost = cost;
        p.ctas = ctas;
        p.lo = p.hi = cost;
        p.x0 = 0;
        p.i0 = a.R;
        if (static_cast<int>(blockIdx.x) < ctas) {
            p.lo = share_border(p, blockIdx.x);
            p.hi = share_border(p, blockIdx.x + 1);
        }
        if (tid == 0 && p.lo >= p.hi)
            plan = p;
        if (p.lo < p.hi && before <= p.lo && p.lo < before + mine) {
            for (int i = r0; i < r1; ++i) {  // the request the share begins in
                ChunkReq c;
                bool bad;
                if (!chunk_request(a, i, c, &bad))
                    continue;
                const long long w = a.Hkv * head_cost(c, tpt);
                if (p.lo < before + w) {
                    p.i0 = i;
                    break;
                }
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

    if (wi >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        CaWalk wk{a, plan, tpt, {}};
        if (wi == 8) {
            // ----------------------------------------------------- producer
            uint32_t pos = 0, items = 0;
            for (bool more = wk.begin(); more && !bad; more = wk.next()) {
                const CaItem &it = wk.it;
                const int len = it.kb - it.ka, pos0 = it.c.len - it.c.n + it.tok0;
                const int32_t *trow = a.tables + (size_t)it.c.row * a.stride;
                const int nblk = (it.c.len + kBlk - 1) / kBlk;
                // pool row of a cache block of this kv head, negative past the
                // request's blocks (the load then fills zeros)
                auto block_y = [&](int q) {
                    if (q >= nblk)
                        return -kBlk;
                    const int blk = trow[q];
                    if (blk < 0 || blk >= a.num_blocks) {
                        set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
                        return -kBlk;
                    }
                    return (blk * a.Hkv + it.h) * kBlk;
                };
                // ids of four key tiles at a time, a lane a block, the next four ahead
                int ids = block_y(it.ka * 8 + lane);
                int ids_next = len > 4 ? block_y((it.ka + 4) * 8 + lane) : 0;
                if (lane == 0)
                    bad = items > 0 && !mbar_wait(qempty, (items - 1) & 1);
                bad = __shfl_sync(0xffffffffu, bad, 0);
                if (bad)
                    break;
                const int tiles = it.single ? 1 : 2;
                if (lane == 0)
                    mbar_arrive_expect_tx(qfull, tiles * PANELS * G * tpt * 128);
                __syncwarp();
                if (lane < tiles * PANELS) {
                    const int x = lane / PANELS, p = lane % PANELS;
                    asm volatile(
                        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx"
                        "::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                            smem_u32(sQ + x * S::TILE + p * S::PANEL)),
                        "l"(&a.qmap), "r"(p * 64), "r"(it.h * G), "r"(it.c.first + it.tok0 + x * tpt),
                        "r"(smem_u32(qfull))
                        : "memory");
                }
                ++items;
                int base = 0;  // key tile `ids` begins at
                auto stage = [&](int t, bool v) {
                    const int s = pos % NS;
                    if (lane == 0) {
                        bad = pos >= NS && !mbar_wait(&empty[s], (pos / NS - 1) & 1);
                        if (!bad) {
                            mbar_arrive_expect_tx(&full[s], S::TILE);
                            // a V tile to be cleaned: the cleaners may not look at the
                            // stage's `full` before it stands at this load
                            if (v && (it.ka + t + 1) * kTile > pos0 + 1)
                                mbar_arrive(&dirty[s]);
                        }
                    }
                    bad = __shfl_sync(0xffffffffu, bad, 0);
                    if (bad)
                        return;
                    // a V tile may lie one group behind the K tile loaded before it
                    const int q = lane / PANELS, p = lane % PANELS;
                    const int src = (t - base) * 8 + (q & 7);
                    const int y0 = __shfl_sync(0xffffffffu, ids, src & 31);
                    const int y1 = __shfl_sync(0xffffffffu, ids_next, src & 31);
                    if (lane < 8 * PANELS)
                        tma_load_2d(ring + s * S::TILE + p * S::PANEL + q * kBlk * 128,
                                    v ? a.vmap : a.kmap, p * 64, src < 32 ? y0 : y1, &full[s]);
                    ++pos;
                };
                auto advance = [&](int t) {  // V tile t is the oldest still to come
                    if (t - base >= 4) {
                        base += 4;
                        ids = ids_next;
                        ids_next = base + 4 < len ? block_y((it.ka + base + 4) * 8 + lane) : 0;
                    }
                };
                if (it.single) {
                    stage(0, false);
                    for (int t = 0; t < len && !bad; ++t) {
                        advance(t);
                        if (t + 1 < len)
                            stage(t + 1, false);
                        if (!bad)
                            stage(t, true);
                    }
                } else {
                    for (int t = 0; t < len && !bad; ++t) {
                        advance(t);
                        stage(t, false);
                        if (!bad)
                            stage(t, true);
                    }
                }
            }
            // every copy issued has landed before the CTA may exit
            if (lane == 0) {
                bool ok = items == 0 || mbar_wait(qfull, (items - 1) & 1);
                for (uint32_t j = pos > NS ? pos - NS : 0; j < pos; ++j)
                    ok &= mbar_wait(&full[j % NS], (j / NS) & 1);
                bad |= !ok;
            }
        } else if (wi == 9) {
            // ----------------------------------------------------- products
            constexpr uint32_t ID_S = ca_idesc(kTile, false), ID_O = ca_idesc(D, true);
            uint32_t base = 0, items = 0, cleaned = 0;  // cleaned: a parity bit a stage
            uint32_t np[2] = {0u, 0u}, no[2] = {0u, 0u};
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (!bad && !mbar_wait(bar, parity))
                    bad = true;
            };
            for (bool more = wk.begin(); more && !bad; more = wk.next()) {
                const CaItem &it = wk.it;
                const int len = it.kb - it.ka, pos0 = it.c.len - it.c.n + it.tok0;
                if (lane == 0) {
                    const bool single = it.single;
                    // A's key tiles of a pair: the ones its last token sees
                    const int na = (pos0 + min(it.ntok, tpt) + kTile - 1) / kTile;
                    const int cnt[2] = {single ? (len + 1) / 2 : max(0, min(it.kb, na) - it.ka),
                                        single ? len / 2 : len};
                    auto kpos = [&](int t) {
                        return base + (single ? (t ? 2 * t - 1 : 0) : 2 * t);
                    };
                    auto vpos = [&](int t) {
                        return base + (single && t + 1 < len ? 2 * t + 2 : 2 * t + 1);
                    };
                    auto need = [&](uint32_t pos) { wait(&full[pos % NS], (pos / NS) & 1); };
                    auto product_s = [&](int x, int t) {
                        const uint32_t kb = smem_u32(ring + (kpos(t) % NS) * S::TILE);
                        const uint32_t qb = smem_u32(sQ + (single ? 0 : x) * S::TILE);
                        fence_after();
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            const uint32_t o = (ks >> 2) * S::PANEL + (ks & 3) * 32;
                            mma_ss(tmem + x * kTile, ca_desc(qb + o, 16), ca_desc(kb + o, 16), ID_S,
                                   ks > 0);
                        }
                        mma_commit(&sfull[x]);
                    };
                    auto product_o = [&](int x, int t, bool first, bool last) {
                        wait(&pready[x], np[x]++ & 1);
                        if (first) {
                            if (no[x] > 0)
                                wait(&oempty[x], (no[x] - 1) & 1);
                            ++no[x];
                        }
                        if (bad)
                            return;
                        fence_after();
                        const uint32_t vb = smem_u32(ring + (vpos(t) % NS) * S::TILE);
#pragma unroll
                        for (int ks = 0; ks < kTile / 16; ++ks)
                            mma_ts(tmem + 256 + x * kTile, tmem + x * kTile + ks * 8,
                                   ca_desc(vb + ks * 2048, S::PANEL), ID_O, !first || ks > 0);
                        if (last)
                            mma_commit(&ofull[x]);
                    };
                    auto need_v = [&](int t) {
                        const uint32_t pos = vpos(t);
                        need(pos);
                        if ((it.ka + t + 1) * kTile > pos0 + 1) {
                            wait(&clean[pos % NS], (cleaned >> (pos % NS)) & 1);
                            cleaned ^= 1u << (pos % NS);
                        }
                    };
                    auto release = [&](uint32_t pos) { mma_commit(&empty[pos % NS]); };
                    wait(qfull, items & 1);
                    need(kpos(0));
                    if (!bad && cnt[0] > 0)
                        product_s(0, 0);
                    if (single) {
                        release(kpos(0));
                        if (len > 1) {
                            need(kpos(1));
                            if (!bad) {
                                product_s(1, 1);
                                release(kpos(1));
                            }
                        }
                        for (int t = 0; t < len && !bad; ++t) {
                            const int x = t & 1;
                            need_v(t);
                            product_o(x, t, t < 2, t + 2 >= len);
                            if (bad)
                                break;
                            release(vpos(t));
                            if (t + 2 < len) {
                                need(kpos(t + 2));
                                if (bad)
                                    break;
                                product_s(x, t + 2);
                                release(kpos(t + 2));
                            }
                        }
                    } else {
                        if (!bad) {
                            product_s(1, 0);
                            release(kpos(0));
                        }
                        for (int t = 0; t < len && !bad; ++t) {
                            need_v(t);
                            if (t + 1 < len)
                                need(kpos(t + 1));
                            if (bad)
                                break;
                            if (t < cnt[0]) {
                                product_o(0, t, t == 0, t + 1 == cnt[0]);
                                if (bad)
                                    break;
                                if (t + 1 < cnt[0])
                                    product_s(0, t + 1);
                            }
                            product_o(1, t, t == 0, t + 1 == len);
                            if (bad)
                                break;
                            release(vpos(t));
                            if (t + 1 < len) {
                                product_s(1, t + 1);
                                release(kpos(t + 1));
                            }
                        }
                    }
                    mma_commit(qempty);
                }
                bad = __shfl_sync(0xffffffffu, bad, 0);
                base += 2 * len;
                ++items;
            }
            if (lane == 0) {  // every product issued is done before the tensor memory is freed
                mma_commit(done);
                bad |= !mbar_wait(done, 0);
            }
            __syncwarp();
        } else {
            // ----------------------------------------------- cleaning of V
            const int w2 = wi - 10;
            uint32_t base = 0, items = 0, dirtied = 0;  // dirtied: a parity bit a stage
            // (a warp that gave up still passes the barrier of every item)
            for (bool more = wk.begin(); more; more = wk.next()) {
                const CaItem &it = wk.it;
                const int len = it.kb - it.ka, pos0 = it.c.len - it.c.n + it.tok0;
                const int buf = items % 3;
                // Q of this item arrived: the S products of the item before are
                // done, so only the epilogues of the two items before still read
                // their buffers
                if (!bad && !mbar_wait(qfull, items & 1))
                    bad = true;
                bad = __any_sync(0xffffffffu, bad);
                if (lane == 0)
                    mbar_arrive(qempty);
                for (int c = w2 * 32 + lane; c < D; c += 64)
                    sBad[buf * D + c] = 0x7fffffff;
                if (w2 == 0 && lane == 0)
                    sFlag[buf] = 0;
                bar_sync(3, 64);
                int t = max(0, (pos0 + 1) / kTile - it.ka);
                for (; t < len && !bad; ++t) {
                    const int k0 = (it.ka + t) * kTile;
                    if (k0 + kTile <= pos0 + 1)
                        continue;
                    const uint32_t pos =
                        base + (it.single && t + 1 < len ? 2 * t + 2 : 2 * t + 1);
                    const int s = pos % NS;
                    if (!mbar_wait(&dirty[s], dirtied >> s & 1) ||
                        !mbar_wait(&full[s], (pos / NS) & 1))
                        bad = true;
                    dirtied ^= 1u << s;
                    bad = __any_sync(0xffffffffu, bad);
                    if (bad)
                        break;
                    constexpr int CPR = D / 8, RPW = 32 / CPR;  // chunks a row, rows a warp
                    const int ch = lane % CPR;
                    for (int r = max(0, pos0 + 1 - k0) + w2 * RPW + lane / CPR; r < kTile;
                         r += 2 * RPW) {
                        const uint32_t at =
                            smem_u32(ring + s * S::TILE) + swz(r, ch, kTile);
                        if (k0 + r >= it.c.len) {
                            st_shared_v4(at, make_uint4(0u, 0u, 0u, 0u));
                            continue;
                        }
                        uint4 v = ld_shared_v4(at);
                        uint32_t *e = reinterpret_cast<uint32_t *>(&v);
                        uint32_t hit = 0;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            if ((e[x] & 0x7f80u) == 0x7f80u) {
                                hit |= 1u << (2 * x);
                                e[x] &= 0xffff0000u;
                            }
                            if ((e[x] & 0x7f800000u) == 0x7f800000u) {
                                hit |= 2u << (2 * x);
                                e[x] &= 0xffffu;
                            }
                        }
                        if (hit) {
                            st_shared_v4(at, v);
                            for (int x = 0; x < 8; ++x)
                                if (hit >> x & 1)
                                    atomicMin(&sBad[buf * D + ch * 8 + x], k0 + r);
                            sFlag[buf] = 1;
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&clean[s]);
                }
                base += 2 * len;
                ++items;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ------------------------------------------------------- softmax
        const int x = wi >> 2;                 // tile A or B
        const int wq = wi & 3;                 // tensor-memory lanes 32 wq ..
        const int r = wq * 32 + lane;          // row of the tile
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tS = tmem + x * kTile + lane_off, tO = tmem + 256 + x * kTile + lane_off;
        const bool neg = a.logit_scale < 0.f;
        const float ls = fmaxf(fabsf(a.logit_scale), 1e-30f);
        const float grow = kRescale / ls;
        const int rtok = r / G, rg = r - rtok * G;
        uint32_t ns = 0, no = 0, items = 0;
        CaWalk wk{a, plan, tpt, {}};
        for (bool more = wk.begin(); more; more = wk.next()) {
            const CaItem &it = wk.it;
            const int len = it.kb - it.ka, pos0 = it.c.len - it.c.n + it.tok0;
            const bool single = it.single;
            const int tile_tok = single || x == 0 ? 0 : tpt;       // its first token in the item
            const int toks = min(it.ntok - tile_tok, tpt);         // its tokens
            const int rows = toks * G;
            const int tok = min(rtok, toks - 1);                   // rows past the last follow it
            const int lim = pos0 + tile_tok + tok + 1;             // keys the row sees
            const int wlim = __shfl_sync(0xffffffffu, lim, 0);     // ... the warp's first row
            const bool live = wq * 32 < rows;
            const int na = (pos0 + min(it.ntok, tpt) + kTile - 1) / kTile;
            const int cnt = single ? (x == 0 ? (len + 1) / 2 : len / 2)
                                   : (x == 0 ? max(0, min(it.kb, na) - it.ka) : len);
            if (!single && tid == 0)
                mbar_arrive(qempty);  // nothing but S reads Q
            float mref = -INFINITY, negm = 0.f;
            float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
            for (int t = 0; t < cnt; ++t) {
                const int k0 = (it.ka + (single ? 2 * t + x : t)) * kTile;
                if (!bad && !mbar_wait(&sfull[x], ns & 1))
                    bad = true;
                ++ns;
                bad = __any_sync(0xffffffffu, bad);
                if (bad)
                    break;
                fence_after();
                if (live) {
                    uint32_t sr[kTile];
#pragma unroll
                    for (int o = 0; o < kTile; o += 16)
                        ld16(tS + o, sr, o);
                    ld_wait(sr);
                    float *s = reinterpret_cast<float *>(sr);
                    if (neg) {
#pragma unroll
                        for (int c = 0; c < kTile; ++c)
                            s[c] = -s[c];
                    }
                    if (k0 + kTile > wlim) {
                        const int m = lim - k0;
#pragma unroll
                        for (int c = 0; c < kTile; ++c)
                            s[c] = c < m ? s[c] : -INFINITY;
                    }
                    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int c = 4; c < kTile; c += 8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            mx[e] = c + 4 + e < kTile ? fmaxf(fmaxf(mx[e], s[c + e]), s[c + 4 + e])
                                                      : fmaxf(mx[e], s[c + e]);
                    }
                    const float m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const bool up = t == 0 ? m_new > -INFINITY : m_new > mref + grow;
                    if (__any_sync(0xffffffffu, up)) {
                        const float old = negm;
                        const bool fresh = mref == -INFINITY;
                        if (up) {
                            mref = m_new;
                            negm = -m_new * ls;
                        }
                        if (t > 0) {
                            const float f = !up ? 1.f : fresh ? 0.f : ex2_approx(negm - old);
                            l0 *= f;
                            l1 *= f;
                            l2 *= f;
                            l3 *= f;
#pragma unroll 1
                            for (int o = 0; o < D; o += 16) {
                                uint32_t ov[16];
                                ld16(tO + o, ov, 0);
                                ld_wait(ov);
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
                                st16(tO + o, ov, 0);
                            }
                        }
                    }
#pragma unroll
                    for (int c = 0; c < kTile; c += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            fma2(s[c + e], s[c + e + 1], ls, negm);
                            fma2(s[c + e + 2], s[c + e + 3], ls, negm);
                            s[c + e] = ex2_approx(s[c + e]);
                            s[c + e + 1] = ex2_approx(s[c + e + 1]);
                            s[c + e + 2] = ex2_approx(s[c + e + 2]);
                            s[c + e + 3] = ex2_approx(s[c + e + 3]);
                            add2(l0, l1, s[c + e], s[c + e + 1]);
                            add2(l2, l3, s[c + e + 2], s[c + e + 3]);
                            pk[e / 2] = pack_bf16x2(s[c + e], s[c + e + 1]);
                            pk[e / 2 + 1] = pack_bf16x2(s[c + e + 2], s[c + e + 3]);
                        }
                        st16(tS + c / 2, pk, 0);
                    }
                    st_wait();
                }
                fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&pready[x]);
            }
            // ----------------------------------------------------- epilogue
            float l = (l0 + l1) + (l2 + l3);
            float m = mref == -INFINITY ? -INFINITY : -negm;  // base 2, scaled
            if (cnt > 0) {
                if (!bad && !mbar_wait(&ofull[x], no & 1))
                    bad = true;
                ++no;
                fence_after();
            }
            bad = __any_sync(0xffffffffu, bad);
            const int buf = items % 3;
            ++items;
            // only the tiles that were cleaned order the flag before this read
            const int last_tile = it.ka + (single ? 2 * (cnt - 1) + x : cnt - 1);
            const bool poisoned =
                !bad && cnt > 0 && (last_tile + 1) * kTile > pos0 + 1 && sFlag[buf] != 0;
            const bool whole = it.ka == 0 && it.kb == it.kt;
            const bool join = single && len > 1;  // B holds the odd key tiles
            // exchange area of the halves: Q of B (a single item has one tile)
            float4 *xo = reinterpret_cast<float4 *>(sQ + S::TILE);
            float2 *xm = reinterpret_cast<float2 *>(sQ + S::TILE + S::TILE / 2);
            auto load_o = [&](int c, uint32_t (&v)[XC]) {  // XC columns of O, poisoned ones NaN
                if (cnt > 0 && live && !bad) {
#pragma unroll
                    for (int o = 0; o < XC; o += 16)
                        ld16(tO + c + o, v, o);
                    ld_wait(v);
                    if (poisoned) {
#pragma unroll
                        for (int e = 0; e < XC; ++e)
                            if (sBad[buf * D + c + e] < lim)
                                v[e] = 0x7fffffffu;
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
                    if (lane == 0)
                        mbar_arrive(&oempty[x]);
                }
            };
            if (single && x == 1) {
                if (join) {
                    xm[r] = make_float2(m, l);
                    for (int c = 0; c < D; c += XC) {
                        uint32_t v[XC];
                        load_o(c, v);
#pragma unroll
                        for (int e = 0; e < XC; e += 4)
                            xo[(e / 4) * kTile + r] =
                                make_float4(__uint_as_float(v[e]), __uint_as_float(v[e + 1]),
                                            __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
                        if (c + XC >= D)
                            o_done();
                        fence_proxy_async_smem();  // Q is loaded over it next
                        bar_sync(4, 256);          // this round is written
                        bar_sync(5, 256);          // and read
                    }
                }
                continue;
            }
            float fa = 1.f, fb = 0.f;
            int bs = 0;
            unsigned parts = 1;
            float *slot = nullptr;
            if (!whole) {
                // the shares the item is cut over: lane k looks at share bs + k
                bs = static_cast<int>(min(static_cast<long long>(plan.ctas - 1),
                                          it.x * plan.ctas / plan.cost));
                while (bs + 1 < plan.ctas && share_border(plan, bs + 1) <= it.x)
                    ++bs;
                while (share_border(plan, bs) > it.x)
                    --bs;
                const int b = bs + lane;
                bool some = false;
                if (b < plan.ctas) {
                    const long long lo = share_border(plan, b), hi = share_border(plan, b + 1);
                    if (lo < it.x + it.w) {
                        const int k0 = lo > it.x ? cut_tile(lo - it.x, it.kt) : 0;
                        const int k1 = hi < it.x + it.w ? cut_tile(hi - it.x, it.kt) : it.kt;
                        some = k0 < k1;
                    }
                }
                parts = __ballot_sync(0xffffffffu, some);
                slot = slot_ptr<D>(a.part, 2 * blockIdx.x + (it.ka == 0));
            }
            const int row = x * kTile + r;  // within a slot
            const size_t tok_row = static_cast<size_t>(it.c.first + it.tok0 + tile_tok + rtok);
            __nv_bfloat16 *dst = a.out + (tok_row * a.Hq + it.h * G + rg) * D;
            float inv = 1.f;
#pragma unroll 1
            for (int c = 0; c < D; c += XC) {
                uint32_t v[XC];
                load_o(c, v);
                if (c + XC >= D)
                    o_done();
                if (join) {
                    bar_sync(4, 256);
                    if (c == 0) {
                        const float2 mb = xm[r];
                        const float mm = fmaxf(m, mb.x);
                        fa = m == -INFINITY ? 0.f : ex2_approx(m - mm);
                        fb = mb.x == -INFINITY ? 0.f : ex2_approx(mb.x - mm);
                        m = mm;
                        l = l * fa + mb.y * fb;
                    }
#pragma unroll
                    for (int e = 0; e < XC; e += 4) {
                        const float4 w = xo[(e / 4) * kTile + r];
                        v[e] = __float_as_uint(__uint_as_float(v[e]) * fa + w.x * fb);
                        v[e + 1] = __float_as_uint(__uint_as_float(v[e + 1]) * fa + w.y * fb);
                        v[e + 2] = __float_as_uint(__uint_as_float(v[e + 2]) * fa + w.z * fb);
                        v[e + 3] = __float_as_uint(__uint_as_float(v[e + 3]) * fa + w.w * fb);
                    }
                    fence_proxy_async_smem();
                    bar_sync(5, 256);
                }
                if (c == 0)
                    inv = l == 0.f ? 0.f : 1.f / l;
                if (r < rows && !bad) {
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < XC; e += 8) {
                            uint4 o;
                            o.x = pack_bf16x2(__uint_as_float(v[e]) * inv,
                                              __uint_as_float(v[e + 1]) * inv);
                            o.y = pack_bf16x2(__uint_as_float(v[e + 2]) * inv,
                                              __uint_as_float(v[e + 3]) * inv);
                            o.z = pack_bf16x2(__uint_as_float(v[e + 4]) * inv,
                                              __uint_as_float(v[e + 5]) * inv);
                            o.w = pack_bf16x2(__uint_as_float(v[e + 6]) * inv,
                                              __uint_as_float(v[e + 7]) * inv);
                            st_global_v4(dst + c + e, o);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < XC; e += 4)
                            st_global_v4(slot + static_cast<size_t>(row) * D + c + e,
                                         make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]));
                    }
                }
            }
            if (single && tid == 0)
                mbar_arrive(qempty);  // the halves are joined: Q may be loaded over
            if (whole)
                continue;
            // a partial result: the last of the item's shares to arrive joins them
            if (r < rows)
                reinterpret_cast<float2 *>(slot + 2 * kTile * D)[row] = make_float2(m, l);
            __threadfence();
            bar_sync(1 + x, 128);
            if (r == 0) {
                const unsigned n = __popc(parts);
                sLast[x] = atomicInc(&a.arrived[2 * bs + x], n - 1) == n - 1;
            }
            bar_sync(1 + x, 128);
            if (!sLast[x])
                continue;
            __threadfence();
            constexpr int LPR = D / 4, RPW = 32 / LPR;  // lanes a row, rows a warp
            const int first = __ffs(parts) - 1;
            for (int rr = wq * RPW + lane / LPR; rr < rows; rr += 4 * RPW) {
                const int cc = (lane % LPR) * 4;
                const int srow = x * kTile + rr;
                float M = -INFINITY;
                for (unsigned q = parts; q; q &= q - 1) {
                    const int k = __ffs(q) - 1;
                    const float *sp = slot_ptr<D>(a.part, 2 * (bs + k) + (k == first));
                    M = fmaxf(M, __ldcg(reinterpret_cast<const float2 *>(sp + 2 * kTile * D) + srow).x);
                }
                float L = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                for (unsigned q = parts; q; q &= q - 1) {
                    const int k = __ffs(q) - 1;
                    const float *sp = slot_ptr<D>(a.part, 2 * (bs + k) + (k == first));
                    const float2 ml =
                        __ldcg(reinterpret_cast<const float2 *>(sp + 2 * kTile * D) + srow);
                    const float4 w = __ldcg(reinterpret_cast<const float4 *>(
                        sp + static_cast<size_t>(srow) * D + cc));
                    const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
                    L += ml.y * f;
                    o.x += w.x * f;
                    o.y += w.y * f;
                    o.z += w.z * f;
                    o.w += w.w * f;
                }
                const float iv = L == 0.f ? 0.f : 1.f / L;
                const int tk = rr / G;
                __nv_bfloat16 *d2 =
                    a.out + (static_cast<size_t>(it.c.first + it.tok0 + tile_tok + tk) * a.Hq +
                             it.h * G + rr - tk * G) * D + cc;
                *reinterpret_cast<uint2 *>(d2) =
                    make_uint2(pack_bf16x2(o.x * iv, o.y * iv), pack_bf16x2(o.z * iv, o.w * iv));
            }
        }
    }
    if (bad)
        set_error(a.sticky, ZP_ERR_TIMEOUT);
    fence_before();
    __syncthreads();
    if (wi == 9) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols)
                     : "memory");
    }
}

template <int D>
static cudaError_t launch_chunk_attn_t(const ChunkAttnArgs &a, int sms, cudaStream_t s)
{
    using S = CaSmem<D>;
    const cudaError_t e = cudaFuncSetAttribute(
        zp_chunk_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::ALLOC);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms), 1, 1);
    cfg.blockDim = dim3(kCaThreads, 1, 1);
    cfg.dynamicSmemBytes = S::ALLOC;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, zp_chunk_attn_kernel<D>, a);
}

cudaError_t launch_chunk_attn(const ChunkAttnArgs &a, int d, int sms, cudaStream_t s)
{
    if (d == 64)
        return launch_chunk_attn_t<64>(a, sms, s);
    if (d == 128)
        return launch_chunk_attn_t<128>(a, sms, s);
    return cudaErrorInvalidValue;
}

}  // namespace zp
