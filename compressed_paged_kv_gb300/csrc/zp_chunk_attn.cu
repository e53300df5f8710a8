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
constexpr int kSmWarps = 8;            // softmax warps a query tile
constexpr int kCaThreads = (2 * kSmWarps + 4) * 32;
constexpr int kSmRegs = 104, kOtherRegs = 64;  // registers a thread after the split
static_assert(kSmRegs * 2 * kSmWarps + kOtherRegs * 4 <= 96 * (2 * kSmWarps + 4),
              "the split draws on the registers of the launch");
constexpr int kItemCost = 128;         // an item's fixed cost, in keys
constexpr int kMinShare = 2 * kTile;   // least cost given to a CTA
constexpr int kMaxSpan = 30;           // CTAs an item is cut over, about (a lane each joins them)
constexpr int kLoadWarp = 2 * kSmWarps;       // then the products' warps of A and of B, the cleaner
constexpr int kMmaWarp = kLoadWarp + 1;
constexpr int kBufs = 8;               // records of cleared elements (an item each, in turn)
constexpr int kTmemCols = 512;         // S/P of A, of B; O of A, of B
constexpr float kRescale = 8.f;        // log2 of the growth that rescales O

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

template <int D>
struct CaSmem {
    static constexpr int PANELS = D / 64;
    static constexpr int PANEL = kTile * 128;            // bytes of 128 rows of 64 dims
    static constexpr int TILE = PANELS * PANEL;
    static constexpr int NS = D == 128 ? 5 : 10;         // K/V ring stages
    static constexpr int XC = D / 4;                     // columns of O a step of the epilogue
    static constexpr int off_q = 0;                      // Q of A, Q of B
    static constexpr int off_ring = off_q + 2 * TILE;
    static constexpr int off_max = off_ring + NS * TILE;  // float [2][2][128]: maxima of row halves
    static constexpr int off_flag = off_max + 4 * kTile * 4;  // int [kBufs]: elements were cleared
    static constexpr int off_plan = off_flag + kBufs * 4;     // CaPlan
    static constexpr int off_scan = off_plan + 80;        // int64 [warps]
    static constexpr int off_bar = off_scan + kCaThreads / 32 * 8;
    // full[NS], empty[NS], clean[NS], Sfull[2], Pready[2], Ofull[2], Oempty[2], Qfull[2], Qempty[2],
    // dirty[2], turn[2], half, taken, done
    static constexpr int NBAR = 3 * NS + 16 + 3;
    static constexpr int off_tmem = off_bar + NBAR * 8;
    static constexpr int off_last = off_tmem + 8;         // int [2]
    static constexpr int BYTES = off_last + 8;
    static_assert(sizeof(CaPlan) <= 80 && off_bar % 8 == 0, "layout");
    static_assert(BYTES <= 232448, "shared memory of a CTA");
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
__host__ __device__ __forceinline__ void make_shares(CaPlan &pl, long long cost, int longest, int grid)
{
    const float span = kMaxSpan * (static_cast<float>(cost) / (longest + kItemCost));
    const long long most = cost / kMinShare;
    int ctas = most < grid ? static_cast<int>(most) : grid;
    if (span < ctas)
        ctas = static_cast<int>(span);
    pl.cost = cost;
    pl.ctas = ctas < 1 ? 1 : ctas;
    pl.share = quotient(cost + pl.ctas - 1, pl.ctas);
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

    __host__ __device__ __forceinline__ void entered(int i)
    {
        it.i = i;
        it.pairs = pair_count(it.c.n, tpt);
        it.span = head_cost(it.c, tpt);
    }

    __host__ __device__ __forceinline__ bool request(int i)
    {
        bool bad;
        for (; i < a.R; ++i)
            if (chunk_request(a, i, it.c, &bad))
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

// Bounded waits: a try suspends the warp for some microseconds, so that this is
// a matter of seconds, and every wait here is for this CTA's own work.
constexpr uint32_t kCaSpins = 1u << 19;

__device__ __forceinline__ bool ca_wait(uint64_t *bar, uint32_t parity)
{
    return mbar_wait(bar, parity, kCaSpins);
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

// The positions of cleared value elements of a CTA's items, behind the slots
// of the partial results: int [kBufs][D], written only when there are some.
template <int D>
__device__ __forceinline__ int *cleared_ptr(float *part)
{
    return reinterpret_cast<int *>(part + static_cast<size_t>(2 * gridDim.x) * (2 * kTile * (D + 2))) +
           static_cast<size_t>(blockIdx.x) * kBufs * D;
}

__device__ __forceinline__ void st_global_v8(void *p, const uint32_t (&v)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
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
    return static_cast<size_t>(sms) * (4 * kTile * (d + 2) + kBufs * d);
}

template <int D>
__global__ void __launch_bounds__(kCaThreads, 1)
    zp_chunk_attn_kernel(const __grid_constant__ ChunkAttnArgs a)
{
    using S = CaSmem<D>;
    constexpr int PANELS = S::PANELS, NS = S::NS, XC = S::XC;
    extern __shared__ __align__(1024) uint8_t smem_aligned[];
    uint8_t *sm = smem_aligned;
    if (smem_u32(sm) & 1023u) {  // the swizzled tiles need it
        if (threadIdx.x == 0)
            set_error(a.sticky, ZP_ERR_UNSUPPORTED);
        return;
    }
    uint8_t *sQ = sm + S::off_q, *ring = sm + S::off_ring;
    float *sMax = reinterpret_cast<float *>(sm + S::off_max);
    int *sFlag = reinterpret_cast<int *>(sm + S::off_flag);
    CaPlan &plan = *reinterpret_cast<CaPlan *>(sm + S::off_plan);
    long long *scan = reinterpret_cast<long long *>(sm + S::off_scan);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + S::off_bar);
    uint64_t *empty = full + NS, *clean = empty + NS, *sfull = clean + NS, *pready = sfull + 2;
    uint64_t *ofull = pready + 2, *oempty = ofull + 2, *qfull = oempty + 2, *qempty = qfull + 2;
    uint64_t *dirty = qempty + 2, *turn = dirty + 2, *half = turn + 2, *taken = half + 1, *done = taken + 1;
    uint32_t *sTmem = reinterpret_cast<uint32_t *>(sm + S::off_tmem);
    int *sLast = reinterpret_cast<int *>(sm + S::off_last);

    const int tid = threadIdx.x, lane = tid & 31, wi = tid >> 5;
    const int G = a.Hq / a.Hkv, tpt = tile_tokens(G);

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 2);  // both products' warps have passed it
            mbar_init(&clean[s], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&sfull[x], 1);
            mbar_init(&pready[x], kSmWarps);
            mbar_init(&ofull[x], 1);
            mbar_init(&oempty[x], kSmWarps);
            mbar_init(&qfull[x], 1);
            mbar_init(&qempty[x], 2);
            mbar_init(&dirty[x], 1);
            mbar_init(&turn[x], 1);
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
        CaPlan p;
        make_shares(p, cost, sLast[0], static_cast<int>(gridDim.x));
        p.lo = share_border(p, blockIdx.x);
        p.hi = share_border(p, blockIdx.x + 1);
        if (tid == 0 && p.lo >= p.hi)
            plan = p;
        if (before <= p.lo && p.lo < before + mine) {
            for (int i = r0; i < r1; ++i) {  // the request the share begins in
                bool bad;
                if (!chunk_request(a, i, p.c0, &bad))
                    continue;
                p.i0 = i;
                const long long w = a.Hkv * head_cost(p.c0, tpt);
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

    if (wi >= 2 * kSmWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        CaWalk wk{a, plan, tpt, {}};
        if (wi == kLoadWarp) {
            // ----------------------------------------------------- producer
            uint32_t loaded = 0, cur = 0, par = 0, qs = 0;  // ring cursor and parity, query tiles
            for (bool more = wk.begin(); more && !bad; more = wk.next()) {
                const CaItem &it = wk.it;
                const int len = it.kb - it.ka;
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
                int base = 0;  // key tile `ids` begins at
                auto stage = [&](int t, bool v) {
                    if (loaded >= NS && !warp_wait(&empty[cur], par ^ 1)) {
                        bad = true;
                        return;
                    }
                    // a V tile may lie one group behind the K tile loaded before it
                    const int src = (t - base) * 8;
                    const int from = src < 32 ? ids : ids_next;
                    int y[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        y[q] = __shfl_sync(0xffffffffu, from, (src & 31) + q);
                    const CUtensorMap *map = v ? a.vmap : a.kmap;
                    uint8_t *dst = ring + cur * S::TILE;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&full[cur], S::TILE);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
#pragma unroll
                            for (int p = 0; p < PANELS; ++p)
                                tma_load_2d(dst + p * S::PANEL + q * kBlk * 128, map, p * 64, y[q],
                                            &full[cur]);
                    }
                    __syncwarp();
                    ++loaded;
                    if (++cur == NS) {
                        cur = 0;
                        par ^= 1;
                    }
                };
                auto advance = [&](int t) {  // V tile t is the oldest still to come
                    if (t - base >= 4) {
                        base += 4;
                        ids = ids_next;
                        ids_next = base + 4 < len ? block_y((it.ka + base + 4) * 8 + lane) : 0;
                    }
                };
                // the first K tile before Q: it does not wait for the item before
                stage(0, false);
                if (bad)
                    break;
                for (int x = 0; x < (it.single ? 1 : 2); ++x, ++qs) {
                    const int j = qs & 1;
                    if (qs >= 2 && !warp_wait(&qempty[j], ((qs >> 1) - 1) & 1)) {
                        bad = true;
                        break;
                    }
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&qfull[j], PANELS * G * tpt * 128);
#pragma unroll
                        for (int p = 0; p < PANELS; ++p)
                            asm volatile(
                                "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier"
                                "::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                                    smem_u32(sQ + j * S::TILE + p * S::PANEL)),
                                "l"(&a.qmap), "r"(p * 64), "r"(it.h * G),
                                "r"(it.c.first + it.tok0 + x * tpt), "r"(smem_u32(&qfull[j]))
                                : "memory");
                    }
                    __syncwarp();
                }
                if (it.single) {
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
                        if (t > 0)
                            stage(t, false);
                        if (!bad)
                            stage(t, true);
                    }
                }
            }
            // every copy issued has landed before the CTA may exit
            for (uint32_t j = qs > 2 ? qs - 2 : 0; j < qs; ++j)
                bad |= !warp_wait(&qfull[j & 1], (j >> 1) & 1);
            for (uint32_t j = loaded > NS ? loaded - NS : 0; j < loaded; ++j)
                bad |= !warp_wait(&full[j % NS], (j / NS) & 1);
        } else if (wi <= kMmaWarp + 1) {
            // ----------------------------------------------------- products
            // One warp a stream, so that the waits of one lie beside the products of
            // the other (the issue of a product waits for a place in a short queue).
            // They take turns at P V and the next S: products of both in the queue
            // at once would end at the same time, and so would the two softmaxes,
            // with nothing left to run beside them.  Both walk the ring in its
            // order and pass every stage, used or not: a stage's parity then never
            // runs ahead of a warp.  The whole warp walks and waits; one lane issues.
            constexpr uint32_t ID_S = ca_idesc(kTile, false), ID_O = ca_idesc(D, true);
            constexpr uint32_t STEP = S::TILE >> 4;
            const int x = wi - kMmaWarp;
            const uint64_t qdesc = ca_desc(smem_u32(sQ), 16), kdesc = ca_desc(smem_u32(ring), 16);
            const uint64_t vdesc = ca_desc(smem_u32(ring), S::PANEL);
            const uint32_t tS = tmem + x * kTile, tO = tmem + 256 + x * kTile;
            uint32_t cur = 0, par = 0, cleaned = 0;  // ring stage and parity; a parity bit a stage
            uint32_t qs = 0, np = 0, no = 0, ow = 0;  // ow: Oempty waited for
            uint32_t items = 0, last_use = 0;        // the item that used O last
            uint32_t turns = 0;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (!bad && !warp_wait(bar, parity))
                    bad = true;
            };
            auto o_free = [&] {  // the epilogue of O's last use has read it
                if (ow < no)
                    wait(&oempty[x], ow++ & 1);
            };
            auto pass = [&](uint64_t *bar, bool used) {  // when the products issued are done, or now
                if (elect_one()) {
                    if (used)
                        mma_commit(bar);
                    else
                        mbar_arrive(bar);
                }
                __syncwarp();
            };
            auto step_on = [&](bool used) {
                pass(&empty[cur], used);
                if (++cur == NS) {
                    cur = 0;
                    par ^= 1;
                }
            };
            for (bool more = wk.begin(); more && !bad; more = wk.next()) {
                const CaItem &it = wk.it;
                const int len = it.kb - it.ka, pos0 = it.c.len - it.c.n + it.tok0;
                const bool single = it.single;
                ++items;
                // the cleared elements of an item are kept until kBufs items on:
                // this stream's epilogue of two items ago has read its own
                if (last_use + 1 < items)
                    o_free();
                // the stream's key tiles: t with t % 2 == x of a single item; of a
                // pair all for B, the ones its last token sees for A
                const int na = x == 0 ? (pos0 + min(it.ntok, tpt) + kTile - 1) / kTile : it.kb;
                const int cnt = single ? (len + 1 - x) / 2 : max(0, min(it.kb, na) - it.ka);
                const int last = single ? 2 * (cnt - 1) + x : cnt - 1;  // the last one
                const uint32_t slot = single ? qs : qs + x;
                const uint64_t qd = qdesc + (slot & 1) * STEP;
                auto product_s = [&](int t) {  // S with the K tile t of stage `cur`
                    const uint64_t kd = kdesc + cur * STEP;
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            const uint32_t o = ((ks >> 2) * S::PANEL + (ks & 3) * 32) >> 4;
                            mma_ss(tS, qd + o, kd + o, ID_S, ks > 0);
                        }
                        mma_commit(&sfull[x]);
                        if (t == last)
                            mma_commit(&qempty[slot & 1]);
                    }
                    __syncwarp();
                    step_on(true);
                };
                auto skip = [&] {  // a stage of the other stream's
                    wait(&full[cur], par);
                    if (!bad)
                        step_on(false);
                };
                auto hides = [&](int t) { return (it.ka + t + 1) * kTile > pos0 + 1; };
                auto skip_v = [&](int t) {
                    if (hides(t))
                        cleaned ^= 1u << cur;
                    skip();
                };
                // P V with V tile t, then S with K tile `next` (the stage behind it)
                auto burst = [&](int t, int next) {
                    wait(&full[cur], par);
                    if (hides(t)) {
                        // it holds keys some row does not see: cleaned beside the
                        // softmax of the tile's S
                        if (!bad && (single || x == 1))
                            pass(&dirty[x], false);
                        wait(&clean[cur], cleaned >> cur & 1);
                        cleaned ^= 1u << cur;
                    }
                    const bool more_s = next <= last;
                    if (next < len) {
                        const bool wrap = cur + 1 == NS;
                        wait(&full[wrap ? 0 : cur + 1], par ^ wrap);
                    }
                    const bool first = t == (single ? x : 0);
                    wait(&pready[x], np++ & 1);
                    if (first) {
                        o_free();
                        ++no;
                        last_use = items;
                    }
                    wait(&turn[x], turns++ & 1);
                    if (bad)
                        return;
                    const uint64_t vd = vdesc + cur * STEP;
                    fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < kTile / 16; ++ks)
                            mma_ts(tO, tS + ks * 8, vd + ks * (2048 >> 4), ID_O, !first || ks > 0);
                        if (t == last)
                            mma_commit(&ofull[x]);
                    }
                    __syncwarp();
                    step_on(true);
                    if (more_s)
                        product_s(next);
                    else if (next < len)
                        step_on(false);
                    pass(&turn[1 - x], false);
                };
                auto no_burst = [&] {
                    wait(&turn[x], turns++ & 1);
                    if (!bad)
                        pass(&turn[1 - x], false);
                };
                wait(&qfull[qs & 1], (qs >> 1) & 1);
                if (!single)
                    wait(&qfull[(qs + 1) & 1], ((qs + 1) >> 1) & 1);
                if (bad)
                    break;
                if (!single)
                    pass(&qempty[(qs + 1 - x) & 1], false);  // the other stream's queries
                if (cnt == 0)
                    pass(&qempty[slot & 1], false);
                auto first_s = [&](bool mine, int t) {
                    wait(&full[cur], par);
                    if (bad)
                        return;
                    if (!mine) {
                        step_on(false);
                        return;
                    }
                    fence_after();
                    product_s(t);
                };
                if (single) {  // K0 K1 | V0 K2 | V1 K3 | ..: the groups in turn A's and B's
                    first_s(x == 0, 0);
                    if (len > 1)
                        first_s(x == 1, 1);
                    for (int t = 0; t < len && !bad; t += 2) {
                        if (x == 1) {
                            skip_v(t);
                            if (t + 2 < len)
                                skip();
                        }
                        if (t + x < len)
                            burst(t + x, t + x + 2);
                        else
                            no_burst();
                        if (x == 0 && t + 1 < len) {
                            skip_v(t + 1);
                            if (t + 3 < len)
                                skip();
                        }
                    }
                } else {  // K0 | V0 K1 | V1 K2 | ..
                    first_s(cnt > 0, 0);
                    for (int t = 0; t < len && !bad; ++t) {
                        if (t < cnt) {
                            burst(t, t + 1);
                        } else {
                            skip_v(t);
                            if (t + 1 < len)
                                skip();
                            no_burst();
                        }
                    }
                }
                qs += single ? 1 : 2;
            }
            // every product issued is done before the tensor memory is freed
            pass(done, true);
            bad |= !warp_wait(done, 0);
        } else {
            // ----------------------------------------------- cleaning of V
            uint32_t base = 0, items = 0, dirtied[2] = {0u, 0u};
            for (bool more = wk.begin(); more && !bad; more = wk.next()) {
                const CaItem &it = wk.it;
                const int len = it.kb - it.ka, pos0 = it.c.len - it.c.n + it.tok0;
                const int buf = items % kBufs;
                const int t0 = max(0, (pos0 + 1) / kTile - it.ka);  // first tile with hidden keys
                bool hit = false;
                int *cleared = cleared_ptr<D>(a.part) + buf * D;
                for (int t = t0; t < len && !bad; ++t) {
                    const int k0 = (it.ka + t) * kTile;
                    const uint32_t pos =
                        base + (it.single && t + 1 < len ? 2 * t + 2 : 2 * t + 1);
                    const int s = pos % NS;
                    // a products' warp has seen the tile arrive, and waits for `clean`
                    const bool by_a = it.single && !(t & 1);
                    if (!warp_wait(by_a ? &dirty[0] : &dirty[1], (by_a ? dirtied[0] : dirtied[1]) & 1) ||
                        !warp_wait(&full[s], (pos / NS) & 1)) {
                        bad = true;
                        break;
                    }
                    ++dirtied[by_a ? 0 : 1];
                    if (t == t0 && lane == 0)
                        sFlag[buf] = 0;
                    // CPR chunks of 16 bytes a row, RPW rows at a time, UN of those in flight
                    constexpr int CPR = D / 8, RPW = 32 / CPR, UN = 8;
                    const int ch = lane % CPR;
                    const uint32_t tile = smem_u32(ring + s * S::TILE);
                    for (int rb = max(0, pos0 + 1 - k0) + lane / CPR; rb - lane / CPR < kTile;
                         rb += UN * RPW) {
                        uint4 v[UN];
                        bool odd = false;
#pragma unroll
                        for (int u = 0; u < UN; ++u) {
                            const int r = min(rb + u * RPW, kTile - 1);
                            v[u] = ld_shared_v4(tile + swz(r, ch, kTile));
                        }
#pragma unroll
                        for (int u = 0; u < UN; ++u) {
                            // an exponent of all ones carries into the element's top bit
                            const uint32_t m = 0x7f807f80u, c = 0x00800080u;
                            const int r = rb + u * RPW;
                            odd |= r < kTile && k0 + r < it.c.len &&
                                   ((((v[u].x & m) + c) | ((v[u].y & m) + c) |
                                     ((v[u].z & m) + c) | ((v[u].w & m) + c)) &
                                    0x80008000u) != 0;
                        }
#pragma unroll
                        for (int u = 0; u < UN; ++u) {
                            const int r = rb + u * RPW;
                            if (r < kTile && k0 + r >= it.c.len)
                                st_shared_v4(tile + swz(r, ch, kTile), make_uint4(0u, 0u, 0u, 0u));
                        }
                        if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
                            for (int u = 0; u < UN; ++u) {
                                const int r = rb + u * RPW;
                                const bool mine = r < kTile && k0 + r < it.c.len;
                                const uint32_t at = tile + swz(min(r, kTile - 1), ch, kTile);
                                uint4 w = ld_shared_v4(at);
                                uint32_t found = 0;
                                auto word = [&](uint32_t &e, int x) {
                                    if ((e & 0x7f80u) == 0x7f80u) {
                                        found |= 1u << x;
                                        e &= 0xffff0000u;
                                    }
                                    if ((e & 0x7f800000u) == 0x7f800000u) {
                                        found |= 2u << x;
                                        e &= 0xffffu;
                                    }
                                };
                                word(w.x, 0);
                                word(w.y, 2);
                                word(w.z, 4);
                                word(w.w, 6);
                                if (!__any_sync(0xffffffffu, mine && found))
                                    continue;
                                if (!hit) {  // the item's first
                                    for (int x = lane; x < D; x += 32)
                                        __stcg(cleared + x, 0x7fffffff);
                                    if (lane == 0)
                                        sFlag[buf] = 1;
                                    __threadfence();
                                    __syncwarp();
                                    hit = true;
                                }
                                if (mine && found) {
                                    st_shared_v4(at, w);
                                    for (int x = 0; x < 8; ++x)
                                        if (found >> x & 1)
                                            atomicMin(cleared + ch * 8 + x, k0 + r);
                                }
                            }
                        }
                    }
                    if (hit)
                        __threadfence();
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
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSmRegs));
        // ------------------------------------------------------- softmax
        // A row belongs to two threads, of warps w (columns 0 .. 63 of S and the
        // first half of O's) and w + 4 (the others), which exchange its maximum
        constexpr int HK = kTile / 2, HD = D / 2;
        const int x = wi / kSmWarps;           // tile A or B
        const int wq = wi & 3;                 // tensor-memory lanes 32 wq ..
        const int hf = (wi >> 2) & 1;          // the row's half
        const int r = wq * 32 + lane;          // row of the tile
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tS = tmem + x * kTile + lane_off, tO = tmem + 256 + x * kTile + lane_off + hf * HD;
        float *max_mine = sMax + (x * 2 + hf) * kTile + r, *max_other = sMax + (x * 2 + 1 - hf) * kTile + r;
        const uint32_t pair_bar = 1 + x * 4 + wq;  // the barrier of this warp and its other half
        const bool neg = a.logit_scale < 0.f;
        const float ls = fmaxf(fabsf(a.logit_scale), 1e-30f);
        const float grow = kRescale / ls;
        const int rtok = r / G, rg = r - rtok * G;
        uint32_t ns = 0, no = 0, items = 0, halves = 0;
        bool lent = false;  // B: its (max, sum) of a join lie in sMax
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
            if (lent && cnt > 0) {  // A has taken what B left in place of its maxima
                if (!bad && !ca_wait(taken, halves++ & 1))
                    bad = true;
                bad = __any_sync(0xffffffffu, bad);
                lent = false;
            }
            float mref = -INFINITY, negm = 0.f;
            float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
            for (int t = 0; t < cnt; ++t) {
                const int k0 = (it.ka + (single ? 2 * t + x : t)) * kTile;
                if (!bad && !ca_wait(&sfull[x], ns & 1))
                    bad = true;
                ++ns;
                bad = __any_sync(0xffffffffu, bad);
                if (bad) {  // a warp that gave up still passes every barrier of its pair
                    if (live)
                        bar_sync(pair_bar, 64);
                    continue;
                }
                fence_after();
                if (live) {
                    uint32_t sr[HK];
#pragma unroll
                    for (int o = 0; o < HK; o += 16)
                        ld16(tS + hf * HK + o, sr, o);
                    ld_wait(sr);
                    float *s = reinterpret_cast<float *>(sr);
                    if (neg) {
#pragma unroll
                        for (int c = 0; c < HK; ++c)
                            s[c] = -s[c];
                    }
                    if (k0 + kTile > wlim) {
                        const int m = lim - k0 - hf * HK;
#pragma unroll
                        for (int c = 0; c < HK; ++c)
                            s[c] = c < m ? s[c] : -INFINITY;
                    }
                    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int c = 4; c < HK; c += 8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            mx[e] = c + 4 + e < HK ? fmaxf(fmaxf(mx[e], s[c + e]), s[c + 4 + e])
                                                   : fmaxf(mx[e], s[c + e]);
                    }
                    float m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    *max_mine = m_new;
                    bar_sync(pair_bar, 64);  // also: both halves of S are in registers
                    m_new = fmaxf(m_new, *max_other);
                    const bool up = t == 0 ? m_new > -INFINITY : m_new > mref + grow;
                    float f = 1.f;
                    if (up) {
                        const float old = negm;
                        const bool fresh = mref == -INFINITY;
                        mref = m_new;
                        negm = -m_new * ls;
                        f = fresh ? 0.f : ex2_approx(negm - old);
                        l0 *= f;
                        l1 *= f;
                        l2 *= f;
                        l3 *= f;
                    }
#pragma unroll
                    for (int c = 0; c < HK; c += 32) {
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
                        st16(tS + hf * (HK / 2) + c / 2, pk, 0);
                    }
                    // O by the factor, this half of the row in flight at once
                    if (t > 0 && __any_sync(0xffffffffu, up)) {
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
            float l = (l0 + l1) + (l2 + l3);
            float m = mref == -INFINITY ? -INFINITY : -negm;  // base 2, scaled
            if (cnt > 0) {
                if (!bad && !ca_wait(&ofull[x], no & 1))
                    bad = true;
                ++no;
                fence_after();
            }
            bad = __any_sync(0xffffffffu, bad);
            if (cnt > 0) {  // the other half's sum
                *max_mine = l;
                bar_sync(pair_bar, 64);
                const float other = *max_other;
                l = hf == 0 ? l + other : other + l;
                bar_sync(pair_bar, 64);  // read before the next maximum is written
            }
            const int buf = items % kBufs;
            ++items;
            const bool whole = it.ka == 0 && it.kb == it.kt;
            const bool join = single && len > 1;  // B holds the odd key tiles
            if (single && x == 1) {
                if (join) {  // A reads both halves of O: the lanes are the same
                    *max_mine = hf == 0 ? m : l;
                    lent = true;
                    fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(half);
                }
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
            // only the tiles that were cleaned order the flag before this read
            const int last_tile = it.ka + (single ? len : cnt) - 1;
            const bool poisoned =
                !bad && cnt > 0 && (last_tile + 1) * kTile > pos0 + 1 && sFlag[buf] != 0;
            const bool read_o = cnt > 0 && live && !bad;
            // XC columns of O, the halves joined, poisoned ones NaN
            auto load_o = [&](int c, uint32_t (&v)[XC]) {
                if (read_o) {
#pragma unroll
                    for (int o = 0; o < XC; o += 16)
                        ld16(tO + c + o, v, o);
                    if (join) {
                        uint32_t w[XC];
#pragma unroll
                        for (int o = 0; o < XC; o += 16)
                            ld16(tO + kTile + c + o, w, o);
                        ld_wait(v);
                        ld_wait(w);
#pragma unroll
                        for (int e = 0; e < XC; ++e)
                            v[e] = __float_as_uint(__uint_as_float(v[e]) * fa +
                                                   __uint_as_float(w[e]) * fb);
                    } else {
                        ld_wait(v);
                    }
                    if (poisoned) {
#pragma unroll
                        for (int e = 0; e < XC; ++e)
                            if (__ldcg(cleared_ptr<D>(a.part) + buf * D + hf * HD + c + e) < lim)
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
                bs = static_cast<int>(quotient(it.x, plan.share));
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
            __nv_bfloat16 *dst = a.out + (tok_row * a.Hq + it.h * G + rg) * D + hf * HD;
            const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
            for (int c = 0; c < HD; c += XC) {
                uint32_t v[XC];
                load_o(c, v);
                if (c + XC >= HD)
                    o_done();
                if (r < rows && !bad) {
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < XC; e += 16) {
                            uint32_t o[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                o[k] = pack_bf16x2(__uint_as_float(v[e + 2 * k]) * inv,
                                                   __uint_as_float(v[e + 2 * k + 1]) * inv);
                            st_global_v8(dst + c + e, o);
                        }
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
            if (whole)
                continue;
            // a partial result: the last of the item's shares to arrive joins them
            if (r < rows && hf == 0)
                reinterpret_cast<float2 *>(slot + 2 * kTile * D)[row] = make_float2(m, l);
            __threadfence();
            bar_sync(9 + x, 32 * kSmWarps);
            if (r == 0 && hf == 0) {
                const unsigned n = __popc(parts);
                sLast[x] = atomicInc(&a.arrived[2 * bs + x], n - 1) == n - 1;
            }
            bar_sync(9 + x, 32 * kSmWarps);
            if (!sLast[x])
                continue;
            __threadfence();
            constexpr int LPR = D / 4, RPW = 32 / LPR;  // lanes a row, rows a warp
            const int first = __ffs(parts) - 1;
            for (int rr = (hf * 4 + wq) * RPW + lane / LPR; rr < rows; rr += kSmWarps * RPW) {
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
    if (wi == kMmaWarp) {
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
        zp_chunk_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
    if (e != cudaSuccess)
        return e;
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
