// zp_sample.cu -- the next token from logits (zp_sample), and the filtered
// probabilities that zp_verify_draft takes (zp_token_probs).
//
// A row's weights are w = exp((l - max l) / T).  Kept are the top_k largest logits
// (ties to the lower index), of these the shortest run of the largest whose weights
// reach top_p of theirs, of these the weights of at least min_p.  All three keep a prefix
// of the row in falling order, so the kept set is "above tau, and the first m of those
// equal to tau", cut off at a gap of T ln(1 / min_p) to the maximum.  The token is the
// lowest kept index whose running sum exceeds u times the sum of all kept.
//
// Weights are whole numbers of 2^-44 (zp_sample.cuh), so every sum is exact and the same
// in whatever order it is formed.  Only where a sum decides nothing (the probabilities
// of a row without top_p) are they plain fp32 numbers.
//
// One cluster of CTAs a row, which lies in their shared memory: it is read from memory
// once.  A warp owns a contiguous run of it, its lanes 16 bytes each side by side.  tau is
// found in one of two ways:
//   top_k of at most kList / 2: the k-th largest of the threads' maxima is a bound below
//       which none of the k largest lies, and few others lie above it.  What does is gathered
//       and sorted by CTA 0, which then has all that may be kept, and finds the cuts and
//       the token by itself.
//   else: a histogram over the gap to the maximum (counts, or weights where a sum is
//       asked for).  The bucket in which the count or the sum is reached is gathered and
//       sorted; one of more than kList entries is cut up again by the bits of its
//       values, until it fits or holds one value alone.
//
// Measured, fp32 logits drawn from a normal distribution of deviation 3, device time of calls in a
// row: 256 rows of 151,936 without filters 152 us (0.16 GB, 1.0 TB/s), with top_k 50 112, with top_p
// 0.9 350; the probabilities of 1,280 rows 634, 670 and 1,530 (1.56 GB, 2.4 to 1.0 TB/s); one row of
// 32,000 8 to 21.  What bounds it: without filters the weights (about 40 instructions each, issue
// slots half full), with them the chains in which CTA 0 finds a cut while the others of its cluster
// wait; a row is held for 15 to 45 us, and shared memory holds 38 rows of that size.
#include <algorithm>

#include "zp_sample.cuh"

namespace zp {

namespace {

constexpr int kSpThreads = 512;
constexpr int kSpCtas = 8;       // of a cluster, at most: the portable most
constexpr int kBuckets = 512;
constexpr int kList = 1024;
constexpr int kSmall = 128;      // entries that are ordered by counting
constexpr int kSpWarps = kSpThreads / 32;

__device__ const WeightTable d_table{};

// What CTA 0 finds out about a cut.
struct Cut {
    uint64_t mass;    // weights above the bucket, then of the whole kept set
    uint32_t above;   // entries above the bucket
    uint32_t in;      // and in it; at the end, those equal to tau
    uint32_t lo, hi;  // the keys of a cut bucket
    int bucket;
    int m;            // of those equal to tau, the ones kept
    float tau;
    int done;         // nothing is left to do for the other CTAs
};

struct SpShared {
    uint64_t bar[kSpWarps];
    uint64_t list[kList];
    uint64_t table[1024];
    uint32_t count[kBuckets];
    uint32_t part[3][kBuckets];  // sums of weights' bits 0 .. 15, 16 .. 31 and 32 ..
    uint64_t runs[kSpCtas * kSpWarps];       // sums of the warps' runs
    uint32_t ties[kSpCtas * kSpWarps];       // their entries equal to tau
    uint64_t scan64[kSpWarps];
    float2 ends[kSpCtas];                    // the CTAs' (largest, smallest finite)
    uint32_t scan32[kSpWarps];
    uint32_t key_lo, key_hi, listed, equal, equal_upto;
    // the row's, as the functions below read it
    float M, per_gap, least, u, top_p;
    int top_k, mis;
    WeightScale scale;
    float2 gap;   // the largest gap to the maximum that min_p allows, as a pair
    Cut cut;      // CTA 0's
    Cut told[2];  // what it told all, the last two times
};

__device__ __forceinline__ void unpack(const uint4 &u, float (&v)[4])
{
    v[0] = __uint_as_float(u.x);
    v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z);
    v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack(const uint4 &u, float (&v)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack(const float (&v)[4])
{
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack(const float (&v)[8])
{
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// An order-preserving key of a logit (-0 as +0), and back.
__device__ __forceinline__ uint32_t key_of(float x) { return f32_order(x + 0.f); }
__device__ __forceinline__ float value_of(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ void st_dsmem_u32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_dsmem_u64(uint32_t addr, uint64_t v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void min_dsmem_u32(uint32_t addr, uint32_t v)
{
    asm volatile("red.shared::cluster.min.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void max_dsmem_u32(uint32_t addr, uint32_t v)
{
    asm volatile("red.shared::cluster.max.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// The cluster's barrier, for warps that come out of loops their lanes leave one by one.
__device__ __forceinline__ void all_ctas()
{
    __syncwarp();
    cluster_sync();
}

template <class T>
__device__ __forceinline__ T warp_incl(T v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o)
            v += y;
    }
    return v;
}

template <class T>
__device__ __forceinline__ T warp_sum(T v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The sum of the threads before this one; `total`: of all.
template <class T>
__device__ __forceinline__ T block_before(T v, T *scratch, T &total)
{
    const int lane = threadIdx.x & 31, wi = threadIdx.x >> 5;
    const T incl = warp_incl(v, lane);
    __syncthreads();  // the last use of the scratch is over
    if (lane == 31)
        scratch[wi] = incl;
    __syncthreads();
    const T w = lane < kSpWarps ? scratch[lane] : 0;
    const T wincl = warp_incl(w, lane);
    total = __shfl_sync(0xffffffffu, wincl, kSpWarps - 1);
    return __shfl_sync(0xffffffffu, wincl - w, wi) + incl - v;
}

// Sorts list[0 .. n) by the CTA, falling; n at most kList = 2 kSpThreads.  Every thread holds
// two neighbours' places; what lies less than 64 apart is compared in a warp's registers.
__device__ __noinline__ void sort_falling(uint64_t *list, int n)
{
    static_assert(kList == 2 * kSpThreads, "two entries a thread");
    const int t = threadIdx.x, lane = t & 31;
    int size = 64;
    while (size < n)
        size *= 2;
    const bool active = (t & ~31) * 2 < size;  // whole warps
    __syncthreads();
    uint64_t a = 2 * t < n ? list[2 * t] : 0, b = 2 * t + 1 < n ? list[2 * t + 1] : 0;
    for (int span = 2; span <= size; span *= 2) {
        const bool falling = (2 * t & span) == 0;
        for (int d = span / 2; d; d /= 2) {
            if (d >= 64) {  // the partner is in another warp
                __syncthreads();
                if (active) {
                    list[2 * t] = a;
                    list[2 * t + 1] = b;
                }
                __syncthreads();
                if (active) {
                    const uint64_t x = list[2 * t ^ d], y = list[2 * t + 1 ^ d];
                    const bool take_more = ((2 * t & d) == 0) == falling;
                    a = (a > x) == take_more ? a : x;
                    b = (b > y) == take_more ? b : y;
                }
            } else if (d >= 2) {
                const uint64_t x = __shfl_xor_sync(0xffffffffu, a, d / 2);
                const uint64_t y = __shfl_xor_sync(0xffffffffu, b, d / 2);
                const bool take_more = ((2 * lane & d) == 0) == falling;
                a = (a > x) == take_more ? a : x;
                b = (b > y) == take_more ? b : y;
            } else if ((a < b) == falling) {
                const uint64_t x = a;
                a = b;
                b = x;
            }
        }
    }
    __syncthreads();
    if (active) {
        list[2 * t] = a;
        list[2 * t + 1] = b;
    }
    __syncthreads();
}

// floor(u * s), u below 1 and not below 0.
__device__ __forceinline__ uint64_t part_of(float u, uint64_t s)
{
    const uint32_t b = __float_as_uint(u);
    const int e = max(static_cast<int>(b >> 23), 1);
    const uint64_t m = (b & 0x7fffffu) | (b >> 23 ? 0x800000u : 0u);
    const int sh = 150 - e;  // u = m 2^-sh, sh >= 24
    const uint64_t hi = __umul64hi(m, s), lo = m * s;
    if (sh < 64)
        return hi << (64 - sh) | lo >> sh;
    return sh < 128 ? hi >> (sh - 64) : 0;
}

// ceil(p * s), p above 0 and below 1.
__device__ __noinline__ uint64_t target_of(float p, uint64_t s)
{
    const uint64_t f = part_of(p, s);
    // exact when p * s has no fraction: p = m 2^-sh
    const uint32_t b = __float_as_uint(p);
    const int sh = 150 - max(static_cast<int>(b >> 23), 1);
    const uint64_t m = (b & 0x7fffffu) | (b >> 23 ? 0x800000u : 0u);
    const uint64_t lo = m * s, hi = __umul64hi(m, s);
    bool rest;
    if (sh < 64)
        rest = (lo & ((1ull << sh) - 1)) != 0;
    else if (sh < 128)
        rest = lo != 0 || (hi & ((1ull << (sh - 64)) - 1)) != 0;
    else
        rest = (lo | hi) != 0;
    return f + rest;
}

// The kept sum that a row's random number asks to be exceeded.
__device__ __forceinline__ uint64_t level_of(float u, uint64_t total)
{
    return u >= 1.f ? total - 1 : u > 0.f ? part_of(u, total) : 0;
}

__device__ __forceinline__ float value_at(uint64_t entry)
{
    return value_of(static_cast<uint32_t>(entry >> 32));
}

// What follows runs once or twice a row, most of it in CTA 0 alone.  In line it made the kernel
// 330 KB of instructions, now 165 (410 and 222 for bf16 logits); the times are the same.

__device__ __noinline__ uint64_t weight_of(const SpShared &S, float v)
{
    uint64_t w, same;
    weights(S.table, S.scale, S.M, v, v, w, same);
    return w;
}

// CTA 0's sums of the CTAs' histograms: of the weights, a bucket's 64 bits in part[1] and
// part[0].
__device__ __noinline__ void gather_sums(SpShared &S, int ctas, int rank, bool counts, bool weights)
{
    const int tid = threadIdx.x;
    static_assert(kBuckets == kSpThreads, "a bucket a thread");
    all_ctas();
    if (rank != 0)
        return;
    uint32_t n[kSpCtas], w[3][kSpCtas];  // all on their way at once
#pragma unroll
    for (int r = 0; r < kSpCtas; ++r) {
        n[r] = w[0][r] = w[1][r] = w[2][r] = 0;
        if (counts && r < ctas)
            n[r] = ld_dsmem_u32(dsmem_addr(&S.count[tid], r));
        if (weights && r < ctas)
#pragma unroll
            for (int k = 0; k < 3; ++k)
                w[k][r] = ld_dsmem_u32(dsmem_addr(&S.part[k][tid], r));
    }
    uint32_t all = 0;
    uint64_t sum = 0;
#pragma unroll
    for (int r = 0; r < kSpCtas; ++r) {
        all += n[r];
        sum += w[0][r] + (static_cast<uint64_t>(w[1][r]) << 16) +
               (static_cast<uint64_t>(w[2][r]) << 32);
    }
    S.count[tid] = all;
    S.part[0][tid] = static_cast<uint32_t>(sum);
    S.part[1][tid] = static_cast<uint32_t>(sum >> 32);
}

// CTA 0 alone: the bucket where `above` + counts reach `k`, or `mass` + weights reach
// `target` (k = 0), from the largest values on, which the last buckets of a `rising`
// histogram hold and the first of the other.  bucket < 0: fewer entries than k.  `in`
// becomes about the number of entries up to the bucket, of a first histogram by weights.
__device__ __noinline__ void find(SpShared &S, uint32_t k, uint64_t target, bool rising)
{
    const int tid = threadIdx.x, lane = tid & 31, wi = tid >> 5;
    const int b = rising ? kBuckets - 1 - tid : tid;  // (the thread's own sums, if falling)
    if (rising)
        __syncthreads();
    const uint32_t n = S.count[b];
    const uint64_t w = static_cast<uint64_t>(S.part[1][b]) << 32 | S.part[0][b];
    const uint32_t upto_n = warp_incl(n, lane);
    const uint64_t upto_w = warp_incl(w, lane);
    if (lane == 31) {
        S.scan32[wi] = upto_n;
        S.scan64[wi] = upto_w;
    }
    __syncthreads();
    const uint32_t sn = lane < kSpWarps ? S.scan32[lane] : 0;
    const uint64_t sw = lane < kSpWarps ? S.scan64[lane] : 0;
    const uint32_t in = warp_incl(sn, lane);
    const uint64_t iw = warp_incl(sw, lane);
    const uint32_t n0 = S.cut.above + __shfl_sync(0xffffffffu, in - sn, wi) + upto_n - n;
    const uint64_t w0 = S.cut.mass + __shfl_sync(0xffffffffu, iw - sw, wi) + upto_w - w;
    const uint32_t all_n = __shfl_sync(0xffffffffu, in, 31);
    const uint64_t all_w = __shfl_sync(0xffffffffu, iw, 31);
    __syncthreads();  // S.cut and the scans are read
    const bool here = k ? n0 < k && n0 + n >= k : w0 < target && w0 + w >= target;
    if (tid == 0 && k > all_n && !rising) {
        S.cut.mass = all_w;
        S.cut.bucket = -1;
        S.cut.tau = -INFINITY;
        S.cut.m = 0x7fffffff;
    }
    if (tid == 0)
        S.cut.in = 0;
    if (here) {
        S.cut.above = n0;
        S.cut.mass = w0;
        S.cut.bucket = b;
    }
    if (!rising && k == 0) {
        __syncthreads();
        if (w0 < target)  // 2^-44 w over the weight in the bucket's middle
            atomicAdd(&S.cut.in,
                      static_cast<uint32_t>(fminf(static_cast<float>(w) * 5.6843419e-14f *
                                                      exp2f((b + 0.5f) / S.per_gap * S.scale.ch),
                                                  1e6f)) + 1);
    }
    __syncthreads();
}

// CTA 0's cut to all, in two places in turn, as a CTA may still read the one before.
__device__ __noinline__ void tell(SpShared &S, int ctas, int rank, int turn)
{
    if (rank == 0) {
        __syncthreads();
        constexpr int W = sizeof(Cut) / 4;
        for (int k = threadIdx.x; k < W * ctas; k += kSpThreads)
            st_dsmem_u32(dsmem_addr(reinterpret_cast<uint32_t *>(&S.told[turn]) + k % W, k / W),
                         reinterpret_cast<const uint32_t *>(&S.cut)[k % W]);
    }
    all_ctas();
}

// CTA 0: of its sorted list of n, the entry at which the count (with `above`) reaches
// k, or the weights (with `mass`) reach `target`; tau, what is kept of it, the weights.
__device__ __noinline__ void cut_list(SpShared &S, int n, uint32_t k, uint64_t target, bool weights)
{
    const int tid = threadIdx.x;
    if (tid == 0)
        S.equal = S.equal_upto = 0;
    constexpr int PL = kList / kSpThreads;
    uint64_t w[PL], sum = 0, all;
#pragma unroll
    for (int j = 0; j < PL; ++j) {
        const int p = tid * PL + j;
        w[j] = weights && p < n ? weight_of(S, value_at(S.list[p])) : 0;
        sum += w[j];
    }
    const uint64_t mass = S.cut.mass;
    const uint32_t above = S.cut.above;
    uint64_t at = mass + block_before(sum, S.scan64, all);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PL; ++j) {
        const int p = tid * PL + j;
        const bool here =
            p < n && (k ? above + p + 1 == k : at < target && at + w[j] >= target);
        at += w[j];
        if (here) {
            S.cut.tau = value_at(S.list[p]);
            S.cut.mass = at;
            S.cut.lo = static_cast<uint32_t>(p);
        }
    }
    __syncthreads();
    const uint32_t key = key_of(S.cut.tau);
    const int last = static_cast<int>(S.cut.lo);
    for (int p = tid; p < n; p += kSpThreads)
        if (static_cast<uint32_t>(S.list[p] >> 32) == key) {
            atomicAdd(&S.equal, 1u);
            if (p <= last)
                atomicAdd(&S.equal_upto, 1u);
        }
    __syncthreads();
    if (tid == 0) {
        S.cut.in = S.equal;
        S.cut.m = static_cast<int>(S.equal_upto);
    }
    __syncthreads();
}

// CTA 0: the same of at most kSmall entries: a thread an entry, which adds up what comes before it
// by value, and then by index.
__device__ __noinline__ void finish_small(SpShared &S, int n, uint64_t row_sum, int32_t *token)
{
    const int tid = threadIdx.x, wi = tid >> 5, top_k = S.top_k;
    const bool by_mass = S.top_p < 1.f;
    const float top_p = S.top_p;
    uint64_t *entries = S.list, *sums = S.list + kSmall;
    const bool mine = tid < n;
    const uint64_t e = mine ? entries[tid] : 0;
    const float v = mine ? value_at(e) : -INFINITY;
    uint64_t w = 0;
    if (wi < kSmall / 32)
        w = mine ? weight_of(S, v) : 0;
    if (tid < kSmall)
        sums[tid] = w;
    if (tid == 0) {
        S.cut.lo = 0;
        S.equal = S.equal_upto = 0;
    }
    __syncthreads();
    int rank_of = 0;
    uint64_t above = 0;
    const int in_k = top_k > 0 ? min(top_k, n) : n;
    if (mine) {
        for (int q = 0; q < n; ++q)
            if (entries[q] > e) {
                ++rank_of;
                above += sums[q];
            }
        if (rank_of == in_k - 1)
            S.scan64[0] = above + w;  // of the top_k
    }
    __syncthreads();
    uint64_t target = ~0ull;
    if (by_mass)
        target = top_p > 0.f
                     ? max(target_of(top_p, row_sum ? row_sum : S.scan64[0]), uint64_t(1))
                     : 1;
    const bool in = mine && rank_of < in_k && above < target;
    const uint64_t kept_w = in && v >= S.least ? w : 0;
    if (tid < kSmall)
        sums[tid] = kept_w;
    if (in)
        atomicMax(&S.cut.lo, static_cast<uint32_t>(rank_of) + 1);
    __syncthreads();
    if (in && rank_of + 1 == static_cast<int>(S.cut.lo))
        S.cut.tau = v;
    uint64_t total = 0, before = 0;
    if (mine)
        for (int q = 0; q < n; ++q) {
            total += sums[q];
            // (the low halves fall with the index)
            if (static_cast<uint32_t>(entries[q]) > static_cast<uint32_t>(e))
                before += sums[q];
        }
    __syncthreads();
    if (mine && v == S.cut.tau) {
        atomicAdd(&S.equal, 1u);
        if (in)
            atomicAdd(&S.equal_upto, 1u);
    }
    if (tid == 0)
        S.cut.mass = total;
    if (mine && token) {
        const uint64_t level = level_of(S.u, total);
        if (before <= level && level < before + kept_w)
            *token = static_cast<int>(0xffffffffu - static_cast<uint32_t>(e)) - S.mis;
    }
    __syncthreads();
    if (tid == 0) {
        S.cut.in = S.equal;
        S.cut.m = static_cast<int>(S.equal_upto);
    }
}

// CTA 0: the cuts of the n entries it has gathered, if they fit in the list, and the token.
// row_sum: the weights that top_p is a part of, 0 for those of the top_k.
__device__ __noinline__ void finish(SpShared &S, int rank, int n, uint64_t row_sum, int32_t *token)
{
    const int tid = threadIdx.x, top_k = S.top_k;
    const float top_p = S.top_p;
    const bool by_mass = top_p < 1.f;
    if (rank != 0)
        return;
    __syncthreads();
    if (tid == 0) {
        S.cut = Cut{};
        S.cut.done = n <= kList;
        S.cut.tau = -INFINITY;
        S.cut.m = 0x7fffffff;
    }
    if (n <= kSmall) {
        finish_small(S, n, row_sum, token);
    } else if (n <= kList) {
        sort_falling(S.list, n);
        int kept = n;
        if (top_k > 0 && n >= top_k) {
            cut_list(S, n, static_cast<uint32_t>(top_k), 0, true);
            kept = top_k;
        }
        if (by_mass) {
            uint64_t sum = row_sum ? row_sum : S.cut.mass;
            if (!row_sum && n < top_k) {  // all there are
                uint64_t s = 0;
                for (int p = tid; p < n; p += kSpThreads)
                    s += weight_of(S, value_at(S.list[p]));
                block_before(s, S.scan64, sum);
            }
            const uint64_t target =
                top_p > 0.f ? max(target_of(top_p, sum), uint64_t(1)) : 1;
            __syncthreads();
            if (tid == 0)
                S.cut.mass = 0;
            __syncthreads();
            cut_list(S, n, 0, target, true);
            kept = static_cast<int>(S.cut.lo) + 1;
        }
        // in the order of their index (which the entry's low half falls with)
        uint64_t e[kList / kSpThreads], sum = 0, total;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kList / kSpThreads; ++j) {
            const int p = j * kSpThreads + tid;
            e[j] = p < kept ? S.list[p] : 0;
            if (p < kept && !(value_at(e[j]) >= S.least))
                e[j] = 0;
            sum += e[j] ? weight_of(S, value_at(e[j])) : 0;
        }
        block_before(sum, S.scan64, total);
        if (tid == 0)
            S.cut.mass = total;
        if (token) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kList / kSpThreads; ++j) {
                const int p = j * kSpThreads + tid;
                if (p < kept)
                    S.list[p] = e[j] << 32 | e[j] >> 32;
            }
            __syncthreads();
            sort_falling(S.list, kept);
            const uint64_t level = level_of(S.u, total);
            constexpr int PL = kList / kSpThreads;
            uint64_t w[PL], s = 0, all;
#pragma unroll
            for (int j = 0; j < PL; ++j) {
                const int p = tid * PL + j;
                const uint64_t v = p < kept ? S.list[p] : 0;
                w[j] = v ? weight_of(S, value_of(static_cast<uint32_t>(v))) : 0;
                s += w[j];
            }
            uint64_t at = block_before(s, S.scan64, all);
#pragma unroll
            for (int j = 0; j < PL; ++j) {
                if (at <= level && level < at + w[j])
                    *token = static_cast<int>(0xffffffffu - static_cast<uint32_t>(
                                                                S.list[tid * PL + j] >> 32)) -
                             S.mis;
                at += w[j];
            }
        }
    }
}

}  // namespace

// A warp's run is J * 32 vectors of 16 bytes; T the logits' type.
template <class T>
__global__ void __launch_bounds__(kSpThreads, 2)
    zp_sample_kernel(const __grid_constant__ SampleArgs a, int ctas, int J)
{
    constexpr int VE = 16 / sizeof(T);
    extern __shared__ __align__(128) uint8_t raw[];
    SpShared &S = *reinterpret_cast<SpShared *>(raw);
    uint4 *x = reinterpret_cast<uint4 *>(raw + (sizeof(SpShared) + 127) / 128 * 128);
    const int tid = threadIdx.x, lane = tid & 31, wi = tid >> 5;
    const int rank = static_cast<int>(cluster_ctarank());
    const int i = blockIdx.x / ctas;
    if (lane == 0) {
        mbar_init(&S.bar[wi], 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();

    // the row as vectors from the 16-byte boundary at or below its first element: vector
    // g holds elements g * VE - mis ..; this warp's are g0 .. g0 + 32 J - 1
    const T *row = static_cast<const T *>(a.logits) + i * a.stride;
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
    const int g0 = (rank * kSpWarps + wi) * J * 32;
    uint4 *run = x + wi * J * 32;
    const int c0 = max(g0, mis ? 1 : 0);  // whole vectors of the row
    const int c1 = min(g0 + J * 32, (mis + a.vocab) / VE);
    if (lane == 0 && c1 > c0) {
        mbar_arrive_expect_tx(&S.bar[wi], (c1 - c0) * 16);
        bulk_g2s(run + (c0 - g0), row + (static_cast<int64_t>(c0) * VE - mis), (c1 - c0) * 16,
                 &S.bar[wi]);
    }

    // the request's parameters
    const int prow = a.req_idx ? a.req_idx[i] : i;
    bool ok = prow >= 0 && prow < a.num_rows;
    const int pr = ok ? prow : 0;
    float temp = a.temperature ? a.temperature[pr] : 1.f;
    int top_k = a.top_k ? a.top_k[pr] : 0;
    const float top_p = a.top_p ? a.top_p[pr] : 1.f;
    const float min_p = a.min_p ? a.min_p[pr] : 0.f;
    const float u = a.u ? a.u[i] : 0.f;
    ok = ok && temp >= 0.f && temp < INFINITY && top_p == top_p && min_p == min_p;
    if (temp == 0.f || !ok) {  // the largest alone
        temp = 1.f;
        top_k = 1;
    }
    temp = fminf(fmaxf(temp, kLeastTemp), kMostTemp);
    if (top_k < 0 || top_k >= a.vocab)
        top_k = 0;
    if (tid == 0) {  // (64-bit arithmetic of a whole CTA would take 3 us)
        const double d = 1.4426950408889634 / static_cast<double>(temp);
        S.scale.ch = static_cast<float>(d);
        S.scale.cl = static_cast<float>(d - static_cast<double>(S.scale.ch));
        S.gap = make_float2(INFINITY, 0.f);
        if (min_p > 0.f) {
            const double g = -static_cast<double>(temp) * log(fmin(static_cast<double>(min_p), 1.0));
            S.gap.x = static_cast<float>(g);
            S.gap.y = static_cast<float>(g - static_cast<double>(S.gap.x));
        }
    }
    for (int k = tid; k < 1024; k += kSpThreads)
        S.table[k] = d_table.v[k];
    for (int b = tid; b < kBuckets; b += kSpThreads)
        S.count[b] = S.part[0][b] = S.part[1][b] = S.part[2][b] = 0;
#pragma unroll 1
    for (int j = 0; j < J; ++j) {
        const int g = g0 + j * 32 + lane;
        if (g >= c0 && g < c1)
            continue;
        float v[VE];
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            const int e = g * VE - mis + k;
            v[k] = e >= 0 && e < a.vocab ? to_f32(row[e]) : -INFINITY;
        }
        run[j * 32 + lane] = pack(v);
    }
    if (c1 > c0 && !mbar_wait(&S.bar[wi], 0))
        set_error(a.sticky, ZP_ERR_TIMEOUT);
    __syncwarp();

    // the largest logit and the smallest finite one; NaN becomes -infinity
    float top = -INFINITY, bottom = INFINITY;
#pragma unroll 1
    for (int j = 0; j < J; ++j) {
        float v[VE];
        unpack(run[j * 32 + lane], v);
        bool nan = false;
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            nan |= v[k] != v[k];
            top = fmaxf(top, v[k]);
            bottom = fminf(bottom, v[k] > -INFINITY ? v[k] : INFINITY);
        }
        if (nan) {
#pragma unroll
            for (int k = 0; k < VE; ++k)
                v[k] = v[k] != v[k] ? -INFINITY : v[k];
            run[j * 32 + lane] = pack(v);
        }
    }
    const float my_top = top;
    top = value_of(__reduce_max_sync(0xffffffffu, key_of(top)));
    bottom = value_of(__reduce_min_sync(0xffffffffu, key_of(bottom)));
    float2 *warp_ends = reinterpret_cast<float2 *>(S.scan64);
    if (lane == 0)
        warp_ends[wi] = make_float2(top, bottom);
    __syncthreads();
    cluster_arrive();  // the other CTAs have started once it is waited for
    const WeightScale c = S.scale;
    const float gap_h = S.gap.x, gap_l = S.gap.y;
    for (int w = 0; w < kSpWarps; ++w) {
        top = fmaxf(top, warp_ends[w].x);
        bottom = fminf(bottom, warp_ends[w].y);
    }
    cluster_wait();
    if (tid < ctas)
        st_dsmem_u64(dsmem_addr(&S.ends[rank], tid),
                     static_cast<uint64_t>(__float_as_uint(bottom)) << 32 | __float_as_uint(top));
    all_ctas();
    for (int r = 0; r < ctas; ++r) {
        top = fmaxf(top, S.ends[r].x);
        bottom = fminf(bottom, S.ends[r].y);
    }
    const float M = top;

    // Writes the row's probabilities from those that `prob` gives for a value and, where ties are
    // cut, the number of entries equal to tau before it.
    auto write_row = [&](auto prob, bool ranked, float tau, int t) {
        const int psz = a.prob_bf16 ? 2 : 4;
        uint8_t *to = static_cast<uint8_t *>(a.probs) + (i * a.prob_stride - mis) * psz;
        const bool whole = reinterpret_cast<uintptr_t>(to) % 16 == 0;
#pragma unroll 1
        for (int j = 0; j < J; ++j) {
            float v[VE], p[VE];
            unpack(run[j * 32 + lane], v);
            if (ranked) {
                int n = 0;
#pragma unroll
                for (int k = 0; k < VE; ++k)
                    n += v[k] == tau;
                const int upto = warp_incl(n, lane);
                int before = t + upto - n;
                t += __shfl_sync(0xffffffffu, upto, 31);
#pragma unroll
                for (int k = 0; k < VE; ++k) {
                    p[k] = prob(v[k], before);
                    before += v[k] == tau;
                }
            } else {
#pragma unroll
                for (int k = 0; k < VE; ++k)
                    p[k] = prob(v[k], 0);
            }
            const int64_t g = g0 + j * 32 + lane;
            if (whole && g >= c0 && g < c1) {
                if (a.prob_bf16) {
                    uint32_t w[VE / 2];
#pragma unroll
                    for (int k = 0; k < VE; k += 2)
                        w[k / 2] = pack_bf16x2(p[k], p[k + 1]);
                    if constexpr (VE == 8)
                        st_global_v4(to + g * VE * 2, make_uint4(w[0], w[1], w[2], w[3]));
                    else
                        *reinterpret_cast<uint2 *>(to + g * VE * 2) = make_uint2(w[0], w[1]);
                } else {
#pragma unroll
                    for (int k = 0; k < VE; k += 4)
                        st_global_v4(to + (g * VE + k) * 4,
                                     make_uint4(__float_as_uint(p[k]), __float_as_uint(p[k + 1]),
                                                __float_as_uint(p[k + 2]),
                                                __float_as_uint(p[k + 3])));
                }
                continue;
            }
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                const int64_t e = g * VE - mis + k;
                if (e < 0 || e >= a.vocab)
                    continue;
                if (a.prob_bf16)
                    reinterpret_cast<__nv_bfloat16 *>(to)[g * VE + k] = __float2bfloat16_rn(p[k]);
                else
                    reinterpret_cast<float *>(to)[g * VE + k] = p[k];
            }
        }
    };
    if (!ok || M == -INFINITY) {  // the whole cluster alike
        if (rank == 0 && tid == 0) {
            set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
            if (a.tokens)
                a.tokens[i] = -1;
        }
        if (a.probs)
            write_row([](float, int) { return 0.f; }, false, 0.f, 0);
        return;
    }
    // The weights of vector j of the lane: `take` gets a value and its weight.
    auto each_weight = [&](int j, auto take) {
        float v[VE];
        unpack(run[j * 32 + lane], v);
#pragma unroll
        for (int k = 0; k < VE; k += 2) {
            uint64_t w0, w1;
            weights(S.table, c, M, v[k], v[k + 1], w0, w1);
            take(v[k], w0);
            take(v[k + 1], w1);
        }
    };
    // The least value whose weight is at least min_p: the gap of T ln(1 / min_p) to the
    // maximum, as a value, is found to within a step or two, and the lanes test the values
    // around.  Without min_p the least finite one.
    float least = -3.4028235e38f;
    if (min_p > 0.f) {
        const double at =
            static_cast<double>(M) - (static_cast<double>(gap_h) + static_cast<double>(gap_l));
        const float near = fmaxf(static_cast<float>(at), least);
        const uint32_t key = key_of(fminf(near, M)) - 16 + lane;
        const float v = value_of(key);
        float h, l;
        gap(M, v, h, l);
        const bool enough = key >= key_of(M) || h < gap_h || (h == gap_h && l <= gap_l);
        const unsigned m = __ballot_sync(0xffffffffu, enough);
        least = fminf(__shfl_sync(0xffffffffu, v, m ? __ffs(m) - 1 : 31), M);
    }
    auto entry_of = [&](float v, int j, int k) {  // falling by value, then rising by index
        return static_cast<uint64_t>(key_of(v)) << 32 |
               (0xffffffffu - static_cast<uint32_t>((g0 + j * 32 + lane) * VE + k));
    };

    // ---------------------------------------------------------------- the cut
    Cut cut{};
    cut.tau = -INFINITY;
    cut.m = 0x7fffffff;
    // (finite, as the maximum's place, 0 times it, is 0: of a range below 1.5e-36 it would not be)
    constexpr float kBig = 3.4e38f;  // (also in place of infinite logits)
    const float range = fminf(64.f / c.ch, M - bottom);
    const float per_gap = range > 0.f ? fminf(kBuckets / range, kBig) : 0.f;
    const float big_M = fminf(M, kBig);
    auto place_of = [&](float v) { return (big_M - fminf(v, kBig)) * per_gap; };  // falls with v
    auto bucket_of = [&](float v) { return min(kBuckets - 1, static_cast<int>(place_of(v))); };
    // Whether v lies in the buckets from .. to: `from` and `to` + 1 as numbers, `to` + 1
    // infinite for the last.
    auto in_buckets = [&](float v, float from, float end) {
        const float at = place_of(v);
        return at >= from && (at < end || end == INFINITY) && v > -INFINITY;
    };
    auto end_of = [&](int b) {
        return b >= kBuckets - 1 ? INFINITY : static_cast<float>(b + 1);
    };
    if (tid == 0) {
        S.M = M;
        S.per_gap = per_gap;
        S.least = least;
        S.u = u;
        S.top_p = top_p;
        S.top_k = top_k;
        S.mis = mis;
    }
    int turn = 0;
    auto told = [&] {  // CTA 0's cut
        turn ^= 1;
        tell(S, ctas, rank, turn);
        cut = S.told[turn];
    };
    // (a CTA has at most 2^15.5 entries, so that no sum of 16 bits of each passes 32)
    auto add_weight = [&](int b, uint64_t w) {
        const uint32_t low = static_cast<uint32_t>(w), high = static_cast<uint32_t>(w >> 32);
        atomicAdd(&S.part[0][b], low & 0xffffu);
        if (low >> 16)
            atomicAdd(&S.part[1][b], low >> 16);
        if (high)
            atomicAdd(&S.part[2][b], high);
    };
    // Every entry above -infinity is counted under `place` (below 0: not at all).
    auto histogram = [&](bool counts, bool weights, auto place) {
#pragma unroll 1
        for (int j = 0; j < J; ++j) {
            float v[VE];
            unpack(run[j * 32 + lane], v);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                const int b = v[k] > -INFINITY ? place(v[k]) : -1;
                if (b < 0)
                    continue;
                if (counts)
                    atomicAdd(&S.count[b], 1u);
                if (weights)
                    add_weight(b, weight_of(S, v[k]));
            }
        }
        gather_sums(S, ctas, rank, counts, weights);
    };
    auto clear = [&] {
        for (int b = tid; b < kBuckets; b += kSpThreads)
            S.count[b] = S.part[0][b] = S.part[1][b] = S.part[2][b] = 0;
        __syncthreads();
    };
    // The entries for which `inside` holds into the CTAs' lists, and these, if that is not too
    // much, one behind the other into CTA 0's; there, how many entries there are.
    auto gather = [&](auto inside) {
        __syncthreads();
        if (tid == 0)
            S.listed = 0;
        __syncthreads();
#pragma unroll 1
        for (int j = 0; j < J; ++j) {
            float v[VE];
            unpack(run[j * 32 + lane], v);
            bool in[VE], any = false;
#pragma unroll
            for (int k = 0; k < VE; ++k)
                any |= in[k] = inside(v[k]);
            if (!any)
                continue;
#pragma unroll
            for (int k = 0; k < VE; ++k)
                if (in[k]) {
                    const uint32_t at = atomicAdd(&S.listed, 1u);
                    if (at < kList)
                        S.list[at] = entry_of(v[k], j, k);
                }
        }
        all_ctas();
        uint32_t n = S.listed;
        if (rank == 0) {
            // lane r: CTA r's entries, and those before them
            const uint32_t theirs =
                lane < ctas ? ld_dsmem_u32(dsmem_addr(&S.listed, lane)) : 0;
            const uint32_t upto = warp_incl(theirs, lane);
            n = __shfl_sync(0xffffffffu, upto, 31);
            // (CTA 0's own lie at the front already)
            uint32_t first[kSpCtas];
#pragma unroll
            for (int r = 0; r < kSpCtas; ++r)
                first[r] = __shfl_sync(0xffffffffu, upto - theirs, r);
            for (uint32_t p = tid; n <= kList && p < n; p += kSpThreads) {
                int from = 0;
                uint32_t at = p;
#pragma unroll
                for (int r = 1; r < kSpCtas; ++r)
                    if (r < ctas && p >= first[r]) {
                        from = r;
                        at = p - first[r];
                    }
                if (from)
                    S.list[p] = ld_dsmem_u64(dsmem_addr(&S.list[at], from));
            }
            __syncthreads();
        }
        return n;
    };
    const bool by_mass = top_p < 1.f;
    int32_t *token = a.tokens ? a.tokens + i : nullptr;
    bool counted = false;  // CTA 0 holds the first histogram's sums
    // The cut where the count reaches k, or (k = 0) the weights reach `target`.
    // `found`: its bucket is.
    auto select = [&](uint32_t k, uint64_t target, bool weights, bool found) {
        if (!counted) {
            clear();
            histogram(k > 0, weights, bucket_of);
        }
        counted = true;
        if (!found) {
            if (rank == 0) {
                __syncthreads();
                if (tid == 0)
                    S.cut = Cut{};
                __syncthreads();
                find(S, k, target, false);
            }
            told();
        }
        const int bucket = cut.bucket;
        if (bucket < 0)
            return;
        uint32_t lo = 0, hi = 0xffffffffu;
        const float from = static_cast<float>(bucket), end = end_of(bucket);
        auto inside = [&](float v) {
            return in_buckets(v, from, end) && key_of(v) >= lo && key_of(v) <= hi;
        };
        for (;;) {
            const uint32_t n = gather(inside);
            if (rank == 0 && tid == 0) {
                S.cut.in = n;
                S.key_lo = 0xffffffffu;
                S.key_hi = 0;
            }
            told();
            if (cut.in <= kList)
                break;
            // too many: by the bits of their values
            counted = false;
            uint32_t a0 = 0xffffffffu, a1 = 0;
#pragma unroll 1
            for (int j = 0; j < J; ++j) {
                float v[VE];
                unpack(run[j * 32 + lane], v);
#pragma unroll
                for (int q = 0; q < VE; ++q)
                    if (inside(v[q])) {
                        a0 = min(a0, key_of(v[q]));
                        a1 = max(a1, key_of(v[q]));
                    }
            }
            a0 = __reduce_min_sync(0xffffffffu, a0);
            a1 = __reduce_max_sync(0xffffffffu, a1);
            if (lane == 0 && a0 <= a1) {
                min_dsmem_u32(dsmem_addr(&S.key_lo, 0), a0);
                max_dsmem_u32(dsmem_addr(&S.key_hi, 0), a1);
            }
            clear();
            all_ctas();
            if (rank == 0 && tid == 0) {
                S.cut.lo = S.key_lo;
                S.cut.hi = S.key_hi;
            }
            told();
            lo = cut.lo;
            hi = cut.hi;
            if (lo == hi) {  // one value alone
                if (rank == 0 && tid == 0) {
                    const float v = value_of(lo);
                    const uint64_t w = weights ? weight_of(S, v) : 0;
                    const int m = k ? static_cast<int>(k - cut.above)
                                    : static_cast<int>((target - cut.mass + w - 1) / w);
                    S.cut.tau = v;
                    S.cut.m = m;
                    S.cut.mass = cut.mass + w * m;
                }
                told();
                return;
            }
            int sh = 0;
            while ((hi - lo) >> sh >= kBuckets)
                ++sh;
            histogram(true, weights, [&](float v) {
                return inside(v) ? static_cast<int>((key_of(v) - lo) >> sh) : -1;
            });
            if (rank == 0)
                find(S, k, target, true);
            told();
            const uint32_t from = lo + (static_cast<uint32_t>(cut.bucket) << sh);
            hi = min(hi, from + ((1u << sh) - 1));
            lo = from;
        }
        if (rank == 0) {
            sort_falling(S.list, static_cast<int>(cut.in));
            cut_list(S, static_cast<int>(cut.in), k, target, weights);
        }
        told();
    };
    const bool few = top_k > 0 && top_k <= kList / 2 && top_k * 2 <= ctas * kSpThreads;
    bool listed = false;  // CTA 0's list holds all that may be kept
    if (few) {
        // the k-th largest of the threads' maxima: no fewer than k entries lie in its
        // bucket or above it
        if (my_top > -INFINITY)
            atomicAdd(&S.count[bucket_of(my_top)], 1u);
        gather_sums(S, ctas, rank, true, false);
        if (rank == 0) {
            if (tid == 0)
                S.cut = Cut{};
            __syncthreads();
            find(S, static_cast<uint32_t>(top_k), 0, false);
        }
        told();
        const float end = end_of(cut.bucket < 0 ? kBuckets - 1 : cut.bucket);
        finish(S, rank,
               static_cast<int>(gather([&](float v) { return in_buckets(v, 0.f, end); })), 0, token);
        told();
        listed = cut.done != 0;
        if (listed && a.tokens)
            return;
        if (!listed) {
            cut = Cut{};
            cut.tau = -INFINITY;
            cut.m = 0x7fffffff;
        }
    }
    if (!listed && top_k > 0)
        select(static_cast<uint32_t>(top_k), 0, by_mass, false);
    auto cluster_total = [&](uint64_t s) {  // of all threads' s; the warps' sums in S.runs
        s = warp_sum(s);
        if (lane < ctas)
            st_dsmem_u64(dsmem_addr(&S.runs[rank * kSpWarps + wi], lane), s);
        all_ctas();
        uint64_t total = 0;
        for (int r = lane; r < ctas * kSpWarps; r += 32)
            total += S.runs[r];
        return warp_sum(total);
    };
    if (!listed && by_mass) {
        uint64_t sum = cut.mass;
        if (top_k == 0) {  // of the whole row
            clear();
            uint64_t s = 0;
            // weights below half of (1 - top_p) / vocab are, together, less than what may be left
            // out: the cut lies above them
            const float low = 17592186044416.f * 0.5f * (1.f - fmaxf(top_p, 0.f)) /
                              static_cast<float>(a.vocab);
            const uint64_t least = max(static_cast<uint64_t>(low), uint64_t(1));
#pragma unroll 1
            for (int j = 0; j < J; ++j)
                each_weight(j, [&](float v, uint64_t w) {
                    s += w;
                    if (w >= least)
                        add_weight(bucket_of(v), w);
                });
            sum = cluster_total(s);
            gather_sums(S, ctas, rank, false, true);
            counted = true;
        }
        const uint64_t target = top_p > 0.f ? max(target_of(top_p, sum), uint64_t(1)) : 1;
        bool found = top_k == 0;
        if (found) {  // all down to the bucket of the cut, if that is not too much
            if (rank == 0) {
                if (tid == 0)
                    S.cut = Cut{};
                __syncthreads();
                find(S, 0, target, false);
            }
            told();
            const float end = end_of(cut.bucket);
            if (cut.in < kList * 9 / 10) {  // (a bucket's weights are within 9 %)
                finish(S, rank,
                       static_cast<int>(gather([&](float v) { return in_buckets(v, 0.f, end); })),
                       sum, token);
                told();
                listed = cut.done != 0;
                if (listed && a.tokens)
                    return;
                found = false;
            }
        }
        if (!listed)
            select(0, target, true, found);
    }
    const bool cuts = top_k > 0 || by_mass;
    const bool partial = cuts && cut.m < static_cast<int>(cut.in);

    // ----------------------------------------------------------- what is kept
    int ties_before = 0;  // entries equal to tau before this warp's run
    if (partial) {
        uint32_t n = 0;
#pragma unroll 1
        for (int j = 0; j < J; ++j) {
            float v[VE];
            unpack(run[j * 32 + lane], v);
#pragma unroll
            for (int k = 0; k < VE; ++k)
                n += v[k] == cut.tau;
        }
        n = warp_sum(n);
        if (lane < ctas)
            st_dsmem_u32(dsmem_addr(&S.ties[rank * kSpWarps + wi], lane), n);
        all_ctas();
        uint32_t t = 0;
        for (int r = lane; r < rank * kSpWarps + wi; r += 32)
            t += S.ties[r];
        ties_before = static_cast<int>(warp_sum(t));
    }
    const float from = fmaxf(cut.tau, least);  // the least value kept
    auto kept = [&](float v, int before) {
        return v >= from && (!partial || v != cut.tau || before < cut.m);
    };
    // Which of the lane's values of step j are kept, a bit each; `t` entries equal to tau come
    // before the step, and t moves on.
    auto step = [&](int j, int &t, float (&v)[VE]) {
        unpack(run[j * 32 + lane], v);
        int before = 0;
        if (partial) {
            int n = 0;
#pragma unroll
            for (int k = 0; k < VE; ++k)
                n += v[k] == cut.tau;
            const int upto = warp_incl(n, lane);
            before = t + upto - n;
            t += __shfl_sync(0xffffffffu, upto, 31);
        }
        unsigned mask = 0;
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            mask |= kept(v[k], before) ? 1u << k : 0u;
            before += v[k] == cut.tau;
        }
        return mask;
    };
    // The lane's kept weights of step j.
    auto step_sum = [&](int j, int &t) {
        float v[VE];
        const unsigned mask = step(j, t, v);
        uint64_t s = 0;
#pragma unroll
        for (int k = 0; k < VE; k += 2)
            if (mask >> k & 3) {
                uint64_t w0, w1;
                weights(S.table, c, M, v[k], v[k + 1], w0, w1);
                s += (mask >> k & 1 ? w0 : 0) + (mask >> k & 2 ? w1 : 0);
            }
        return s;
    };
    if (a.tokens) {
        uint64_t s = 0;
        int t = ties_before;
        if (!cuts && !(min_p > 0.f))
#pragma unroll 1
            for (int j = 0; j < J; ++j)
                each_weight(j, [&](float, uint64_t w) { s += w; });
        else {
            // few are kept: the values of kept ones side by side, 64 at a time
            float *line = reinterpret_cast<float *>(&S.part[0][0]) + wi * 96;
            static_assert(sizeof(S.part) >= kSpWarps * 96 * 4, "a line a warp");
            int n = 0;
            auto take = [&] {
                uint64_t w0, w1;
                __syncwarp();
                weights(S.table, c, M, lane < n ? line[lane] : -INFINITY,
                        lane + 32 < n ? line[lane + 32] : -INFINITY, w0, w1);
                s += w0 + w1;
                const float rest = line[lane + 64];
                __syncwarp();
                line[lane] = rest;
                __syncwarp();
                n -= 64;
            };
#pragma unroll 1
            for (int j = 0; j < J; ++j) {
                float v[VE];
                const unsigned mask = step(j, t, v);
#pragma unroll
                for (int k = 0; k < VE; ++k) {
                    const unsigned m = __ballot_sync(0xffffffffu, mask >> k & 1);
                    if (!m)
                        continue;
                    if (mask >> k & 1)
                        line[n + __popc(m & ((1u << lane) - 1))] = v[k];
                    n += __popc(m);
                    if (n >= 64)
                        take();
                }
            }
            take();
        }
        all_ctas();  // (S.runs may still be read)
        const uint64_t total = cluster_total(s);
        const uint64_t level = level_of(u, total);
        // the run that the level falls into: four runs a lane
        constexpr int RL = kSpCtas * kSpWarps / 32;
        const int runs = ctas * kSpWarps;
        uint64_t part[RL], local = 0;
#pragma unroll
        for (int k = 0; k < RL; ++k) {
            part[k] = lane * RL + k < runs ? S.runs[lane * RL + k] : 0;
            local += part[k];
        }
        uint64_t at = warp_incl(local, lane) - local, mine = 0;
        bool here = false;
#pragma unroll
        for (int k = 0; k < RL; ++k) {
            if (lane * RL + k == rank * kSpWarps + wi && at <= level && level < at + part[k]) {
                here = true;
                mine = at;
            }
            at += part[k];
        }
        const unsigned who = __ballot_sync(0xffffffffu, here);
        if (!who)
            return;
        at = __shfl_sync(0xffffffffu, mine, __ffs(who) - 1);
        t = ties_before;
#pragma unroll 1
        for (int j = 0; j < J; ++j) {
            int t0 = t;
            const uint64_t w = step_sum(j, t);
            const uint64_t upto = at + warp_incl(w, lane);
            const unsigned past = __ballot_sync(0xffffffffu, upto > level);
            if (!past) {
                at = __shfl_sync(0xffffffffu, upto, 31);
                continue;
            }
            float v[VE];
            const unsigned mask = step(j, t0, v);
            if (lane == __ffs(past) - 1) {
                uint64_t sum = upto - w;
                int tok = -1;
#pragma unroll
                for (int k = 0; k < VE; ++k)
                    if (tok < 0 && (mask >> k & 1)) {
                        sum += weight_of(S, v[k]);
                        if (sum > level)
                            tok = (g0 + j * 32 + lane) * VE + k - mis;
                    }
                a.tokens[i] = tok;
            }
            return;
        }
        return;
    }

    // 2^-y times a number near 1 for the low parts of y: an fp32 number's worth of a weight
    auto weight32 = [&](float v) {
        float h, l;
        gap(M, v, h, l);
        const float y = h * c.ch;
        const float e = fmaf(l, c.ch, fmaf(h, c.cl, fmaf(h, c.ch, -y)));
        return y < 150.f ? ex2_approx(-y) * fmaf(e, -0.693147182f, 1.f) : 0.f;
    };
    uint64_t total = cut.mass;
    if (!cuts || (!listed && (min_p > 0.f || !by_mass))) {
        // (the weights of a cut by sums are known, but for what min_p takes off)
        float s = 0.f;
        int t = ties_before;
#pragma unroll 1
        for (int j = 0; j < J; ++j) {
            float v[VE], p[VE];
            unpack(run[j * 32 + lane], v);
            int before = 0;
            if (partial) {
                int n = 0;
#pragma unroll
                for (int k = 0; k < VE; ++k)
                    n += v[k] == cut.tau;
                const int upto = warp_incl(n, lane);
                before = t + upto - n;
                t += __shfl_sync(0xffffffffu, upto, 31);
            }
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                p[k] = kept(v[k], before) ? weight32(v[k]) : 0.f;
                before += v[k] == cut.tau;
            }
#pragma unroll
            for (int k = 1; k < VE; k *= 2)
#pragma unroll
                for (int q = 0; q < VE; q += 2 * k)
                    p[q] += p[q + k];
            s += p[0];
        }
        all_ctas();  // (S.runs may still be read)
        total = cluster_total(__float2ull_rn(s * 17592186044416.f));
    }
    const float inv = 17592186044416.f / static_cast<float>(total);
    write_row([&](float v, int before) { return kept(v, before) ? weight32(v) * inv : 0.f; },
              partial, cut.tau, ties_before);
}

// Vectors a lane of a row's `ctas` CTAs, and their shared memory; T the logits' type.
template <class T>
static int steps_of(int vocab, int ctas)
{
    constexpr int VE = 16 / sizeof(T);
    return (vocab + 2 * VE - 2) / VE / (ctas * kSpThreads) + 1;
}
template <class T>
static size_t bytes_of(int vocab, int ctas)
{
    constexpr size_t kShared = (sizeof(SpShared) + 127) / 128 * 128;
    return kShared + static_cast<size_t>(steps_of<T>(vocab, ctas)) * kSpThreads * 16;
}

// Up to which a call has fewer CTAs a row than kSpCtas: two of them fit on an SM.
constexpr size_t kSpBytes = 112 * 1024;

template <class T>
static cudaError_t prepare_sample_t()
{
    const size_t most = std::max(kSpBytes, bytes_of<T>(kSampleMaxVocab, kSpCtas));
    return cudaFuncSetAttribute(zp_sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(most));
}

cudaError_t prepare_sample()
{
    const cudaError_t err = prepare_sample_t<float>();
    return err != cudaSuccess ? err : prepare_sample_t<__nv_bfloat16>();
}

template <class T>
static cudaError_t launch_sample_t(const SampleArgs &a, int sms, cudaStream_t s)
{
    // As many CTAs as the SMs hold at once, two each, up to eight a row and up to a vector a
    // lane; at least so many that two fit on an SM (96 rows of 50,257 bf16 logits with
    // filters of all kinds: 3 CTAs a row 56 us, 2 67)
    const int most = static_cast<int>(std::min<long long>(kSpCtas, std::max(1, 2 * sms / a.R)));
    int ctas = 1;
    while (ctas < kSpCtas && (bytes_of<T>(a.vocab, ctas) > kSpBytes || ctas < most) &&
           steps_of<T>(a.vocab, ctas) > 1)
        ++ctas;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.R) * static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(kSpThreads, 1, 1);
    cfg.dynamicSmemBytes = bytes_of<T>(a.vocab, ctas);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, zp_sample_kernel<T>, a, ctas, steps_of<T>(a.vocab, ctas));
}

cudaError_t launch_sample(const SampleArgs &a, bool bf16, int sms, cudaStream_t s)
{
    return bf16 ? launch_sample_t<__nv_bfloat16>(a, sms, s) : launch_sample_t<float>(a, sms, s);
}

}  // namespace zp
