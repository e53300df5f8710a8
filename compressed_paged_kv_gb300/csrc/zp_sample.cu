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
// in whatever order it is formed.
//
// One cluster of CTAs a row, which lies in their shared memory: it is read from memory
// once.  A thread owns a contiguous run of it, so that the threads' sums, scanned, say
// whose run a level falls into.  tau is found by a histogram over the gap to the maximum
// (counts, and weights where a sum is asked for): the bucket in which the count or the
// sum is reached is gathered and sorted; one of more than kList entries is cut up again by
// the bits of its values, until it fits or holds one value alone.
#include "zp_sample.cuh"

namespace zp {

namespace {

constexpr int kSpThreads = 512;
constexpr int kSpCtas = 8;       // of a cluster, at most: the portable most
constexpr int kBuckets = 2048;
constexpr int kList = 1024;
constexpr int kSpWarps = kSpThreads / 32;

__device__ const WeightTable d_table{};

// What CTA 0 finds out about a cut.
struct Cut {
    uint64_t mass;    // weights above the bucket, then of the whole kept set
    uint32_t above;   // entries above the bucket
    uint32_t in;      // and in it; at the end, those equal to tau
    uint32_t lo, hi;  // the keys of a cut bucket
    int bucket;       // of the first histogram
    int m;            // of those equal to tau, the ones kept
    float tau;
};

struct SpShared {
    uint64_t bar;
    uint64_t mass[kBuckets];
    uint64_t list[kList];
    uint64_t table[1024];
    uint32_t count[kBuckets];
    uint64_t sums[kSpCtas];      // of the CTAs
    uint64_t scan64[kSpWarps + 1];
    float2 ends[kSpCtas];        // the CTAs' (largest, smallest finite)
    uint32_t scan32[kSpWarps + 1];
    uint32_t ties[kSpCtas];
    uint32_t key_lo, key_hi, listed, equal, equal_upto;
    Cut cut;      // CTA 0's
    Cut told[2];  // what it told all, the last two times
};

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
__device__ __forceinline__ uint32_t add_dsmem_u32(uint32_t addr, uint32_t v)
{
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
                 : "=r"(old)
                 : "r"(addr), "r"(v)
                 : "memory");
    return old;
}
__device__ __forceinline__ void min_dsmem_u32(uint32_t addr, uint32_t v)
{
    asm volatile("red.shared::cluster.min.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void max_dsmem_u32(uint32_t addr, uint32_t v)
{
    asm volatile("red.shared::cluster.max.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
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
__device__ __forceinline__ uint64_t target_of(float p, uint64_t s)
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

}  // namespace

// `per` elements a thread; T the logits' type.
template <class T>
__global__ void __launch_bounds__(kSpThreads, 2)
    zp_sample_kernel(const __grid_constant__ SampleArgs a, int ctas, int per)
{
    constexpr int VE = 16 / sizeof(T);
    extern __shared__ __align__(128) uint8_t raw[];
    SpShared &S = *reinterpret_cast<SpShared *>(raw);
    T *x = reinterpret_cast<T *>(raw + (sizeof(SpShared) + 127) / 128 * 128);
    const int tid = threadIdx.x, lane = tid & 31, wi = tid >> 5;
    const int rank = static_cast<int>(cluster_ctarank());
    const int i = blockIdx.x / ctas;
    const int seg = per * kSpThreads;
    if (tid == 0) {
        mbar_init(&S.bar, 1);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();

    // the row as slots from the 16-byte boundary at or below its first element: it
    // fills slots mis .. mis + vocab - 1, this CTA holds `seg` from `s0` on
    const T *row = static_cast<const T *>(a.logits) + i * a.stride;
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
    const int s0 = rank * seg;
    const int lo = mis ? VE : 0, hi = (mis + a.vocab) / VE * VE;  // whole vectors
    const int c0 = max(s0, lo), c1 = min(s0 + seg, hi);
    if (tid == 0 && c1 > c0) {
        mbar_arrive_expect_tx(&S.bar, static_cast<uint32_t>((c1 - c0) * sizeof(T)));
        bulk_g2s(x + (c0 - s0), row + (c0 - mis), static_cast<uint32_t>((c1 - c0) * sizeof(T)),
                 &S.bar);
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
    if (top_k < 0 || top_k >= a.vocab)
        top_k = 0;
    WeightScale c;
    float gap_h, gap_l;  // the largest gap to the maximum that min_p allows
    {
        const double s = fmin(1.4426950408889634 / static_cast<double>(temp), 1.2e30);
        c.ch = static_cast<float>(s);
        c.cl = static_cast<float>(s - static_cast<double>(c.ch));
        gap_h = INFINITY;
        gap_l = 0.f;
        if (min_p > 0.f) {
            const double g = -static_cast<double>(temp) * log(fmin(static_cast<double>(min_p), 1.0));
            gap_h = static_cast<float>(g);
            gap_l = static_cast<float>(g - static_cast<double>(gap_h));
        }
    }
    for (int k = tid; k < 1024; k += kSpThreads)
        S.table[k] = d_table.v[k];
    for (int s = tid; s < seg; s += kSpThreads)
        if (s0 + s < c0 || s0 + s >= c1) {
            const int e = s0 + s - mis;
            x[s] = e >= 0 && e < a.vocab ? row[e] : static_cast<T>(-INFINITY);
        }
    if (c1 > c0 && !mbar_wait(&S.bar, 0))
        set_error(a.sticky, ZP_ERR_TIMEOUT);
    __syncthreads();
    cluster_arrive();  // the other CTAs have started once it is waited for

    // the largest logit and the smallest finite one; NaN becomes -infinity
    T *mine = x + tid * per;
    float top = -INFINITY, bottom = INFINITY;
    for (int k = 0; k < per; ++k) {
        const float v = to_f32(mine[k]);
        if (v != v)
            mine[k] = static_cast<T>(-INFINITY);
        top = fmaxf(top, v);
        bottom = fminf(bottom, v > -INFINITY ? v : INFINITY);
    }
    top = value_of(__reduce_max_sync(0xffffffffu, key_of(top)));
    bottom = value_of(__reduce_min_sync(0xffffffffu, key_of(bottom)));
    float2 *warp_ends = reinterpret_cast<float2 *>(S.scan64);
    if (lane == 0)
        warp_ends[wi] = make_float2(top, bottom);
    __syncthreads();
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
    const bool none = M == -INFINITY;
    if (!ok || none) {  // the whole cluster alike
        if (rank == 0 && tid == 0) {
            set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
            if (a.tokens)
                a.tokens[i] = -1;
        }
        for (int s = tid; s < seg && a.probs; s += kSpThreads) {
            const int e = s0 + s - mis;
            if (e < 0 || e >= a.vocab)
                continue;
            if (a.prob_bf16)
                static_cast<__nv_bfloat16 *>(a.probs)[i * a.prob_stride + e] =
                    __float2bfloat16_rn(0.f);
            else
                static_cast<float *>(a.probs)[i * a.prob_stride + e] = 0.f;
        }
        all_ctas();
        return;
    }
    auto weight_of = [&](float v) {
        float h, l;
        gap(M, v, h, l);
        return weight(S.table, c, h, l);
    };

    // ---------------------------------------------------------------- the cut
    Cut cut{};
    cut.tau = -INFINITY;
    cut.m = 0x7fffffff;
    const float range = fminf(64.f / c.ch, M - bottom);
    const float per_gap = range > 0.f ? kBuckets / range : 0.f;
    auto bucket_of = [&](float v) {  // falls with v
        const float b = v == M ? 0.f : (M - v) * per_gap;
        return min(kBuckets - 1, static_cast<int>(b));
    };
    // Every entry of the histogram's range is counted under `place` (below 0: not at
    // all), CTA 0 sums up, and finds the bucket in which the target is reached, with
    // `above` entries and `mass` above the first.
    auto histogram = [&](bool weights, auto place) {
        for (int b = tid; b < kBuckets; b += kSpThreads) {
            S.count[b] = 0;
            S.mass[b] = 0;
        }
        __syncthreads();
        for (int k = 0; k < per; ++k) {
            const float v = to_f32(mine[k]);
            const int b = v > -INFINITY ? place(v) : -1;
            if (b < 0)
                continue;
            atomicAdd(&S.count[b], 1u);
            if (weights)
                atomicAdd(reinterpret_cast<unsigned long long *>(&S.mass[b]),
                          static_cast<unsigned long long>(weight_of(v)));
        }
        all_ctas();
        if (rank == 0)
            for (int b = tid; b < kBuckets; b += kSpThreads) {
                uint32_t n = S.count[b];
                uint64_t w = S.mass[b];
                for (int r = 1; r < ctas; ++r) {
                    uint32_t y;
                    asm volatile("ld.shared::cluster.u32 %0, [%1];"
                                 : "=r"(y)
                                 : "r"(dsmem_addr(&S.count[b], r))
                                 : "memory");
                    n += y;
                    if (weights)
                        w += ld_dsmem_u64(dsmem_addr(&S.mass[b], r));
                }
                S.count[b] = n;
                S.mass[b] = w;
            }
    };
    // CTA 0 alone: the bucket where `above` + counts reach `k`, or `mass` + weights reach
    // `target` (k = 0), from the largest values on, which the last buckets of a `rising`
    // histogram hold and the first of the other.
    auto find = [&](uint32_t k, uint64_t target, bool rising) {
        constexpr int PB = kBuckets / kSpThreads;
        __syncthreads();
        uint32_t n = 0, all_n;
        uint64_t w = 0, all_w;
#pragma unroll
        for (int j = 0; j < PB; ++j) {
            const int b = rising ? kBuckets - 1 - (tid * PB + j) : tid * PB + j;
            n += S.count[b];
            w += S.mass[b];
        }
        uint32_t n0 = S.cut.above + block_before(n, S.scan32, all_n);
        uint64_t w0 = S.cut.mass + block_before(w, S.scan64, all_w);
        __syncthreads();  // S.cut is read
        if (tid == 0 && k > all_n && !rising) {  // fewer entries above -infinity: all of them
            S.cut.mass = all_w;
            S.cut.bucket = -1;
            S.cut.tau = -INFINITY;
            S.cut.m = 0x7fffffff;
        }
        for (int j = 0; j < PB; ++j) {
            const int b = rising ? kBuckets - 1 - (tid * PB + j) : tid * PB + j;
            const uint32_t nb = S.count[b];
            const uint64_t wb = S.mass[b];
            const bool here = k ? n0 < k && n0 + nb >= k : w0 < target && w0 + wb >= target;
            if (here) {
                S.cut.above = n0;
                S.cut.mass = w0;
                S.cut.in = nb;
                S.cut.bucket = b;
            }
            n0 += nb;
            w0 += wb;
        }
        __syncthreads();
    };
    int turn = 0;
    auto tell = [&] {  // CTA 0's cut to all: into two places in turn, as a CTA may still
                       // read the one before
        turn ^= 1;
        if (rank == 0) {
            __syncthreads();
            constexpr int W = sizeof(Cut) / 4;
            for (int k = tid; k < W * ctas; k += kSpThreads)
                st_dsmem_u32(
                    dsmem_addr(reinterpret_cast<uint32_t *>(&S.told[turn]) + k % W, k / W),
                    reinterpret_cast<const uint32_t *>(&S.cut)[k % W]);
        }
        all_ctas();
        cut = S.told[turn];
    };
    bool counted = false;  // CTA 0 holds the first histogram's sums
    // The cut where the count reaches k, or (k = 0) the weights reach `target`.
    auto select = [&](uint32_t k, uint64_t target, bool weights) {
        if (!counted)
            histogram(weights, bucket_of);
        counted = true;
        if (rank == 0) {
            __syncthreads();
            if (tid == 0)
                S.cut = Cut{};
            find(k, target, false);
        }
        tell();
        const int bucket = cut.bucket;
        if (bucket < 0)
            return;
        uint32_t lo = 0, hi = 0xffffffffu;
        auto inside = [&](float v) {
            const uint32_t key = key_of(v);
            return v > -INFINITY && bucket_of(v) == bucket && key >= lo && key <= hi;
        };
        bool one = false;  // one value alone is left
        while (cut.in > kList && !one) {
            counted = false;
            if (rank == 0 && tid == 0) {
                S.key_lo = 0xffffffffu;
                S.key_hi = 0;
            }
            all_ctas();
            uint32_t a0 = 0xffffffffu, a1 = 0;
            for (int j = 0; j < per; ++j) {
                const float v = to_f32(mine[j]);
                if (inside(v)) {
                    a0 = min(a0, key_of(v));
                    a1 = max(a1, key_of(v));
                }
            }
            a0 = __reduce_min_sync(0xffffffffu, a0);
            a1 = __reduce_max_sync(0xffffffffu, a1);
            if (lane == 0 && a0 <= a1) {
                min_dsmem_u32(dsmem_addr(&S.key_lo, 0), a0);
                max_dsmem_u32(dsmem_addr(&S.key_hi, 0), a1);
            }
            all_ctas();
            if (rank == 0 && tid == 0) {
                S.cut.lo = S.key_lo;
                S.cut.hi = S.key_hi;
            }
            tell();
            lo = cut.lo;
            hi = cut.hi;
            one = lo == hi;
            if (one)
                break;
            int sh = 0;
            while ((hi - lo) >> sh >= kBuckets)
                ++sh;
            histogram(weights, [&](float v) {
                return inside(v) ? static_cast<int>((key_of(v) - lo) >> sh) : -1;
            });
            if (rank == 0)
                find(k, target, true);
            tell();
            const uint32_t from = lo + (static_cast<uint32_t>(cut.bucket) << sh);
            hi = min(hi, from + ((1u << sh) - 1));
            lo = from;
        }
        if (one) {
            if (rank == 0 && tid == 0) {
                const float v = value_of(lo);
                const uint64_t w = weights ? weight_of(v) : 0;
                const int m = k ? static_cast<int>(k - cut.above)
                                : static_cast<int>((target - cut.mass + w - 1) / w);
                S.cut.tau = v;
                S.cut.m = m;
                S.cut.mass = cut.mass + w * m;
            }
            tell();
            return;
        }
        if (rank == 0 && tid == 0)
            S.listed = 0;
        all_ctas();
        for (int j = 0; j < per; ++j) {
            const float v = to_f32(mine[j]);
            if (inside(v)) {
                const uint32_t at = add_dsmem_u32(dsmem_addr(&S.listed, 0), 1);
                if (at < kList)
                    st_dsmem_u64(dsmem_addr(&S.list[at], 0),
                                 static_cast<uint64_t>(key_of(v)) << 32 |
                                     (0xffffffffu - static_cast<uint32_t>(s0 + tid * per + j)));
            }
        }
        all_ctas();
        if (rank == 0) {
            // falling by value, then rising by index
            const int n = min(static_cast<int>(S.listed), kList);
            int size = 2;
            while (size < n)
                size *= 2;
            for (int j = n + tid; j < size; j += kSpThreads)
                S.list[j] = 0;
            for (int span = 2; span <= size; span *= 2)
                for (int d = span / 2; d; d /= 2) {
                    __syncthreads();
                    for (int t = tid; t < size / 2; t += kSpThreads) {
                        const int p = 2 * t - (t & (d - 1)), q = p + d;
                        const bool falling = (p & span) == 0;
                        const uint64_t v = S.list[p], w = S.list[q];
                        if ((v < w) == falling) {
                            S.list[p] = w;
                            S.list[q] = v;
                        }
                    }
                }
            if (tid == 0)
                S.equal = S.equal_upto = 0;
            __syncthreads();
            // two entries a thread, and the sums before them
            constexpr int PL = kList / kSpThreads;
            uint64_t w[PL], sum = 0, all;
#pragma unroll
            for (int j = 0; j < PL; ++j) {
                const int p = tid * PL + j;
                w[j] = weights && p < n
                           ? weight_of(value_of(static_cast<uint32_t>(S.list[p] >> 32)))
                           : 0;
                sum += w[j];
            }
            uint64_t at = cut.mass + block_before(sum, S.scan64, all);
#pragma unroll
            for (int j = 0; j < PL; ++j) {
                const int p = tid * PL + j;
                const bool here = p < n && (k ? cut.above + p + 1 == k
                                              : at < target && at + w[j] >= target);
                at += w[j];
                if (here) {
                    S.cut.tau = value_of(static_cast<uint32_t>(S.list[p] >> 32));
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
        }
        tell();
    };
    const bool by_mass = top_p < 1.f;
    if (top_k > 0)
        select(static_cast<uint32_t>(top_k), 0, by_mass);
    if (by_mass) {
        uint64_t sum = cut.mass;
        if (top_k == 0) {  // of the whole row
            uint64_t s = 0, all;
            for (int k = 0; k < per; ++k)
                s += weight_of(to_f32(mine[k]));
            block_before(s, S.scan64, all);
            if (tid < ctas)
                st_dsmem_u64(dsmem_addr(&S.sums[rank], tid), all);
            all_ctas();
            sum = 0;
            for (int r = 0; r < ctas; ++r)
                sum += S.sums[r];
        }
        const uint64_t target = top_p > 0.f ? max(target_of(top_p, sum), uint64_t(1)) : 1;
        select(0, target, true);
    }
    const bool partial = (top_k > 0 || by_mass) && cut.m < static_cast<int>(cut.in);

    // ----------------------------------------------------------- what is kept
    auto within = [&](float v) {  // min_p's part
        float h, l;
        gap(M, v, h, l);
        return h < gap_h || (h == gap_h && l <= gap_l);
    };
    const int slot0 = s0 + tid * per;  // this thread's first
    int ties_before = 0;               // entries equal to tau before it
    if (partial) {
        uint32_t n = 0, all;
        for (int k = 0; k < per; ++k)
            n += to_f32(mine[k]) == cut.tau;
        ties_before = static_cast<int>(block_before(n, S.scan32, all));
        if (tid < ctas)
            st_dsmem_u32(dsmem_addr(&S.ties[rank], tid), all);
        all_ctas();
        for (int r = 0; r < rank; ++r)
            ties_before += static_cast<int>(S.ties[r]);
    }
    uint64_t sum = 0, all, total = 0, before;
    {
        int t = ties_before;
        for (int k = 0; k < per; ++k) {
            const float v = to_f32(mine[k]);
            const bool tie = v == cut.tau;
            if ((v > cut.tau || (tie && t < cut.m)) && within(v))
                sum += weight_of(v);
            t += tie && partial;
        }
    }
    before = block_before(sum, S.scan64, all);
    __syncthreads();
    if (tid < ctas)
        st_dsmem_u64(dsmem_addr(&S.sums[rank], tid), all);
    all_ctas();
    for (int r = 0; r < ctas; ++r) {
        before += r < rank ? S.sums[r] : 0;
        total += S.sums[r];
    }
    if (a.tokens) {
        // the thread whose run the level falls into; its warp looks through the run
        const uint64_t level = u >= 1.f ? total - 1 : u > 0.f ? part_of(u, total) : 0;
        const unsigned who = __ballot_sync(0xffffffffu, before <= level && level < before + sum);
        if (who == 0)
            return;
        const int src = __ffs(who) - 1;
        uint64_t at = __shfl_sync(0xffffffffu, before, src);
        int t = __shfl_sync(0xffffffffu, ties_before, src);
        const int first = __shfl_sync(0xffffffffu, slot0, src);
        for (int k0 = 0; k0 < per; k0 += 32) {
            const float v = k0 + lane < per ? to_f32(x[first - s0 + k0 + lane]) : -INFINITY;
            const bool tie = v == cut.tau;
            const unsigned same = __ballot_sync(0xffffffffu, tie);
            const int my_t = t + __popc(same & ((1u << lane) - 1));
            uint64_t w = 0;
            if ((v > cut.tau || (tie && (!partial || my_t < cut.m))) && within(v))
                w = weight_of(v);
            const uint64_t upto = at + warp_incl(w, lane);
            const unsigned past = __ballot_sync(0xffffffffu, upto > level);
            if (past) {
                if (lane == __ffs(past) - 1)
                    a.tokens[i] = first + k0 + lane - mis;
                return;
            }
            at = __shfl_sync(0xffffffffu, upto, 31);
            t += __popc(same);
        }
        return;
    }

    // the probabilities: a warp's runs lie one behind the other
    const float inv = static_cast<float>(17592186044416.0 / static_cast<double>(total));
    const int w0 = (tid - lane) * per;
    int t = __shfl_sync(0xffffffffu, ties_before, 0);
    for (int k0 = 0; k0 < 32 * per; k0 += 32) {
        const int s = w0 + k0 + lane;
        const float v = to_f32(x[s]);
        const bool tie = v == cut.tau;
        int my_t = t;
        if (partial) {
            const unsigned same = __ballot_sync(0xffffffffu, tie);
            my_t += __popc(same & ((1u << lane) - 1));
            t += __popc(same);
        }
        float p = 0.f;
        if ((v > cut.tau || (tie && (!partial || my_t < cut.m))) && within(v)) {
            float h, l;
            gap(M, v, h, l);
            const float y = h * c.ch;
            const float e = fmaf(l, c.ch, fmaf(h, c.cl, fmaf(h, c.ch, -y)));
            p = y < 150.f ? ex2_approx(-y) * fmaf(e, -0.693147182f, 1.f) * inv : 0.f;
        }
        const int e = s0 + s - mis;
        if (e < 0 || e >= a.vocab)
            continue;
        if (a.prob_bf16)
            static_cast<__nv_bfloat16 *>(a.probs)[i * a.prob_stride + e] = __float2bfloat16_rn(p);
        else
            static_cast<float *>(a.probs)[i * a.prob_stride + e] = p;
    }
}

template <class T>
static cudaError_t launch_sample_t(const SampleArgs &a, int sms, cudaStream_t s)
{
    constexpr size_t kShared = (sizeof(SpShared) + 127) / 128 * 128;
    constexpr int WORD = 4 / sizeof(T);  // elements a word: a thread's run is an odd number of words
    auto per_of = [&](int ctas) {
        const int slots = a.vocab + 16 / static_cast<int>(sizeof(T)) - 1;
        const int words = (slots + ctas * kSpThreads * WORD - 1) / (ctas * kSpThreads * WORD);
        return (words | 1) * WORD;
    };
    auto bytes_of = [&](int ctas) { return kShared + per_of(ctas) * kSpThreads * sizeof(T); };
    int ctas = 1;
    while (ctas < kSpCtas && (bytes_of(ctas) > 110 * 1024 || a.R * 2ll * ctas <= 2ll * sms) &&
           per_of(ctas) > 4 * WORD)
        ctas *= 2;
    const size_t bytes = bytes_of(ctas);
    cudaError_t err = cudaFuncSetAttribute(zp_sample_kernel<T>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(bytes));
    if (err != cudaSuccess)
        return err;
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
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, zp_sample_kernel<T>, a, ctas, per_of(ctas));
}

cudaError_t launch_sample(const SampleArgs &a, bool bf16, int sms, cudaStream_t s)
{
    return bf16 ? launch_sample_t<__nv_bfloat16>(a, sms, s) : launch_sample_t<float>(a, sms, s);
}

}  // namespace zp
