// zp_fp8_append.cu -- new tokens' keys and values rounded into an 8-bit cache:
// zp_append_kv and zp_append_kv_chunk of such a cache.
//
// The new tokens of a request that fall into one block are a group.  Per kv head, K and
// V apart, with A the largest magnitude of the group's rows (NaN not counted):
//     S' = the least power of two, 2^-32 .. 2^32, with A / S' <= 448
//     S  = S' if the group begins at slot 0, else max(S', the block's scale)
//     number = x / S, to the nearest e4m3 number, ties to even
// and where S is above the block's scale, the numbers that the slots before the group
// hold are rounded again to number * (scale / S).  A division by a power of two is
// exact, so a number is rounded once for the group it came with, and again
// only below 2^-6 (where e4m3 has fewer bits).
//
// One warp a (group, kv head): the group's rows of K and of V stay in registers between
// the maximum and the rounding, so that each is read once.  Work is found from the packed
// tokens: a warp looks at `span` of them and takes the groups whose first token is among
// them.
//
// Measured, 8 heads of 128: 16 prompts, 34.9 K tokens, 0.19 GB (16 bits read, 8 written and read
// back where a block is shared out) in 33 us = 5.8 TB/s, 0.85 of the copy peak; one token each of
// 256 requests 4.6 us, the chain offsets -> block id -> scale -> rows.
#include "zp_fp8.cuh"

namespace zp {

namespace {

constexpr int kF8Threads = 128;
constexpr int kVec = 8;  // 16-byte vectors of new rows a lane holds: 16 rows of 128

struct Group {
    int t0;     // packed row of its first token
    int cnt;    // its tokens
    int slot;   // of the first
    int blk;    // < 0: none
};

// The last i in [0, R) with starts[i] <= t, or 0 (the caller checks that the chunk
// holds t).
__device__ __forceinline__ int request_of(const int32_t *starts, int R, long long t)
{
    int lo = 0, hi = R;
    while (hi - lo > 1) {
        const int m = (lo + hi) / 2;
        if (starts[m] <= t)
            lo = m;
        else
            hi = m;
    }
    return lo;
}

// The same as a warp: every round the 32 lanes probe the range at equal steps.
__device__ __forceinline__ int warp_request_of(const int32_t *starts, int R, long long t, int lane)
{
    int lo = 0, n = R;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool le = lane * step < n && starts[i] <= t;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int k = m ? 31 - __clz(m) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// The group that begins with packed token t, if one does.
__device__ __forceinline__ Group group_at(const Fp8KvArgs &a, int i, long long t, bool report)
{
    Group g{static_cast<int>(t), 0, 0, -1};
    int p, n_left, row;
    if (a.starts) {
        ChunkReq c;
        bool bad;
        if (!chunk_request(a, i, c, &bad) || t < c.first || t >= c.first + c.n)
            return g;  // a bad request, or a row of no request: padding
        const int j = static_cast<int>(t - c.first);
        p = c.len - c.n + j;
        if (j > 0 && p % kBlk != 0)
            return g;
        n_left = c.n - j;
        row = c.row;
    } else {
        row = a.req_idx ? a.req_idx[i] : i;
        const bool fits = row >= 0 && row < a.num_rows;
        p = fits ? a.lengths[row] - 1 : -1;
        if (p < 0 || p >= a.stride * kBlk) {
            if (report)
                set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
            return g;
        }
        n_left = 1;
    }
    const int blk = a.tables[static_cast<size_t>(row) * a.stride + p / kBlk];
    if (blk < 0 || blk >= a.num_blocks) {
        if (report)
            set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
        return g;
    }
    g.slot = p % kBlk;
    g.cnt = min(kBlk - g.slot, n_left);
    g.blk = blk;
    return g;
}

// One pool's rows of a group and kv head.
template <int D>
struct Rows {
    static constexpr int VPR = D / 8;  // 16-byte vectors of a new row
    uint4 v[kVec];

    __device__ __forceinline__ void load(const __nv_bfloat16 *src, int64_t stride, int cnt, int lane)
    {
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            const int x = k * 32 + lane, r = x / VPR;
            v[k] = make_uint4(0u, 0u, 0u, 0u);
            if (r < cnt)
                v[k] = ld_global_nc_v4(src + r * stride + x % VPR * 8);
        }
    }

    // The bits of the largest magnitude.
    __device__ __forceinline__ uint32_t most() const
    {
        __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)  // (a NaN gives the other operand)
                m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i])));
        }
        return __reduce_max_sync(0xffffffffu,
                                 __float_as_uint(fmaxf(__low2float(m), __high2float(m))));
    }

    __device__ __forceinline__ void store(uint8_t *slab, float *scale, const Group &g, int lane)
    {
        uint32_t e = exp2_bits(fp8_scale_exp(most()));
        bool write = true;
        if (g.slot > 0) {
            const float before = *scale, s = fmaxf(__uint_as_float(e), before);
            if (before < s) {  // the older rows, to the larger scale
                const float f = before / s;
                for (int x = lane; x < g.slot * (D / 4); x += 32) {
                    uint32_t *at = reinterpret_cast<uint32_t *>(slab) + x;
                    const uint32_t w = *at, lo = f16x2_of_e4m3(w), hi = f16x2_of_e4m3(w >> 16);
                    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
                    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                    *at = e4m3x2(a.x * f, a.y * f) | e4m3x2(b.x * f, b.y * f) << 16;
                }
            }
            write = !(before >= s);
            e = __float_as_uint(s);
            __syncwarp();  // every lane has read the scale
        }
        if (lane == 0 && write)
            *scale = __uint_as_float(e);
        const float inv = 1.f / __uint_as_float(e);
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            const int x = k * 32 + lane, r = x / VPR;
            if (r >= g.cnt)
                continue;
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[i] = e4m3x2(__uint_as_float(w[i] << 16) * inv,
                              __uint_as_float(w[i] & 0xffff0000u) * inv);
            *reinterpret_cast<uint2 *>(slab + (g.slot + r) * D + x % VPR * 8) =
                make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
        }
    }
};

// SPAN packed tokens a warp: 1 or 16.
template <int D, int SPAN>
__global__ void __launch_bounds__(kF8Threads) zp_fp8_append_kernel(const Fp8KvArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    if (a.starts)  // every request is checked once, whether or not a token finds it
        for (long long i = blockIdx.x * static_cast<long long>(kF8Threads) + threadIdx.x; i < a.R;
             i += static_cast<long long>(gridDim.x) * kF8Threads) {
            ChunkReq c;
            bool bad;
            chunk_request(a, static_cast<int>(i), c, &bad);
            if (bad)
                set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
        }
    const long long warp =
        blockIdx.x * static_cast<long long>(kF8Threads / 32) + static_cast<int>(threadIdx.x >> 5);
    const int h = static_cast<int>(warp % a.Hkv);
    const long long base = warp / a.Hkv * SPAN;
    if (base >= a.total)
        return;
    Group mine{0, 0, 0, -1};
    if (SPAN == 1) {
        const int i = a.starts ? warp_request_of(a.starts, a.R, base, lane) : static_cast<int>(base);
        mine = group_at(a, i, base, h == 0 && lane == 0);
    } else if (lane < SPAN && base + lane < a.total) {
        const long long t = base + lane;
        mine = group_at(a, request_of(a.starts, a.R, t), t, h == 0);
    }
    unsigned todo = SPAN == 1 ? static_cast<unsigned>(mine.blk >= 0)
                              : __ballot_sync(0xffffffffu, mine.blk >= 0);
    for (; todo; todo &= todo - 1) {
        Group g = mine;
        if (SPAN > 1) {
            const int l = __ffs(todo) - 1;
            g.t0 = __shfl_sync(0xffffffffu, mine.t0, l);
            g.cnt = __shfl_sync(0xffffffffu, mine.cnt, l);
            g.slot = __shfl_sync(0xffffffffu, mine.slot, l);
            g.blk = __shfl_sync(0xffffffffu, mine.blk, l);
        }
        const size_t slab = static_cast<size_t>(g.blk) * a.Hkv + h;
        Rows<D> k, v;
        k.load(a.k_new + g.t0 * a.k_stride + h * D, a.k_stride, g.cnt, lane);
        v.load(a.v_new + g.t0 * a.v_stride + h * D, a.v_stride, g.cnt, lane);
        k.store(a.kpool + slab * (kBlk * D), a.kscale + slab, g, lane);
        v.store(a.vpool + slab * (kBlk * D), a.vscale + slab, g, lane);
    }
}

template <int D, int SPAN>
cudaError_t launch_t(const Fp8KvArgs &a, cudaStream_t s)
{
    const long long warps = (a.total + SPAN - 1ll) / SPAN * a.Hkv;
    const long long ctas = (warps * 32 + kF8Threads - 1) / kF8Threads;
    if (ctas > 0x7fffffffll)
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(kF8Threads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, zp_fp8_append_kernel<D, SPAN>, a);
}

}  // namespace

cudaError_t launch_fp8_append(const Fp8KvArgs &a, cudaStream_t s)
{
    const bool wide = a.starts && a.total >= 8ll * a.R;
    if (a.d == 64)
        return wide ? launch_t<64, 16>(a, s) : launch_t<64, 1>(a, s);
    if (a.d == 128)
        return wide ? launch_t<128, 16>(a, s) : launch_t<128, 1>(a, s);
    return cudaErrorInvalidValue;
}

}  // namespace zp
