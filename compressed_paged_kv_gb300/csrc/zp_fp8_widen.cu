// zp_fp8_widen.cu -- blocks of an 8-bit cache as bf16, for the attention of long chunks.
//
// The chunk kernel over an 8-bit cache makes fp16 tiles of V as it goes, once for every 256
// query rows.  A request with many of them has its tiles made over and over, and the tensor
// cores wait.  So the blocks of such requests are widened once: value = scale * number, exact
// in bf16 (three bits of mantissa, scales powers of two), into a workspace of the handle, one
// request behind the other, and their attention is the bf16 kernel's over that.
//
// Every CTA goes through the requests and keeps those that are widened, in their order, as
// long as they fit (the others are left to the 8-bit kernel); then the CTAs take the blocks
// in turn, 16 bytes a thread at a time.  Bound by HBM: one byte read and two written an element.
//
// Measured, with the bf16 kernel behind it against the 8-bit kernel alone: 2,048 tokens over 30,001,
// 32 heads of 128 over 8, 687 us and 879; 16 prompts of 331 to 4,007, 28 heads of 64 over 4, 467 and
// 644.  Of a bf16 cache the first takes 645.  This kernel alone, from cold caches: 39 us (4.7 TB/s) and
// 16.7 (with eight vectors a thread on their way and four CTAs an SM 40 and 18.4).
#include "zp_fp8.cuh"

namespace zp {

namespace {

constexpr int kWdThreads = 256;
constexpr int kWdMost = 1024;  // requests kept
constexpr int kWdLoads = 4;    // vectors a thread has on their way

}  // namespace

int fp8_wide_blocks(int num_blocks, int hkv, int d)
{
    const size_t most = kWideBytes / (static_cast<size_t>(hkv) * kBlk * d * 4);
    const size_t n = most < static_cast<size_t>(num_blocks) ? most : num_blocks;
    return n < 1 ? 1 : static_cast<int>(n);
}

__global__ void __launch_bounds__(kWdThreads) zp_fp8_widen_kernel(const Fp8WidenArgs a)
{
    __shared__ int s_scan[kWdThreads / 32 + 1];
    __shared__ int s_row[kWdMost], s_end[kWdMost];  // of the kept: table row, end of its blocks
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    long long used = 0;
    int kept = 0;
    for (int i0 = 0; i0 < a.R; i0 += kWdThreads) {
        const int i = i0 + tid;
        ChunkReq c;
        bool bad = false;
        const bool wide = i < a.R && chunk_request(a, i, c, &bad) && c.n >= a.least;
        // what does not fit into the workspace by itself takes no room
        const int need = wide && (c.len + kBlk - 1) / kBlk <= a.capacity ? (c.len + kBlk - 1) / kBlk : 0;
        int total, count;
        // (sums of 256 needs of at most the capacity, in units that fit: capacities are
        // below 2^22 blocks)
        const int before = block_excl_scan<kWdThreads>(need, s_scan, total);
        const bool fits = need > 0 && used + before + need <= a.capacity;
        const int nth = block_excl_scan<kWdThreads>(fits, s_scan, count);
        const bool mine = fits && kept + nth < kWdMost;
        if (mine) {
            s_row[kept + nth] = c.row;
            s_end[kept + nth] = static_cast<int>(used) + before + need;
        }
        if (blockIdx.x == 0 && i < a.R)
            a.places[i] = mine ? static_cast<int>(used) + before : -1;
        used += total;
        kept = min(kept + count, kWdMost);
    }
    __syncthreads();
    const int vpb = a.Hkv * kBlk * a.d / 16;  // vectors of a block
    for (int q = 0, x = blockIdx.x; q < kept; ++q) {
        // (a request that did not fit leaves a gap before the next one: its blocks are skipped)
        const int row = s_row[q], end = s_end[q];
        const int len = a.lengths[row], first = end - (len + kBlk - 1) / kBlk;
        while (x < first)
            x += gridDim.x;
        for (; x < end; x += gridDim.x) {
            const int blk = a.tables[static_cast<size_t>(row) * a.stride + (x - first)];
            if (blk < 0 || blk >= a.num_blocks) {
                if (tid == 0)
                    set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
                continue;
            }
            const uint8_t *kv[2] = {a.kpool, a.vpool};
            for (int v0 = 0; v0 < vpb; v0 += kWdLoads / 2 * kWdThreads) {
                uint4 u[kWdLoads];  // K's and V's
                float s[kWdLoads];
#pragma unroll
                for (int k = 0; k < kWdLoads; ++k) {
                    const int v = min(v0 + k / 2 * kWdThreads + tid, vpb - 1);
                    u[k] = ld_global_nc_v4(kv[k & 1] + (static_cast<size_t>(blk) * vpb + v) * 16);
                    s[k] = (k & 1 ? a.vscale : a.kscale)[static_cast<size_t>(blk) * a.Hkv +
                                                         v / (kBlk * a.d / 16)];
                }
#pragma unroll
                for (int k = 0; k < kWdLoads; ++k) {
                    const int v = v0 + k / 2 * kWdThreads + tid;
                    if (v >= vpb)
                        continue;
                    const uint32_t b[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
                    uint32_t o[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t lo = f16x2_of_e4m3(b[i]), hi = f16x2_of_e4m3(b[i] >> 16);
                        const float2 x0 = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
                        const float2 x1 = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                        o[2 * i] = pack_bf16x2(x0.x * s[k], x0.y * s[k]);
                        o[2 * i + 1] = pack_bf16x2(x1.x * s[k], x1.y * s[k]);
                    }
                    uint8_t *to = reinterpret_cast<uint8_t *>(k & 1 ? a.vwide : a.kwide) +
                                  (static_cast<size_t>(x) * vpb + v) * 32;
                    st_global_v4(to, make_uint4(o[0], o[1], o[2], o[3]));
                    st_global_v4(to + 16, make_uint4(o[4], o[5], o[6], o[7]));
                }
            }
        }
    }
}

cudaError_t launch_fp8_widen(const Fp8WidenArgs &a, int sms, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(6 * sms), 1, 1);
    cfg.blockDim = dim3(kWdThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, zp_fp8_widen_kernel, a);
}

}  // namespace zp
