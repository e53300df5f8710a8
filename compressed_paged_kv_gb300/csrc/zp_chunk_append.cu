// zp_chunk_append.cu -- the keys and values of a ragged chunk of new tokens
// into the paged slots reserved for them: the many-token form of
// zp_append_kv.
//
// A pure copy (2 * Hkv * d * 2 bytes read and written a token), bound by HBM
// for many tokens (35,000 of 8 x 128: 45 us = 6.3 TB/s, 0.93 of the copy peak)
// and by the chain of dependent reads (chunk offsets, row and length -> block
// id) for few (40 tokens: 2.7 us on the device, calls in a captured graph; 8 us a
// call with the host's side).  One warp a token: it finds the request by a 32-ary
// search of the chunk offsets (one round of loads up to 32 requests, two up to
// 1,024), then moves the token's K and V rows 16 bytes a lane.
#include "zp_chunk.cuh"

namespace zp {

namespace {

constexpr int kCkThreads = 256;

// The last i in [0, R) with starts[i] <= t, or 0 (the caller checks that the
// chunk holds t): every round the 32 lanes probe the range at equal steps.
__device__ __forceinline__ int find_request(const int32_t *starts, int R, long long t, int lane)
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

}  // namespace

__global__ void __launch_bounds__(kCkThreads) zp_append_kv_chunk_kernel(const ChunkKvArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const long long t =
        blockIdx.x * static_cast<long long>(kCkThreads / 32) + static_cast<int>(threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    ChunkReq c;
    bool bad = false;
    // every request is checked once, whether or not a token finds it
    for (long long i = blockIdx.x * static_cast<long long>(kCkThreads) + threadIdx.x; i < a.R;
         i += static_cast<long long>(gridDim.x) * kCkThreads) {
        chunk_request(a, static_cast<int>(i), c, &bad);
        if (bad)
            set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
    }
    if (t >= a.total)
        return;
    const int i = find_request(a.starts, a.R, t, lane);
    if (!chunk_request(a, i, c, &bad) || t < c.first || t >= c.first + c.n)
        return;  // a bad request, or a row of no request: padding
    const int p = c.len - c.n + static_cast<int>(t - c.first);
    const int blk = a.tables[(size_t)c.row * a.stride + p / kBlk];
    if (blk < 0 || blk >= a.num_blocks) {
        if (lane == 0)
            set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
        return;
    }
    const int vpr = a.d / 8;  // 16-byte vectors per head row
    const int nv = a.Hkv * vpr;
    const uint4 *ks = reinterpret_cast<const uint4 *>(a.k_new + t * a.k_stride);
    const uint4 *vs = reinterpret_cast<const uint4 *>(a.v_new + t * a.v_stride);
    uint4 *kd = reinterpret_cast<uint4 *>(a.kpool);
    uint4 *vd = reinterpret_cast<uint4 *>(a.vpool);
    const size_t base = (size_t)blk * a.Hkv * kBlk + p % kBlk;
    for (int v = lane; v < nv; v += 32) {
        const size_t dst = (base + (size_t)(v / vpr) * kBlk) * vpr + v % vpr;
        kd[dst] = ld_global_nc_v4(ks + v);
        vd[dst] = ld_global_nc_v4(vs + v);
    }
}

cudaError_t launch_append_kv_chunk(const ChunkKvArgs &a, cudaStream_t s)
{
    const long long threads = static_cast<long long>(a.total) * 32;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((threads + kCkThreads - 1) / kCkThreads), 1, 1);
    cfg.blockDim = dim3(kCkThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, zp_append_kv_chunk_kernel, a);
}

}  // namespace zp
