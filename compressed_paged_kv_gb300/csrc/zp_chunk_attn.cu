// zp_chunk_attn.cu -- attention of a ragged chunk of new tokens over the paged
// cache: the many-query form of the decode attention.
//
// Query j of a chunk of n tokens sits at position p = length - n + j and sees
// the keys t <= p.  The G query heads of a kv head share its keys: a query row
// is (token, head of the group), token-major, 64 rows a CTA and 16 a warp.
// One pass over the 16-key blocks with a running maximum and sum a row (fp32,
// base 2), S = Q K^T and O += P V with mma.sync (P rounded to bf16).
//
// A value row hidden from some rows of the tile meets a probability of 0
// there, and 0 times an infinity or NaN is NaN: such elements of the rows past
// the tile's first position are cleared in shared memory, the lowest position
// is kept a column, and the output elements of the rows that see it are NaN.
#include "zp_chunk.cuh"

namespace zp {

namespace {
constexpr int kCaWarps = 4;
constexpr int kCaThreads = kCaWarps * 32;
constexpr int kCaRows = kCaWarps * 16;
}  // namespace

template <int D>
__global__ void __launch_bounds__(kCaThreads) zp_chunk_attn_kernel(const ChunkAttnArgs a)
{
    constexpr int CPR = D / 8, KS = D / 16;
    __shared__ __align__(1024) uint8_t sQ[kCaRows * D * 2];
    __shared__ __align__(1024) uint8_t sK[kBlk * D * 2];
    __shared__ __align__(1024) uint8_t sV[kBlk * D * 2];
    __shared__ int s_req[2];
    __shared__ int sBad[D];  // a column's lowest position with a cleared element
    const int tid = threadIdx.x, lane = tid & 31, wi = tid >> 5, mi = lane >> 3;
    const int h = blockIdx.y, G = a.Hq / a.Hkv;

    // the request and row tile of this CTA
    if (tid == 0) {
        int x = blockIdx.x, req = -1;
        for (int i = 0; i < a.R; ++i) {
            ChunkReq c;
            bool bad;
            const bool work = chunk_request(a, i, c, &bad);
            if (bad && blockIdx.x == 0 && h == 0)
                set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
            if (!work)
                continue;
            const int tiles = (c.n * G + kCaRows - 1) / kCaRows;
            if (req < 0 && x < tiles) {
                req = i;
                s_req[1] = x;
            }
            x -= tiles;
        }
        s_req[0] = req;
    }
    __syncthreads();
    if (s_req[0] < 0)
        return;
    ChunkReq c;
    bool bad;
    chunk_request(a, s_req[0], c, &bad);
    const int r0 = s_req[1] * kCaRows;  // first row of the tile
    const int rows = c.n * G;
    for (int e = tid; e < kCaRows * CPR; e += kCaThreads) {
        const int rr = e / CPR, ch = e % CPR, row = r0 + rr;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows)
            v = ld_global_nc_v4(a.q + (size_t)(c.first + row / G) * a.q_stride +
                                (size_t)(h * G + row % G) * D + ch * 8);
        st_shared_v4(smem_u32(sQ) + swz(rr, ch, kCaRows), v);
    }
    for (int e = tid; e < D; e += kCaThreads)
        sBad[e] = 0x7fffffff;
    __syncthreads();
    uint32_t qa[KS][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
        ldsm_x4(smem_u32(sQ) + swz(wi * 16 + (mi & 1) * 8 + (lane & 7), ks * 2 + (mi >> 1), kCaRows),
                qa[ks]);
    int lim[2];  // keys row hh of this thread sees
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int row = r0 + wi * 16 + (lane >> 2) + hh * 8;
        lim[hh] = row < rows ? c.len - c.n + row / G + 1 : 0;
    }
    const int last = min(r0 + kCaRows, rows) - 1;
    const int keys = c.len - c.n + last / G + 1;  // keys the tile's last row sees
    const int first_pos = c.len - c.n + r0 / G;          // position of the tile's first row
    float m_run[2] = {-1e30f, -1e30f}, l_run[2] = {0.f, 0.f};
    float o[D / 8][4];
#pragma unroll
    for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[nt][e] = 0.f;
    for (int t0 = 0; t0 < keys; t0 += kBlk) {
        int blk = a.tables[(size_t)c.row * a.stride + t0 / kBlk];
        if (blk < 0 || blk >= a.num_blocks) {
            set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
            blk = 0;
        }
        const size_t base = ((size_t)blk * a.Hkv + h) * kBlk * D;
        __syncthreads();
        for (int e = tid; e < kBlk * CPR; e += kCaThreads) {
            const int rr = e / CPR, ch = e % CPR;
            uint4 kv = make_uint4(0u, 0u, 0u, 0u), vv = kv;
            if (t0 + rr < c.len) {
                kv = ld_global_nc_v4(a.kpool + base + rr * D + ch * 8);
                vv = ld_global_nc_v4(a.vpool + base + rr * D + ch * 8);
                if (t0 + rr > first_pos) {
                    uint16_t *e16 = reinterpret_cast<uint16_t *>(&vv);
                    for (int x = 0; x < 8; ++x)
                        if ((e16[x] & 0x7f80) == 0x7f80) {
                            e16[x] = 0;
                            atomicMin(&sBad[ch * 8 + x], t0 + rr);
                        }
                }
            }
            st_shared_v4(smem_u32(sK) + swz(rr, ch, kBlk), kv);
            st_shared_v4(smem_u32(sV) + swz(rr, ch, kBlk), vv);
        }
        __syncthreads();
        float sacc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t kb[4];
            ldsm_x4(smem_u32(sK) + swz((mi >> 1) * 8 + (lane & 7), ks * 2 + (mi & 1), kBlk), kb);
            mma_bf16(sacc[0], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], kb[0], kb[1]);
            mma_bf16(sacc[1], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], kb[2], kb[3]);
        }
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            float mx = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int key = t0 + nt * 8 + (lane & 3) * 2 + e;
                    float v = sacc[nt][hh * 2 + e] * a.logit_scale;
                    if (key >= lim[hh])
                        v = -INFINITY;
                    sacc[nt][hh * 2 + e] = v;
                    mx = fmaxf(mx, v);
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float m_new = fmaxf(m_run[hh], mx);
            const float corr = ex2_approx(m_run[hh] - m_new);
            m_run[hh] = m_new;
            l_run[hh] *= corr;
#pragma unroll
            for (int nt = 0; nt < D / 8; ++nt) {
                o[nt][hh * 2] *= corr;
                o[nt][hh * 2 + 1] *= corr;
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float p = ex2_approx(sacc[nt][hh * 2 + e] - m_new);
                    sacc[nt][hh * 2 + e] = p;
                    l_run[hh] += p;
                }
        }
        const uint32_t pa0 = pack_bf16x2(sacc[0][0], sacc[0][1]);
        const uint32_t pa1 = pack_bf16x2(sacc[0][2], sacc[0][3]);
        const uint32_t pa2 = pack_bf16x2(sacc[1][0], sacc[1][1]);
        const uint32_t pa3 = pack_bf16x2(sacc[1][2], sacc[1][3]);
#pragma unroll
        for (int dp = 0; dp < D / 16; ++dp) {
            uint32_t vb[4];
            ldsm_x4_t(smem_u32(sV) + swz((mi & 1) * 8 + (lane & 7), dp * 2 + (mi >> 1), kBlk), vb);
            mma_bf16(o[2 * dp], pa0, pa1, pa2, pa3, vb[0], vb[1]);
            mma_bf16(o[2 * dp + 1], pa0, pa1, pa2, pa3, vb[2], vb[3]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        float l = l_run[hh];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int row = r0 + wi * 16 + (lane >> 2) + hh * 8;
        if (row >= rows)
            continue;
        const float inv = 1.0f / l;
        __nv_bfloat16 *dst = a.out + ((size_t)(c.first + row / G) * a.Hq + h * G + row % G) * D;
#pragma unroll
        for (int nt = 0; nt < D / 8; ++nt) {
            const int col = nt * 8 + (lane & 3) * 2;
            const float x0 = sBad[col] < lim[hh] ? NAN : o[nt][hh * 2] * inv;
            const float x1 = sBad[col + 1] < lim[hh] ? NAN : o[nt][hh * 2 + 1] * inv;
            *reinterpret_cast<uint32_t *>(dst + col) = pack_bf16x2(x0, x1);
        }
    }
}

cudaError_t launch_chunk_attn(const ChunkAttnArgs &a, int d, cudaStream_t s)
{
    const int G = a.Hq / a.Hkv;
    const long long tiles = static_cast<long long>(a.total) * G / kCaRows + a.R;
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(a.Hkv), 1);
    if (d == 64)
        zp_chunk_attn_kernel<64><<<grid, kCaThreads, 0, s>>>(a);
    else if (d == 128)
        zp_chunk_attn_kernel<128><<<grid, kCaThreads, 0, s>>>(a);
    else
        return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace zp
