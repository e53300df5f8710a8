// zp_fp8_decode.cu -- attention of few query rows over an 8-bit paged cache:
// zp_paged_decode_attn of such a cache, and the requests of zp_paged_chunk_attn whose
// chunk has up to 24 rows (tokens times heads of a group).
//
// A key is ks * k8 and a value vs * v8, with one ks and one vs for the 16 tokens of
// a block: neither is multiplied out.  With t = scale (q . k8) ks + log2 vs and
// p = 2^t (base 2),
//     out = sum p v8 / sum (p / vs),
// so ks enters once a logit, log2 vs is added to it, and 1 / vs enters once a block's
// sum.  The running maximum is that of t: what the maximum keeps in range is the
// weight that a number gets in the product with V.
//
// Both products run on the tensor cores in fp16 (mma.sync m16n8k16, fp32
// accumulation), which holds every e4m3 number exactly and into which the hardware
// converts two at a time.  q is scaled by a power of two for each head, so that its
// largest element lies below 2^15 (fp16 then keeps all of bf16's bits of elements down to
// 2^-28 of that); p is taken against 2^14 over the maximum, and rounded to 11 bits down
// to 2^-28 of the largest, where bf16 would round to 8.
//
// The keys are the products' rows and q's rows of the kv head their columns, in eights (NT):
// S^T = K Q^T, O^T = V^T P^T.  With the heads as rows, of which 16 would be computed for a
// group of four, the kernel took twice the products and twice the registers.  Fragments come
// by ldmatrix: a matrix of 8 keys x 16 bytes gives a lane four neighbouring dims of a key, so
// q's fragments are laid out to match; for V, the transposed matrix gives a lane two dims of
// two keys, which a byte permutation turns into the pairs of keys that the product takes, the
// even dims as its rows 0-7 and the odd ones as 8-15.  P turns from rows of keys to rows of
// heads by movmatrix.
//
// Grid (request and split, kv head), four warps a CTA.  A CTA owns a contiguous range of
// blocks, the row's over its splits but no fewer than eight; a warp takes every fourth pair of
// them through its own ring of pairs (one TMA box a slab).  Warps join in shared memory, and up
// to eight splits, a cluster, too; more clusters of a long row leave partial results to a
// second kernel.
//
// Measured, 32 heads of 128 over 8 kv heads: 256 requests of 1,024 to 2,039 tokens, 0.81 GB in
// 133 us = 6.1 TB/s, 0.90 of the copy peak (with 16 rows of heads and two CTAs an SM 166 us);
// one of 2,000 tokens 6.5 us, the chain row -> block ids -> slabs -> joins; bound by HBM where
// the rows fill the GPU.  256 chunks of 1, 4 and 6 tokens over 1,536, 0.81 GB: 149, 182 and
// 262 us (in the kernel for tiles of 128 rows 289, 295 and 297); with more columns a warp waits
// for its own products, three and two CTAs an SM being all that registers and rings leave
// (schedulers issue in 45 % of the cycles).  Four eights took 300 us.
#include <algorithm>

#include "zp_fp8.cuh"

namespace zp {

namespace {

constexpr int kD8Warps = 4;
constexpr int kD8Threads = kD8Warps * 32;
constexpr float kTop = 14.f;   // log2 of the largest p
constexpr float kHuge = 3e38f;  // minus the maximum of no keys (an infinity less itself is NaN)
constexpr int kD8Cluster = 8;  // splits that a cluster joins
constexpr int kD8Blocks = 8;   // of a split, at least
constexpr int kD8Groups = 16;  // clusters a (request, kv head), at most

template <int D, int NT>
struct D8Smem {
    static constexpr int STAGES = D == 128 ? 2 : 3;  // of a pair of blocks, K and V
    static constexpr int SLAB = kBlk * D;
    static constexpr int STAGE = 4 * SLAB;  // K of two blocks, V of two blocks
    static constexpr int RING = kD8Warps * STAGES * STAGE;
    static constexpr int ROW = D + 2;       // o, then (maximum, sum), of a head
    static constexpr int MERGE = kD8Warps * 8 * NT * ROW * 4;  // reuses the ring
    static constexpr int off_part = MERGE;  // the CTA's own, for the cluster
    static constexpr int JOIN = MERGE + 8 * NT * ROW * 4;
    static constexpr int off_bar = RING > JOIN ? RING : JOIN;
    static constexpr int off_q = off_bar + kD8Warps * STAGES * 8;  // q's fragments, if there
    static constexpr bool QS = NT > 2;
    static constexpr int off_f = off_q + (QS ? NT * (D / 16) * 32 * 8 : 0);
    static constexpr int BYTES = off_f + (QS ? 8 * NT * 4 : 0);
    static constexpr int ALLOC = BYTES + 1024;
};

// An infinity as the largest number, so that a score of 0 times it is 0; NaN stays NaN.
__device__ __forceinline__ float finite(float x)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(__uint_as_float(0xff7fffffu)));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(y), "f"(__uint_as_float(0x7f7fffffu)));
    return y;
}

// An 8x8 matrix of 16-bit elements, a row's two neighbours a lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

}  // namespace

// NT: eights of columns of a warp.
template <int D, int NT, bool CHUNK>
__global__ void __launch_bounds__(kD8Threads, NT > 2 ? (D == 128 ? 2 : 3) : D == 128 ? 3 : 4)
    zp_fp8_decode_kernel(const __grid_constant__ Fp8AttnArgs a)
{
    if constexpr (CHUNK) {
        // A launch behind another of the same call starts as that one's CTAs end.  The first CTAs,
        // and with them the grid, end no sooner than that one, so that who waits for this grid
        // waits for both (end_of_grid below).
        if (a.follows) {
            await_visible(a.visible);
        } else {
            pdl_wait();
            if (a.visible && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
                say_visible(a.visible);
        }
        pdl_launch_dependents();
    } else {
        pdl_wait();
    }
    using S = D8Smem<D, NT>;
    constexpr int KS = D / 16, ROW = S::ROW, COLS = 8 * NT;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + (1024 - (smem_u32(smem_raw) & 1023) & 1023);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + S::off_bar);
    float *part = reinterpret_cast<float *>(sm + S::off_part);

    const int tid = threadIdx.x, lane = tid & 31, wi = tid >> 5;
    const int split = blockIdx.x % a.splits, r = blockIdx.x / a.splits, h = blockIdx.y;
    const int G = a.Hq / a.Hkv;
    ChunkReq rq{r, 1, 0, 0};
    [[maybe_unused]] auto end_of_grid = [&] {
        if (!a.follows || blockIdx.x != 0)
            return;
        pdl_wait();
        if (a.last && blockIdx.y == 0 && tid == 0)
            clear_visible(a.visible);
    };
    if constexpr (CHUNK) {
        // By the offsets first, as in some batches most CTAs have no more to do.  The first launch
        // of a call checks every request but the longer ones (not past the total: so there is
        // another kernel, which checks them).
        const int n = __ldcg(a.starts + r + 1) - __ldcg(a.starts + r);
        const bool longer = n > COLS / G && n <= a.total;
        bool bad = false, work = false;
        if (a.over == 0 ? !longer : n > a.over && n <= COLS / G)
            work = chunk_request(a, r, rq, &bad);
        if (bad && tid == 0 && split == 0 && h == 0)
            set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
        if (!work || rq.n > COLS / G) {  // (the whole cluster alike)
            end_of_grid();
            return;
        }
    } else {
        rq.row = a.req_idx ? a.req_idx[r] : r;
        const bool row_ok = rq.row >= 0 && rq.row < a.num_rows;
        rq.len = row_ok ? a.lengths[rq.row] : 0;
        if (!row_ok || rq.len < 0 || rq.len > a.stride * kBlk) {
            if (tid == 0 && split == 0 && h == 0)
                set_error(a.sticky, row_ok ? ZP_ERR_DEVICE_CHECK : ZP_ERR_INVALID_ARG);
            rq.len = 0;
            rq.row = 0;
        }
    }
    // q's rows of the kv head, heads of a token side by side, are the columns
    const int len = rq.len, rows = rq.n * G;
    const int nblk = (len + kBlk - 1) / kBlk;
    const int bps = max(kD8Blocks, ((nblk + a.splits - 1) / a.splits + 1) & ~1);
    const int b_begin = split * bps;
    const int b_end = min(nblk, b_begin + bps);

    uint64_t *my_bar = bars + wi * S::STAGES;
    if (lane < S::STAGES)
        mbar_init(&my_bar[lane], 1);
    fence_mbar_init();
    __syncwarp();

    // this warp's pairs of blocks: wi, wi + 4, .. of the range
    const int pairs = b_end > b_begin ? (b_end - b_begin + 1) / 2 : 0;
    const int my_n = pairs > wi ? (pairs - wi + kD8Warps - 1) / kD8Warps : 0;
    uint8_t *my_stage = sm + wi * S::STAGES * S::STAGE;
    const int32_t *trow = a.tables + static_cast<size_t>(rq.row) * a.stride;

    // block ids and scales of 16 pairs, a block a lane, and of the 16 after them
    auto load_id = [&](int i) {
        const int b = b_begin + 2 * (wi + kD8Warps * (i + (lane >> 1))) + (lane & 1);
        int id = b < b_end ? trow[b] : 0;
        if (id < 0 || id >= a.num_blocks) {
            set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
            id = 0;
        }
        return id;
    };
    auto scale_at = [&](const float *s, int id) { return s[static_cast<size_t>(id) * a.Hkv + h]; };
    int id = my_n > 0 ? load_id(0) : 0, id_next = 0;

    auto issue = [&](int i, int ids) {
        const int l = (i & 15) * 2;
        const int y0 = (__shfl_sync(0xffffffffu, ids, l) * a.Hkv + h) * kBlk;
        const int y1 = (__shfl_sync(0xffffffffu, ids, l + 1) * a.Hkv + h) * kBlk;
        if (lane == 0) {
            const bool two = b_begin + 2 * (wi + kD8Warps * i) + 1 < b_end;
            const int s = i % S::STAGES;
            uint8_t *kd = my_stage + s * S::STAGE, *vd = kd + 2 * S::SLAB;
            mbar_arrive_expect_tx(&my_bar[s], two ? S::STAGE : S::STAGE / 2);
            tma_load_2d(kd, a.kmap, 0, y0, &my_bar[s]);
            if (two)
                tma_load_2d(kd + S::SLAB, a.kmap, 0, y1, &my_bar[s]);
            tma_load_2d(vd, a.vmap, 0, y0, &my_bar[s]);
            if (two)
                tma_load_2d(vd + S::SLAB, a.vmap, 0, y1, &my_bar[s]);
        }
        __syncwarp();
    };
    for (int i = 0; i < my_n && i < S::STAGES; ++i)
        issue(i, id);
    float ks = scale_at(a.kscale, id), vs = scale_at(a.vscale, id), ks_next = 0.f, vs_next = 0.f;

    // q's fragments: column 8 n + g, dims 16 c + 4 t .. + 3
    const int g = lane >> 2, t4 = lane & 3;
    auto fragments = [&](int n, uint32_t (&f)[KS][2]) {
        const int col = n * 8 + g, in = min(col, rows - 1), tok = CHUNK ? in / G : 0;
        const __nv_bfloat16 *src =
            a.q + (rq.first + tok) * a.q_stride + (h * G + in - tok * G) * D + t4 * 4;
        uint2 u[KS];
        uint32_t most = 0;  // the largest finite magnitude's bits
#pragma unroll
        for (int c = 0; c < KS; ++c) {
            u[c] = make_uint2(0u, 0u);
            if (col < rows)
                u[c] = *reinterpret_cast<const uint2 *>(src + c * 16);
            const uint32_t w[4] = {u[c].x << 16, u[c].x, u[c].y << 16, u[c].y};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t m = w[e] & 0x7fff0000u;
                most = max(most, m < 0x7f800000u ? m : 0u);
            }
        }
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        // to below 2^15; two factors, as 2^e may not be an fp32 number
        const int e = 14 - (static_cast<int>(most >> 23) - 127);
        const int e1 = max(min(e, 100), -100), e2 = e - e1;
        const float f1 = __uint_as_float(exp2_bits(e1)), f2 = __uint_as_float(exp2_bits(e2));
#pragma unroll
        for (int c = 0; c < KS; ++c) {
            f[c][0] = pack_f16x2(__uint_as_float(u[c].x << 16) * f1 * f2,
                                 __uint_as_float(u[c].x & 0xffff0000u) * f1 * f2);
            f[c][1] = pack_f16x2(__uint_as_float(u[c].y << 16) * f1 * f2,
                                 __uint_as_float(u[c].y & 0xffff0000u) * f1 * f2);
        }
        return a.logit_scale * __uint_as_float(exp2_bits(-e1)) * __uint_as_float(exp2_bits(-e2));
    };
    // in registers, or (more than 16 columns) in shared memory
    uint32_t qb[S::QS ? 1 : NT][KS][2];
    float fr[NT][2];  // columns 8 n + 2 t, + 1: what a logit is multiplied by, but for ks
    uint2 *sQ = reinterpret_cast<uint2 *>(sm + S::off_q);
    if constexpr (S::QS) {
        float *sF = reinterpret_cast<float *>(sm + S::off_f);
        if (wi < NT) {
            const float back = fragments(wi, qb[0]);
#pragma unroll
            for (int c = 0; c < KS; ++c)
                sQ[(wi * KS + c) * 32 + lane] = make_uint2(qb[0][c][0], qb[0][c][1]);
            if (t4 == 0)
                sF[wi * 8 + g] = back;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            fr[n][0] = sF[n * 8 + t4 * 2];
            fr[n][1] = sF[n * 8 + t4 * 2 + 1];
        }
    } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float back = fragments(n, qb[n]);
            fr[n][0] = __shfl_sync(0xffffffffu, back, t4 * 8);
            fr[n][1] = __shfl_sync(0xffffffffu, back, t4 * 8 + 4);
        }
    }

    // a chunk's columns 8 n + 2 t, + 1: the keys they see
    [[maybe_unused]] int lim[NT][2];
    [[maybe_unused]] const int sees = len - rq.n + 1;  // keys that every column sees
    if constexpr (CHUNK) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                lim[n][e] = sees + min(n * 8 + t4 * 2 + e, rows - 1) / G;
    }
    
    float m_run[NT][2], l_run[NT][2];
    float o[NT][KS][4];  // dims 16 c + 2 g (+ 1 in [2], [3]), columns 8 n + 2 t, + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m_run[n][0] = m_run[n][1] = -kHuge;
        l_run[n][0] = l_run[n][1] = 0.f;
#pragma unroll
        for (int c = 0; c < KS; ++c)
            o[n][c][0] = o[n][c][1] = o[n][c][2] = o[n][c][3] = 0.f;
    }
    bool ok = true;
    const int mi = lane >> 3;

    for (int i = 0; i < my_n; ++i) {
        const int s = i % S::STAGES;
        const int b0 = b_begin + 2 * (wi + kD8Warps * i);
        const bool two = b0 + 1 < b_end;
        const int tok0 = b0 * kBlk;
        const int l = (i & 15) * 2;
        if ((i & 15) == 0 && i + 16 < my_n)
            id_next = load_id(i + 16);
        if ((i & 15) == 8 && i + 8 < my_n) {
            ks_next = scale_at(a.kscale, id_next);
            vs_next = scale_at(a.vscale, id_next);
        }
        ok &= mbar_wait(&my_bar[s], (i / S::STAGES) & 1);
        uint8_t *kd = my_stage + s * S::STAGE, *vd = kd + 2 * S::SLAB;
        if (len - tok0 < (two ? 2 : 1) * kBlk) {
            // the slots past the length get probability 0, but 0 times a NaN is NaN: their
            // V rows are cleared
            const int fill = len - tok0;  // >= 1
            for (int c = lane; c < 2 * kBlk * (D / 16); c += 32) {
                const int rr = c / (D / 16);
                if (rr >= fill && (two || rr < kBlk))
                    st_shared_v4(smem_u32(vd) + rr * D + c % (D / 16) * 16,
                                 make_uint4(0u, 0u, 0u, 0u));
            }
            __syncwarp();
        }
        const uint32_t kb = smem_u32(kd), vb = smem_u32(vd);

        // S^T: keys 16 blk + g (in [0], [1]) and + 8, columns 8 n + 2 t, + 1
        float sacc[2][NT][4];
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                sacc[blk][n][0] = sacc[blk][n][1] = sacc[blk][n][2] = sacc[blk][n][3] = 0.f;
        // chunks c and c + 1 of a block's keys; f: q's fragments for them
        auto products = [&](int blk, int c, const uint32_t (&f)[NT][2][2]) {
            // matrices: keys 0-7 and 8-15 of chunk c, then of c + 1
            uint32_t kr[4];
            ldsm_x4(kb + blk * S::SLAB + swz8<D>((mi & 1) * 8 + (lane & 7), c + (mi >> 1)), kr);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t a0 = f16x2_of_e4m3(kr[2 * x]), a1 = f16x2_of_e4m3(kr[2 * x + 1]);
                const uint32_t a2 = f16x2_of_e4m3(kr[2 * x] >> 16);
                const uint32_t a3 = f16x2_of_e4m3(kr[2 * x + 1] >> 16);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma_f16(sacc[blk][n], a0, a1, a2, a3, f[n][x][0], f[n][x][1]);
            }
        };
        if constexpr (S::QS) {
#pragma unroll
            for (int c = 0; c < KS; c += 2) {
                uint32_t f[NT][2][2];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint2 v = sQ[(n * KS + c + x) * 32 + lane];
                        f[n][x][0] = v.x;
                        f[n][x][1] = v.y;
                    }
                products(0, c, f);
                if (two)
                    products(1, c, f);
            }
        } else {
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
                if (blk && !two)
                    break;
#pragma unroll
                for (int c = 0; c < KS; c += 2) {
                    uint32_t f[NT][2][2];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            f[n][x][0] = qb[n][c + x][0];
                            f[n][x][1] = qb[n][c + x][1];
                        }
                    products(blk, c, f);
                }
            }
        }
        float iv[2];
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
            const float kx = __shfl_sync(0xffffffffu, ks, l + blk);
            const float vx = __shfl_sync(0xffffffffu, vs, l + blk);
            const float lv = log2f(vx);
            iv[blk] = blk && !two ? 0.f : 1.f / vx;
            const int key = blk * kBlk + g;
            const bool there = two || !blk;
            const bool in0 = tok0 + key < len && there, in1 = tok0 + key + 8 < len && there;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = fmaf(sacc[blk][n][e], finite(fr[n][e & 1] * kx), lv);
                    bool in = e < 2 ? in0 : in1;
                    if constexpr (CHUNK)
                        in = tok0 + key + (e < 2 ? 0 : 8) < lim[n][e & 1] && there;
                    sacc[blk][n][e] = in ? v : -INFINITY;
                }
        }
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float corr[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(fmaxf(sacc[0][n][e], sacc[0][n][e + 2]),
                                 fmaxf(sacc[1][n][e], sacc[1][n][e + 2]));
                if (!two)
                    mx = fmaxf(sacc[0][n][e], sacc[0][n][e + 2]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float m_new = fmaxf(m_run[n][e], mx);
                corr[e] = ex2_approx(m_run[n][e] - m_new);
                m_run[n][e] = m_new;
                const float at = m_new - kTop;
#pragma unroll
                for (int blk = 0; blk < 2; ++blk) {
                    sacc[blk][n][e] = ex2_approx(sacc[blk][n][e] - at);
                    sacc[blk][n][e + 2] = ex2_approx(sacc[blk][n][e + 2] - at);
                }
                const float s0 = sacc[0][n][e] + sacc[0][n][e + 2];
                const float s1 = sacc[1][n][e] + sacc[1][n][e + 2];
                l_run[n][e] = fmaf(l_run[n][e], corr[e], fmaf(s0, iv[0], two ? s1 * iv[1] : 0.f));
            }
            if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
                for (int c = 0; c < KS; ++c) {
                    o[n][c][0] *= corr[0];
                    o[n][c][1] *= corr[1];
                    o[n][c][2] *= corr[0];
                    o[n][c][3] *= corr[1];
                }
            }
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
                pb[blk][n][0] = transposed(pack_f16x2(sacc[blk][n][0], sacc[blk][n][1]));
                pb[blk][n][1] = transposed(pack_f16x2(sacc[blk][n][2], sacc[blk][n][3]));
            }
        }
        // A value that is NaN: 0 times it is NaN, for the columns too that do not see its key.
        // Among the keys that some do not see, NaN counts as 0 and is added to the columns that
        // do see it: those for which a product of ones, at the NaNs and at the keys seen, is
        // above 0.
        [[maybe_unused]] bool nan_v = false;
        if constexpr (CHUNK) {
            const int last = (two ? 2 : 1) * kBlk;
            if (rq.n > 1 && tok0 + last > sees) {
                for (int x = lane; x < last * (D / 16); x += 32) {
                    const uint4 v = ld_shared_v4(vb + x * 16);
                    nan_v |= numbers4(v.x) != v.x || numbers4(v.y) != v.y ||
                             numbers4(v.z) != v.z || numbers4(v.w) != v.w;
                }
                nan_v = __any_sync(0xffffffffu, nan_v);
            }
            if (nan_v) {
#pragma unroll 1
                for (int n = 0; n < NT; ++n)
#pragma unroll 1
                    for (int c = 0; c < KS; ++c) {
                        float at[4] = {0.f, 0.f, 0.f, 0.f};
                        for (int blk = 0; blk < (two ? 2 : 1); ++blk) {
                            const int key = tok0 + blk * kBlk + g;
                            int l0 = 0, l1 = 0;
#pragma unroll
                            for (int k = 0; k < NT; ++k)
                                if (k == n) {
                                    l0 = lim[k][0];
                                    l1 = lim[k][1];
                                }
                            const uint32_t p0 = transposed(pack_f16x2(key < l0, key < l1));
                            const uint32_t p1 = transposed(pack_f16x2(key + 8 < l0, key + 8 < l1));
                            uint32_t vr[4];
                            ldsm_x4_t(vb + blk * S::SLAB +
                                          swz8<D>((mi & 1) * 8 + (lane & 7), (c & ~1) + (mi >> 1)),
                                      vr);
                            const uint32_t v0 = c & 1 ? vr[2] : vr[0], v1 = c & 1 ? vr[3] : vr[1];
                            const uint32_t lo = __byte_perm(ones4(v0), 0, 0x3120);
                            const uint32_t hi = __byte_perm(ones4(v1), 0, 0x3120);
                            mma_f16(at, f16x2_of_e4m3(lo), f16x2_of_e4m3(lo >> 16),
                                    f16x2_of_e4m3(hi), f16x2_of_e4m3(hi >> 16), p0, p1);
                        }
#pragma unroll
                        for (int k = 0; k < NT; ++k)
#pragma unroll
                            for (int q = 0; q < KS; ++q)
                                if (k == n && q == c)
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        if (at[e] > 0.f)
                                            o[k][q][e] = INFINITY - INFINITY;
                    }
            }
        }
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
            if (blk && !two)
                break;
#pragma unroll
            for (int c = 0; c < KS; c += 2) {
                // matrices: keys 0-7 and 8-15 of chunk c, then of c + 1
                uint32_t vr[4];
                ldsm_x4_t(vb + blk * S::SLAB + swz8<D>((mi & 1) * 8 + (lane & 7), c + (mi >> 1)),
                          vr);
                if (CHUNK && nan_v)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        vr[k] = numbers4(vr[k]);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    // bytes: key 2 t (dims 2 g, 2 g + 1), key 2 t + 1 (the same)
                    const uint32_t lo = __byte_perm(vr[2 * x], 0, 0x3120);
                    const uint32_t hi = __byte_perm(vr[2 * x + 1], 0, 0x3120);
                    const uint32_t a0 = f16x2_of_e4m3(lo), a1 = f16x2_of_e4m3(lo >> 16);
                    const uint32_t a2 = f16x2_of_e4m3(hi), a3 = f16x2_of_e4m3(hi >> 16);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_f16(o[n][c + x], a0, a1, a2, a3, pb[blk][n][0], pb[blk][n][1]);
                }
            }
        }
        __syncwarp();
        if (i + S::STAGES < my_n) {
            fence_proxy_async_smem();
            __syncwarp();
            issue(i + S::STAGES, ((i + S::STAGES) ^ i) & 16 ? id_next : id);
        }
        if ((i & 15) == 15) {
            id = id_next;
            ks = ks_next;
            vs = vs_next;
        }
    }
    if (!ok && lane == 0)
        set_error(a.sticky, ZP_ERR_TIMEOUT);
    if constexpr (!CHUNK)
        pdl_launch_dependents();  // the combine kernel may be scheduled
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l_run[n][e] += __shfl_xor_sync(0xffffffffu, l_run[n][e], 4);
            l_run[n][e] += __shfl_xor_sync(0xffffffffu, l_run[n][e], 8);
            l_run[n][e] += __shfl_xor_sync(0xffffffffu, l_run[n][e], 16);
        }
    __syncthreads();  // every stage consumed: reuse the area for the merge

    float *mrg = reinterpret_cast<float *>(sm);  // [warp][COLS][ROW]
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float *mine = mrg + (wi * COLS + n * 8 + t4 * 2 + e) * ROW;
            if (g == 0) {
                mine[D] = m_run[n][e];
                mine[D + 1] = l_run[n][e];
            }
#pragma unroll
            for (int c = 0; c < KS; ++c)
                *reinterpret_cast<float2 *>(mine + c * 16 + g * 2) =
                    make_float2(o[n][c][e], o[n][c][e + 2]);
        }
    __syncthreads();
    // the four warps', then the cluster's; two dims a thread
    const int cs = a.splits / a.groups, rank = split % cs;  // a cluster's CTAs
    // the output's row of (token, head) of a column
    auto row_of = [&](int col) {
        const int tok = CHUNK ? col / G : 0;
        return static_cast<size_t>(rq.first + tok) * a.Hq + h * G + col - tok * G;
    };
    auto join = [&](int hd, int c, const float *src, int step, int count, float &M, float &L,
                    float2 &O) {
        M = -kHuge;
        for (int w = 0; w < count; ++w)
            M = fmaxf(M, src[w * step + hd * ROW + D]);
        L = 0.f;
        O = make_float2(0.f, 0.f);
        for (int w = 0; w < count; ++w) {
            const float *p = src + w * step + hd * ROW;
            const float f = ex2_approx(p[D] - M);
            const float2 v = *reinterpret_cast<const float2 *>(p + c);
            L += p[D + 1] * f;
            O.x += v.x * f;
            O.y += v.y * f;
        }
    };
    auto write = [&](int hd, int c, float L, float2 O) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        __nv_bfloat16 *to = a.out + row_of(hd) * D + c;  // (2-byte aligned)
        to[0] = __float2bfloat16_rn(O.x * inv);
        to[1] = __float2bfloat16_rn(O.y * inv);
    };
    for (int x = tid; x < rows * (D / 2); x += kD8Threads) {
        const int hd = x / (D / 2), c = x % (D / 2) * 2;
        float M, L;
        float2 O;
        join(hd, c, mrg, COLS * ROW, kD8Warps, M, L, O);
        if (a.splits == 1) {
            write(hd, c, L, O);
            continue;
        }
        float *p = part + hd * ROW;
        *reinterpret_cast<float2 *>(p + c) = O;
        if (c == 0)
            *reinterpret_cast<float2 *>(p + D) = make_float2(M, L);
    }
    if (a.splits == 1) {
        if constexpr (CHUNK)
            end_of_grid();
        return;
    }
    cluster_sync();
    // each CTA joins its part of the dims
    for (int x = rank * kD8Threads + tid; x < rows * (D / 2); x += cs * kD8Threads) {
        const int hd = x / (D / 2), c = x % (D / 2) * 2;
        float2 ml[kD8Cluster], v[kD8Cluster];
#pragma unroll
        for (int w = 0; w < kD8Cluster; ++w) {
            ml[w] = make_float2(-kHuge, 0.f);
            v[w] = make_float2(0.f, 0.f);
            if (w < cs) {
                ml[w] = ld_dsmem_f32x2(dsmem_addr(part + hd * ROW + D, w));
                v[w] = ld_dsmem_f32x2(dsmem_addr(part + hd * ROW + c, w));
            }
        }
        float M = -kHuge, L = 0.f;
        float2 O = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kD8Cluster; ++w)
            M = fmaxf(M, ml[w].x);
#pragma unroll
        for (int w = 0; w < kD8Cluster; ++w) {
            const float f = ex2_approx(ml[w].x - M);
            L += ml[w].y * f;
            O.x += v[w].x * f;
            O.y += v[w].y * f;
        }
        if (a.groups == 1) {
            write(hd, c, L, O);
            continue;
        }
        float *p = a.part + (row_of(hd) * a.groups + split / cs) * ROW;
        *reinterpret_cast<float2 *>(p + c) = O;
        if (c == 0)
            *reinterpret_cast<float2 *>(p + D) = make_float2(M, L);
    }
    cluster_sync();  // no CTA leaves while its part is read
    if constexpr (CHUNK)
        end_of_grid();
}

template <int D>
__global__ void __launch_bounds__(D) zp_fp8_combine_kernel(const Fp8AttnArgs a)
{
    pdl_wait();
    const int rh = blockIdx.x;  // request * Hq + hq
    const int c = threadIdx.x;
    const float *base = a.part + static_cast<size_t>(rh) * a.groups * (D + 2);
    float M = -kHuge;
    for (int s = 0; s < a.groups; ++s)
        M = fmaxf(M, base[s * (D + 2) + D]);
    float L = 0.f, O = 0.f;
    for (int s = 0; s < a.groups; ++s) {
        const float f = ex2_approx(base[s * (D + 2) + D] - M);
        L += base[s * (D + 2) + D + 1] * f;
        O += base[s * (D + 2) + c] * f;
    }
    a.out[static_cast<size_t>(rh) * D + c] = __float2bfloat16_rn(L == 0.f ? 0.f : O / L);
}

template <int D, int NT, bool CHUNK>
static cudaError_t launch_fp8_decode_t(const Fp8AttnArgs &a, cudaStream_t s)
{
    using Sm = D8Smem<D, NT>;
    cudaError_t err = cudaFuncSetAttribute(zp_fp8_decode_kernel<D, NT, CHUNK>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, Sm::ALLOC);
    if (err != cudaSuccess)
        return err;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.splits / a.groups);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.splits) * static_cast<unsigned>(a.R),
                       static_cast<unsigned>(a.Hkv), 1);
    cfg.blockDim = dim3(kD8Threads, 1, 1);
    cfg.dynamicSmemBytes = Sm::ALLOC;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = a.splits > 1 ? 2 : 1;
    err = cudaLaunchKernelEx(&cfg, zp_fp8_decode_kernel<D, NT, CHUNK>, a);
    if (err != cudaSuccess || a.groups == 1)
        return err;
    cfg.gridDim = dim3(static_cast<unsigned>(a.R * a.Hq), 1, 1);
    cfg.blockDim = dim3(D, 1, 1);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, zp_fp8_combine_kernel<D>, a);
}

// Two CTAs an SM, of at least 8 blocks each; more than a cluster of them where each then has
// 16 blocks, which pays for the second launch (one row of 30,000 tokens 17 us, with 16
// splits 24).
int fp8_decode_splits(long long pairs, int bt_stride, int num_sms, int *groups)
{
    const long long want = (2 * num_sms + pairs - 1) / pairs;
    int splits = static_cast<int>(std::min<long long>({want, kD8Cluster, bt_stride / 8}));
    splits = std::max(1, splits);
    *groups = static_cast<int>(std::min<long long>(
        {want / kD8Cluster, kD8Groups, bt_stride / (16 * kD8Cluster)}));
    if (*groups > 1)
        splits = kD8Cluster * *groups;
    else
        *groups = 1;
    return splits;
}

// A large batch has a launch for up to 16 rows (8 of a mean of 8 or less), unless its mean says that
// hardly any chunk has so few, and one for up to 24 of a mean of no more.  Measured with 8 kv heads
// against the other kernel alone: 256 chunks of 2 to 9 tokens, four heads a group, 273 and 303 us; of
// 1 to 5, 217 and 305; 200 single tokens beside 8 pieces of 600, 279 and 373; where none is short, 256
// of 8 tokens 302 and 295, of 20 tokens 325 and 318.  A small batch, where a launch more costs
// more than it gains (38 chunks of 2 to 9 over 1,500: 47 and 73 us with two), has the one of its mean,
// if that is at most 20.  Too few units (request, kv head) for the splits to fill the GPU want short
// rows (one request of four tokens: 2,000 keys 10 us, 8,192 21 and 30,000 57; the other kernel 20.5,
// 25 and 37).
FewRows fp8_few_rows(long long rows, int R, int hkv, int G, int bt_stride, int num_sms)
{
    const long long mean = (rows + R - 1) / R, units = static_cast<long long>(R) * hkv;
    FewRows f{0, 0};
    if (units >= 4 * num_sms) {
        if (mean <= 128) {
            f.first = mean <= 8 && G <= 8 ? 8 : 16;
            f.second = mean <= 24 && 24 / G > f.first / G && rows > f.first ? 24 : 0;
        }
        return f;
    }
    const int few = static_cast<int>((std::min<long long>(mean, 24) + 7) / 8 * 8);
    const bool filled = units * kD8Cluster >= 2 * num_sms;
    if (mean <= 20 && (filled || static_cast<long long>(few) * bt_stride <= 8192))
        f.first = few;
    return f;
}

cudaError_t launch_fp8_decode(const Fp8AttnArgs &a, int d, cudaStream_t s)
{
    const bool wide = a.Hq / a.Hkv > 8;
    if (d == 64)
        return wide ? launch_fp8_decode_t<64, 2, false>(a, s) : launch_fp8_decode_t<64, 1, false>(a, s);
    if (d == 128)
        return wide ? launch_fp8_decode_t<128, 2, false>(a, s) : launch_fp8_decode_t<128, 1, false>(a, s);
    return cudaErrorInvalidValue;
}

cudaError_t launch_fp8_few_rows(const Fp8AttnArgs &a, int rows, int d, cudaStream_t s)
{
    switch (rows | d) {
    case 8 | 64: return launch_fp8_decode_t<64, 1, true>(a, s);
    case 16 | 64: return launch_fp8_decode_t<64, 2, true>(a, s);
    case 24 | 64: return launch_fp8_decode_t<64, 3, true>(a, s);
    case 8 | 128: return launch_fp8_decode_t<128, 1, true>(a, s);
    case 16 | 128: return launch_fp8_decode_t<128, 2, true>(a, s);
    case 24 | 128: return launch_fp8_decode_t<128, 3, true>(a, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace zp
