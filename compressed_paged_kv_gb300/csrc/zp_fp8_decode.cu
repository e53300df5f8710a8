// zp_fp8_decode.cu -- attention of single tokens over an 8-bit paged cache:
// zp_paged_decode_attn of such a cache.
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
// Grid (request, kv head, split), four warps a CTA.  A CTA owns a contiguous range of
// `bps` blocks; a warp takes every fourth pair of them through its own ring of
// kStages pairs (one TMA box a slab).  Fragments come by ldmatrix: a matrix of 8 keys x 16
// bytes gives a lane four neighbouring dims of a key, so q's fragments are laid out to
// match; for V, the transposed matrix gives a lane two dims of two keys, which a byte
// permutation turns into the pairs of keys that the product takes (even and odd dims as
// two tiles).  Warps join in shared memory, splits in a second kernel.
#include "zp_fp8.cuh"

namespace zp {

namespace {

constexpr int kD8Warps = 4;
constexpr int kD8Threads = kD8Warps * 32;
constexpr int kD8Stages = 3;   // of a pair of blocks, K and V
constexpr float kTop = 14.f;   // log2 of the largest p

template <int D>
struct D8Smem {
    static constexpr int SLAB = kBlk * D;
    static constexpr int STAGE = 4 * SLAB;  // K of two blocks, V of two blocks
    static constexpr int STAGES = kD8Warps * kD8Stages * STAGE;
    static constexpr int MERGE = kD8Warps * 16 * (D + 2) * 4;  // reuses the stages
    static constexpr int off_bar = STAGES > MERGE ? STAGES : MERGE;
    static constexpr int BYTES = off_bar + kD8Warps * kD8Stages * 8;
    static constexpr int ALLOC = BYTES + 1024;
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(kD8Threads, 2)
    zp_fp8_decode_kernel(const __grid_constant__ Fp8AttnArgs a)
{
    pdl_wait();
    using S = D8Smem<D>;
    constexpr int KS = D / 16;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + S::off_bar);

    const int tid = threadIdx.x, lane = tid & 31, wi = tid >> 5;
    const int r = blockIdx.x, h = blockIdx.y, split = blockIdx.z;
    const int G = a.Hq / a.Hkv;
    int row = 0, len = 0;
    bool live = true;  // a row with an output
    if (a.starts) {    // one token of a chunk, by its packed row
        int lo = 0, hi = a.R;
        while (hi - lo > 1) {
            const int m = (lo + hi) / 2;
            if (a.starts[m] <= r)
                lo = m;
            else
                hi = m;
        }
        ChunkReq c;
        bool bad = false;
        live = chunk_request(a, lo, c, &bad) && r >= c.first && r < c.first + c.n;
        if (live) {
            row = c.row;
            len = c.len - c.n + (r - c.first) + 1;
        }
        if (r == 0 && h == 0 && split == 0)
            for (int i = tid; i < a.R; i += kD8Threads) {
                chunk_request(a, i, c, &bad);
                if (bad)
                    set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
            }
    } else {
        row = a.req_idx ? a.req_idx[r] : r;
        const bool row_ok = row >= 0 && row < a.num_rows;
        len = row_ok ? a.lengths[row] : 0;
        if (!row_ok || len < 0 || len > a.stride * kBlk) {
            if (tid == 0 && split == 0 && h == 0)
                set_error(a.sticky, row_ok ? ZP_ERR_DEVICE_CHECK : ZP_ERR_INVALID_ARG);
            len = 0;
            row = 0;
        }
    }
    if (!live) {
        pdl_launch_dependents();
        return;
    }
    const int nblk = (len + kBlk - 1) / kBlk;
    const int b_begin = split * a.bps;
    const int b_end = min(nblk, b_begin + a.bps);

    if (tid < kD8Warps * kD8Stages)
        mbar_init(&bars[tid], 1);
    if (tid == 0)
        fence_mbar_init();
    __syncthreads();

    // this warp's pairs of blocks: wi, wi + 4, .. of the range
    const int pairs = b_end > b_begin ? (b_end - b_begin + 1) / 2 : 0;
    const int my_n = pairs > wi ? (pairs - wi + kD8Warps - 1) / kD8Warps : 0;
    uint8_t *my_stage = sm + wi * kD8Stages * S::STAGE;
    uint64_t *my_bar = bars + wi * kD8Stages;
    const int32_t *trow = a.tables + static_cast<size_t>(row) * a.stride;

    // block ids and scales of 16 pairs, a block a lane, and of the 16 after them
    auto block_of = [&](int i) { return b_begin + 2 * (wi + kD8Warps * (i + (lane >> 1))) + (lane & 1); };
    auto load_id = [&](int i) {
        const int b = block_of(i);
        int id = b < b_end ? trow[b] : 0;
        if (id < 0 || id >= a.num_blocks) {
            set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
            id = 0;
        }
        return id;
    };
    auto scale_at = [&](const float *s, int id) { return s[static_cast<size_t>(id) * a.Hkv + h]; };
    int id = load_id(0), id_next = 0;

    auto issue = [&](int i, int ids) {
        const int l = (i & 15) * 2;
        const int y0 = (__shfl_sync(0xffffffffu, ids, l) * a.Hkv + h) * kBlk;
        const int y1 = (__shfl_sync(0xffffffffu, ids, l + 1) * a.Hkv + h) * kBlk;
        if (lane == 0) {
            const bool two = b_begin + 2 * (wi + kD8Warps * i) + 1 < b_end;
            const int s = i % kD8Stages;
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
    for (int i = 0; i < my_n && i < kD8Stages; ++i)
        issue(i, id);
    float ks = scale_at(a.kscale, id), vs = scale_at(a.vscale, id), ks_next = 0.f, vs_next = 0.f;

    // q's fragments: rows g and g + 8, dims 16 c + 4 t .. + 3 of each 16-byte chunk
    uint32_t qa[KS][4];
    float fr[2];  // what a logit is multiplied by, but for ks
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int g = (lane >> 2) + hh * 8;
        const __nv_bfloat16 *src =
            a.q + r * a.q_stride + (h * G + min(g, G - 1)) * D + (lane & 3) * 4;
        uint2 u[KS];
        uint32_t most = 0;  // the largest finite magnitude's bits
#pragma unroll
        for (int c = 0; c < KS; ++c) {
            u[c] = make_uint2(0u, 0u);
            if (g < G)
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
        fr[hh] = a.logit_scale * __uint_as_float(exp2_bits(-e1)) * __uint_as_float(exp2_bits(-e2));
#pragma unroll
        for (int c = 0; c < KS; ++c) {
            qa[c][hh] = pack_f16x2(__uint_as_float(u[c].x << 16) * f1 * f2,
                                   __uint_as_float(u[c].x & 0xffff0000u) * f1 * f2);
            qa[c][2 + hh] = pack_f16x2(__uint_as_float(u[c].y << 16) * f1 * f2,
                                       __uint_as_float(u[c].y & 0xffff0000u) * f1 * f2);
        }
    }

    float m_run[2] = {-1e30f, -1e30f};
    float l_run[2] = {0.f, 0.f};
    float o[KS][8];  // dims 16 c + 4 t + {0, 2 | 1, 3} of row g, then of g + 8: two tiles
#pragma unroll
    for (int c = 0; c < KS; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            o[c][e] = 0.f;
    bool ok = true;
    const int mi = lane >> 3;

    for (int i = 0; i < my_n; ++i) {
        const int s = i % kD8Stages;
        const int b0 = b_begin + 2 * (wi + kD8Warps * i);
        const bool two = b0 + 1 < b_end;
        const int tok0 = b0 * kBlk;
        const int l = (i & 15) * 2;
        const float ks0 = __shfl_sync(0xffffffffu, ks, l), ks1 = __shfl_sync(0xffffffffu, ks, l + 1);
        const float vs0 = __shfl_sync(0xffffffffu, vs, l), vs1 = __shfl_sync(0xffffffffu, vs, l + 1);
        if ((i & 15) == 0 && i + 16 < my_n)
            id_next = load_id(i + 16);
        if ((i & 15) == 8 && i + 8 < my_n) {
            ks_next = scale_at(a.kscale, id_next);
            vs_next = scale_at(a.vscale, id_next);
        }
        ok &= mbar_wait(&my_bar[s], (i / kD8Stages) & 1);
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

        // S of 32 keys: tiles of 8 keys; a matrix of tile nt, chunk c: a lane holds dims
        // 4 t .. 4 t + 3 of key g
        float sacc[4][4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sacc[nt][e] = 0.f;
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
            if (blk && !two)
                break;
#pragma unroll
            for (int c = 0; c < KS; c += 2) {
                // matrices: keys 0-7 of chunks c, c + 1, then keys 8-15
                uint32_t kr[4];
                ldsm_x4(kb + blk * S::SLAB + swz8<D>((mi >> 1) * 8 + (lane & 7), c + (mi & 1)), kr);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int cc = c + (x & 1), nt = blk * 2 + (x >> 1);
                    mma_f16(sacc[nt], qa[cc][0], qa[cc][1], qa[cc][2], qa[cc][3],
                            f16x2_of_e4m3(kr[x]), f16x2_of_e4m3(kr[x] >> 16));
                }
            }
        }
        const float lv0 = log2f(vs0), lv1 = log2f(vs1);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = nt * 8 + (lane & 3) * 2 + (e & 1);
                const float v =
                    fmaf(sacc[nt][e], fr[e >> 1] * (nt < 2 ? ks0 : ks1), nt < 2 ? lv0 : lv1);
                sacc[nt][e] = key < kBlk * (two ? 2 : 1) && tok0 + key < len ? v : -INFINITY;
            }
        const float iv0 = 1.f / vs0, iv1 = two ? 1.f / vs1 : 0.f;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            float mx = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
                mx = fmaxf(mx, fmaxf(sacc[nt][hh * 2], sacc[nt][hh * 2 + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float m_new = fmaxf(m_run[hh], mx);
            const float corr = ex2_approx(m_run[hh] - m_new);
            m_run[hh] = m_new;
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                o[c][hh * 2] *= corr;
                o[c][hh * 2 + 1] *= corr;
                o[c][4 + hh * 2] *= corr;
                o[c][4 + hh * 2 + 1] *= corr;
            }
            const float at = m_new - kTop;
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                sacc[nt][hh * 2] = ex2_approx(sacc[nt][hh * 2] - at);
                sacc[nt][hh * 2 + 1] = ex2_approx(sacc[nt][hh * 2 + 1] - at);
            }
            const float s0 = (sacc[0][hh * 2] + sacc[0][hh * 2 + 1]) +
                             (sacc[1][hh * 2] + sacc[1][hh * 2 + 1]);
            const float s1 = (sacc[2][hh * 2] + sacc[2][hh * 2 + 1]) +
                             (sacc[3][hh * 2] + sacc[3][hh * 2 + 1]);
            l_run[hh] = fmaf(l_run[hh], corr, fmaf(s0, iv0, two ? s1 * iv1 : 0.f));
        }
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
            if (blk && !two)
                break;
            const uint32_t p0 = pack_f16x2(sacc[blk * 2][0], sacc[blk * 2][1]);
            const uint32_t p1 = pack_f16x2(sacc[blk * 2][2], sacc[blk * 2][3]);
            const uint32_t p2 = pack_f16x2(sacc[blk * 2 + 1][0], sacc[blk * 2 + 1][1]);
            const uint32_t p3 = pack_f16x2(sacc[blk * 2 + 1][2], sacc[blk * 2 + 1][3]);
#pragma unroll
            for (int c = 0; c < KS; c += 2) {
                // matrices: keys 0-7 and 8-15 of chunk c, then of c + 1
                uint32_t vr[4];
                ldsm_x4_t(vb + blk * S::SLAB + swz8<D>((mi & 1) * 8 + (lane & 7), c + (mi >> 1)),
                          vr);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    // bytes: key 2 t (dims 2 g, 2 g + 1), key 2 t + 1 (the same)
                    const uint32_t lo = __byte_perm(vr[2 * x], 0, 0x3120);
                    const uint32_t hi = __byte_perm(vr[2 * x + 1], 0, 0x3120);
                    float(&even)[4] = *reinterpret_cast<float(*)[4]>(&o[c + x][0]);
                    float(&odd)[4] = *reinterpret_cast<float(*)[4]>(&o[c + x][4]);
                    mma_f16(even, p0, p1, p2, p3, f16x2_of_e4m3(lo), f16x2_of_e4m3(hi));
                    mma_f16(odd, p0, p1, p2, p3, f16x2_of_e4m3(lo >> 16), f16x2_of_e4m3(hi >> 16));
                }
            }
        }
        __syncwarp();
        if (i + kD8Stages < my_n) {
            fence_proxy_async_smem();
            __syncwarp();
            issue(i + kD8Stages, ((i + kD8Stages) ^ i) & 16 ? id_next : id);
        }
        if ((i & 15) == 15) {
            id = id_next;
            ks = ks_next;
            vs = vs_next;
        }
    }
    if (!ok && lane == 0)
        set_error(a.sticky, ZP_ERR_TIMEOUT);
    pdl_launch_dependents();  // the combine kernel may be scheduled
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        l_run[hh] += __shfl_xor_sync(0xffffffffu, l_run[hh], 1);
        l_run[hh] += __shfl_xor_sync(0xffffffffu, l_run[hh], 2);
    }
    __syncthreads();  // every stage consumed: reuse the area for the merge

    float *mrg = reinterpret_cast<float *>(sm);  // [warp][16][D + 2]
    {
        float *mine = mrg + wi * 16 * (D + 2);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int rr = (lane >> 2) + hh * 8;
            if ((lane & 3) == 0) {
                mine[rr * (D + 2) + D] = m_run[hh];
                mine[rr * (D + 2) + D + 1] = l_run[hh];
            }
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                float *to = mine + rr * (D + 2) + c * 16 + (lane & 3) * 4;
                to[0] = o[c][hh * 2];
                to[2] = o[c][hh * 2 + 1];
                to[1] = o[c][4 + hh * 2];
                to[3] = o[c][4 + hh * 2 + 1];
            }
        }
    }
    __syncthreads();
    for (int idx = tid; idx < G * D; idx += kD8Threads) {
        const int g = idx / D, c = idx - g * D;
        float M = -1e30f;
#pragma unroll
        for (int w2 = 0; w2 < kD8Warps; ++w2)
            M = fmaxf(M, mrg[(w2 * 16 + g) * (D + 2) + D]);
        float L = 0.f, O = 0.f;
#pragma unroll
        for (int w2 = 0; w2 < kD8Warps; ++w2) {
            const float *src = mrg + (w2 * 16 + g) * (D + 2);
            const float f = exp2f(src[D] - M);
            L += src[D + 1] * f;
            O += src[c] * f;
        }
        const size_t hq = static_cast<size_t>(r) * a.Hq + h * G + g;
        if (a.splits == 1) {
            a.out[hq * D + c] = __float2bfloat16_rn(L == 0.f ? 0.f : O / L);
        } else {
            float *p = a.part + (hq * a.splits + split) * (D + 2);
            p[c] = O;
            if (c == 0) {
                p[D] = M;
                p[D + 1] = L;
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(D) zp_fp8_combine_kernel(const Fp8AttnArgs a)
{
    pdl_wait();
    const int rh = blockIdx.x;  // token * Hq + hq
    const int c = threadIdx.x;
    const float *base = a.part + static_cast<size_t>(rh) * a.splits * (D + 2);
    float M = -1e30f;
    for (int s = 0; s < a.splits; ++s)
        M = fmaxf(M, base[s * (D + 2) + D]);
    float L = 0.f, O = 0.f;
    for (int s = 0; s < a.splits; ++s) {
        const float f = exp2f(base[s * (D + 2) + D] - M);
        L += base[s * (D + 2) + D + 1] * f;
        O += base[s * (D + 2) + c] * f;
    }
    a.out[static_cast<size_t>(rh) * D + c] = __float2bfloat16_rn(L == 0.f ? 0.f : O / L);
}

template <int D>
static cudaError_t launch_fp8_decode_t(const Fp8AttnArgs &a, cudaStream_t s)
{
    using Sm = D8Smem<D>;
    cudaError_t err = cudaFuncSetAttribute(zp_fp8_decode_kernel<D>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, Sm::ALLOC);
    if (err != cudaSuccess)
        return err;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const unsigned tokens = static_cast<unsigned>(a.starts ? a.total : a.R);
    cfg.gridDim = dim3(tokens, static_cast<unsigned>(a.Hkv), static_cast<unsigned>(a.splits));
    cfg.blockDim = dim3(kD8Threads, 1, 1);
    cfg.dynamicSmemBytes = Sm::ALLOC;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, zp_fp8_decode_kernel<D>, a);
    if (err != cudaSuccess || a.splits == 1)
        return err;
    cfg.gridDim = dim3(tokens * static_cast<unsigned>(a.Hq), 1, 1);
    cfg.blockDim = dim3(D, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, zp_fp8_combine_kernel<D>, a);
}

cudaError_t launch_fp8_decode(const Fp8AttnArgs &a, int d, cudaStream_t s)
{
    if (d == 64)
        return launch_fp8_decode_t<64>(a, s);
    if (d == 128)
        return launch_fp8_decode_t<128>(a, s);
    return cudaErrorInvalidValue;
}

}  // namespace zp
