// zp_fp8.cuh -- launch arguments and shared device code of the calls on an 8-bit
// cache: rows rounded into it (zp_fp8_append.cu) and the attention of few query
// rows over it (zp_fp8_decode.cu).  Internal: not part of the C ABI.
//
// A pool [num_blocks][Hkv][16][d] holds e4m3 numbers, and a scale [num_blocks][Hkv]
// goes with each of its slabs: value = scale * number.  Scales are powers of two
// from 2^-32 to 2^32, so a value has the three bits of mantissa that its number has, and
// numbers move to a larger scale by a rounding of the smallest of them alone.
#pragma once

#include <cuda_fp16.h>

#include "zp_chunk.cuh"

namespace zp {

constexpr int kFp8MinExp = -32, kFp8MaxExp = 32;  // of a scale

// starts null: request i brings the one row i.
struct Fp8KvArgs {
    uint8_t *kpool, *vpool;
    float *kscale, *vscale;
    const __nv_bfloat16 *k_new, *v_new;
    int64_t k_stride, v_stride;  // elements from a token to the next
    const int32_t *starts;
    int32_t total;
    const int32_t *tables;
    int32_t stride, num_rows;
    const int32_t *lengths;
    const int32_t *req_idx;
    int32_t R, Hkv, d, num_blocks;
    int32_t *sticky;
};

struct Fp8AttnArgs {
    const CUtensorMap *kmap, *vmap;
    const float *kscale, *vscale;
    const __nv_bfloat16 *q;
    int64_t q_stride;  // elements from a token's row of q to the next
    const int32_t *starts;  // of a chunk: its requests of more than `over` tokens
    int32_t total, over;
    int32_t follows;        // behind a kernel of the call that it may overlap
    int32_t last;           // of such kernels
    uint32_t *visible;      // their word; null where one kernel takes all requests
    const int32_t *tables;
    int32_t stride, num_rows;
    const int32_t *lengths;
    const int32_t *req_idx;
    int32_t R, Hkv, Hq, num_blocks;
    int32_t splits;       // per (request, kv head)
    int32_t groups;       // clusters they are
    float logit_scale;    // scale * log2(e)
    __nv_bfloat16 *out;
    float *part;          // [R][Hq][groups][d + 2] (o[d], m, l) of more than one group
    int32_t *sticky;
};

// The blocks of the requests with many query rows to bf16 (zp_fp8_widen.cu).
struct Fp8WidenArgs {
    const uint8_t *kpool, *vpool;
    const float *kscale, *vscale;
    __nv_bfloat16 *kwide, *vwide;  // [capacity][Hkv][16][d]
    int32_t *places;               // [R], out
    int32_t capacity;              // in blocks
    int32_t least;                 // tokens of a chunk whose request is widened
    const int32_t *starts;
    int32_t total;
    const int32_t *tables;
    int32_t stride, num_rows;
    const int32_t *lengths;
    const int32_t *req_idx;
    int32_t R, Hkv, d, num_blocks;
    int32_t *sticky;
};

// A request whose chunk has at least so many query rows (tokens times heads of a group) is
// widened.
constexpr int kWideRows = 1536;
constexpr int kWideMeanRows = 768;  // of a batch's requests, for any to be widened
constexpr size_t kWideBytes = 256u << 20;  // of widened blocks, at most
// Blocks of the workspace for a pool of num_blocks.
int fp8_wide_blocks(int num_blocks, int hkv, int d);

cudaError_t launch_fp8_widen(const Fp8WidenArgs &a, int sms, cudaStream_t s);
cudaError_t launch_fp8_append(const Fp8KvArgs &a, cudaStream_t s);
// Splits per (request, kv head) of a decode over `pairs` of them; *groups (at most 16):
// clusters that the splits are.
int fp8_decode_splits(long long pairs, int bt_stride, int num_sms, int *groups);
cudaError_t launch_fp8_decode(const Fp8AttnArgs &a, int d, cudaStream_t s);
// The rows (tokens times heads of a group; 8, 16 or 24) up to which a batch's requests are
// launch_fp8_few_rows's, in one or two launches; 0: none, all are launch_fp8_chunk_attn's.
struct FewRows {
    int first, second;
};
FewRows fp8_few_rows(long long rows, int R, int hkv, int G, int bt_stride, int num_sms);
cudaError_t launch_fp8_few_rows(const Fp8AttnArgs &a, int rows, int d, cudaStream_t s);
cudaError_t launch_fp8_chunk_attn(const ChunkAttnArgs &a, int d, int sms, cudaStream_t s);
// Once a device, before launch_fp8_chunk_attn.
cudaError_t prepare_fp8_chunk_attn(int d);
// The swizzled 2D map of an 8-bit pool: a box is one slab, 16 rows of d bytes, with
// the 128-byte swizzle (the 64-byte one for rows of 64).
bool encode_fp8_pool_map(CUtensorMap *map, const void *pool, int num_blocks, int hkv, int d);

#ifdef __CUDACC__

// Kernels of one call that overlap: a later one takes other requests than those before it, and may
// start as soon as the first has been let start, without the wait by which the work before the call
// becomes visible to a grid.  So the first kernel, behind its own wait, releases a word
// of the workspace, and every thread of a later one begins with an acquire of it: what was visible
// to the first then is to the later one, and by the fence to its TMA loads.  A thread that does not
// find the word waits for the first kernel's end instead.  The last kernel clears the word when all
// before it have ended.
__device__ __forceinline__ void say_visible(uint32_t *word)
{
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(word), "r"(1u) : "memory");
}
__device__ __forceinline__ void await_visible(const uint32_t *word)
{
    uint32_t said;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(said) : "l"(word) : "memory");
    if (!said)
        pdl_wait();
    asm volatile("fence.proxy.async.global;" ::: "memory");
}
__device__ __forceinline__ void clear_visible(uint32_t *word)
{
    asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(word), "r"(0u) : "memory");
}

// The exponent of the least scale that takes `most` (>= 0, or infinite) into 448.
__host__ __device__ __forceinline__ int fp8_scale_exp(uint32_t most_bits)
{
    // most = 1.m 2^E <= 448 2^e = 1.75 2^(e + 8)
    const int e = static_cast<int>(most_bits >> 23) - 127 - 8 + ((most_bits & 0x7fffffu) > 0x600000u);
    return e < kFp8MinExp ? kFp8MinExp : e > kFp8MaxExp ? kFp8MaxExp : e;
}

// 2^e for a normal result.
__host__ __device__ __forceinline__ uint32_t exp2_bits(int e)
{
    return static_cast<uint32_t>(e + 127) << 23;
}

// Two numbers to e4m3, the nearest (ties to even), magnitudes past 448 to 448, NaN to
// NaN: `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
    return v;
}

// Two e4m3 numbers as fp16 (exact), the low byte's in the low half.
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t v)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// D += A(16x16, row) * B(16x8, col), fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 numbers with 0 in place of NaN.
__device__ __forceinline__ uint32_t numbers4(uint32_t v)
{
    const uint32_t nan = ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // 0x80 a NaN
    return v & ~(nan | (nan - (nan >> 7)));
}

// 1 in place of NaN and 0 of the others.
__device__ __forceinline__ uint32_t ones4(uint32_t v)
{
    return (((v & 0x7f7f7f7fu) + 0x01010101u) >> 7 & 0x01010101u) * 0x38u;
}

// Byte offset of 16-byte chunk `ch` of row `row` in a slab of rows of D bytes as the
// pool's map leaves it in an aligned buffer (512 bytes for D = 64, 1024 for 128).
template <int D>
__device__ __forceinline__ uint32_t swz8(int row, int ch)
{
    return static_cast<uint32_t>(row * D +
                                 ((ch ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4));
}

#endif  // __CUDACC__

}  // namespace zp
