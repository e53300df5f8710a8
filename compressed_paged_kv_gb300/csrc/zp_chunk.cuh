// zp_chunk.cuh -- launch arguments and shared device code of the calls on a
// ragged chunk of new tokens: K/V rows written into the cache
// (zp_chunk_append.cu), attention over the cache (zp_chunk_attn.cu) and the
// verification of drafted tokens (zp_verify.cu).  Internal: not part of the
// C ABI.
//
// The chunk of request i is rows starts[i] .. starts[i+1]-1 of the packed
// tensors; its last token is the last of the request's lengths[row] tokens.
#pragma once

#include "zp_internal.cuh"

namespace zp {

struct ChunkKvArgs {
    __nv_bfloat16 *kpool, *vpool;
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

struct ChunkAttnArgs {
    const CUtensorMap *kmap;
    const CUtensorMap *vmap;
    const __nv_bfloat16 *kpool, *vpool, *q;
    int64_t q_stride;  // elements from a token of q to the next
    CUtensorMap qmap;  // q as [total][Hq][d]: boxes of 64 dims x a group's heads x a tile's tokens
    const int32_t *starts;
    int32_t total;
    const int32_t *tables;
    int32_t stride, num_rows;
    const int32_t *lengths;
    const int32_t *req_idx;
    int32_t R, Hkv, Hq, num_blocks;
    float logit_scale;  // scale * log2(e)
    __nv_bfloat16 *out;
    float *part;        // partial results of the items cut between CTAs
    uint32_t *arrived;  // [2][2 * SMs] of them that are written: two sets, used in turn
    uint32_t *entered;  // CTAs that have entered a call, modulo two calls'
    int32_t *sticky;
};

struct VerifyArgs {
    const int32_t *tokens;
    const int32_t *starts;
    int32_t total;
    const void *target, *draft;  // draft: null when the drafted tokens come without probabilities
    int32_t vocab;
    int64_t prob_stride;  // elements from a row to the next
    const float *accept_u, *sample_u;
    int32_t *lengths;  // null: not committed
    int32_t num_rows;
    const int32_t *req_idx;
    int32_t R;
    int32_t *accepted, *next;
    int32_t *sticky;
};

cudaError_t launch_append_kv_chunk(const ChunkKvArgs &a, cudaStream_t s);
cudaError_t launch_chunk_attn(const ChunkAttnArgs &a, int d, int sms, cudaStream_t s);
// Floats of ChunkAttnArgs::part for a GPU of `sms` SMs.
size_t chunk_attn_part_floats(int d, int sms);
// The map ChunkAttnArgs::qmap of a packed q (tokens `stride` elements apart).
bool encode_chunk_q_map(CUtensorMap *map, const void *q, int total, int64_t stride, int Hq, int G,
                        int d);
cudaError_t launch_verify_draft(const VerifyArgs &a, bool bf16, int sms, cudaStream_t s);
// Once a device, before launch_chunk_attn.
cudaError_t prepare_chunk_attn(int d);

#ifdef __CUDACC__

// One request's chunk: its first packed row, its tokens, its table row and
// cached length.
struct ChunkReq {
    int first, n, row, len;
};

// Reads and checks request i: true with n >= 1 when it has work; an empty
// chunk is no work (whatever its row and length are), and one whose offsets,
// row or length are out of range sets *bad.  The loads do not wait for the
// checks: a chain of two (or, with req_idx, three) of them costs most of a
// microsecond each.
template <class Args>
__host__ __device__ __forceinline__ bool chunk_request(const Args &a, int i, ChunkReq &c, bool *bad)
{
    c.row = a.req_idx ? a.req_idx[i] : i;
    const bool fits = c.row >= 0 && c.row < a.num_rows;
    c.len = a.lengths[fits ? c.row : 0];
    c.first = a.starts[i];
    const int end = a.starts[i + 1];
    c.n = end - c.first;
    const bool offsets = c.first >= 0 && end >= c.first && end <= a.total;
    *bad = !offsets || (c.n > 0 && !(fits && c.len >= c.n && c.len <= a.stride * kBlk));
    return !*bad && c.n > 0;
}

#endif  // __CUDACC__

}  // namespace zp
