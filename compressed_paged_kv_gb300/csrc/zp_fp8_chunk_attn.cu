// zp_fp8_chunk_attn.cu -- the attention of chunks over an 8-bit cache.
#include "zp_chunk_attn.cuh"

namespace zp {

cudaError_t prepare_fp8_chunk_attn(int d)
{
    return d == 64 ? prepare_chunk_attn_t<64, true>() : prepare_chunk_attn_t<128, true>();
}

cudaError_t launch_fp8_chunk_attn(const ChunkAttnArgs &a, int d, int sms, cudaStream_t s)
{
    if (d == 64)
        return launch_chunk_attn_t<64, true>(a, sms, s);
    if (d == 128)
        return launch_chunk_attn_t<128, true>(a, sms, s);
    return cudaErrorInvalidValue;
}

}  // namespace zp
