// zp_chunk_attn.cu -- the attention of chunks over a bf16 cache.
#include "zp_chunk_attn.cuh"

namespace zp {

size_t chunk_attn_part_floats(int d, int sms)
{
    return static_cast<size_t>(2 * sms) * (2 * kTile * (d + 2));
}

cudaError_t prepare_chunk_attn(int d)
{
    return d == 64 ? prepare_chunk_attn_t<64, false>() : prepare_chunk_attn_t<128, false>();
}

cudaError_t launch_chunk_attn(const ChunkAttnArgs &a, int d, int sms, cudaStream_t s)
{
    if (d == 64)
        return launch_chunk_attn_t<64, false>(a, sms, s);
    if (d == 128)
        return launch_chunk_attn_t<128, false>(a, sms, s);
    return cudaErrorInvalidValue;
}

}  // namespace zp
