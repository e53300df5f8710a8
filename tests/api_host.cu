// Host check of the C ABI's chunk calls and of the status, without a GPU: the
// entry points of zp_api.cu with the CUDA runtime and the launches replaced by
// functions that record what they are called with.
#include <cuda_runtime.h>

#include <cstdio>
#include <cstring>
#include <vector>

struct Clear {
    void *p;
    size_t n;
};
static std::vector<Clear> g_clears;
static int32_t g_sticky;
static int g_launches;

static cudaError_t fake_get_device(int *d)
{
    *d = 0;
    return cudaSuccess;
}
static cudaError_t fake_memcpy_async(void *to, const void *, size_t n, cudaMemcpyKind, cudaStream_t)
{
    std::memcpy(to, &g_sticky, n);
    return cudaSuccess;
}
static cudaError_t fake_memset_async(void *p, int, size_t n, cudaStream_t)
{
    g_clears.push_back({p, n});
    return cudaSuccess;
}
static cudaError_t fake_synchronize(cudaStream_t) { return cudaSuccess; }

#define cudaGetDevice fake_get_device
#define cudaMemcpyAsync fake_memcpy_async
#define cudaMemsetAsync fake_memset_async
#define cudaStreamSynchronize fake_synchronize
#include "zp_api.cu"

namespace zp {
cudaError_t launch_append_kv_chunk(const ChunkKvArgs &, cudaStream_t)
{
    ++g_launches;
    return cudaSuccess;
}
cudaError_t launch_chunk_attn(const ChunkAttnArgs &, int, int, cudaStream_t)
{
    ++g_launches;
    return cudaSuccess;
}
cudaError_t launch_verify_draft(const VerifyArgs &, bool, int, cudaStream_t)
{
    ++g_launches;
    return cudaSuccess;
}
bool encode_chunk_q_map(CUtensorMap *, const void *, int, int64_t, int, int, int) { return true; }
}  // namespace zp

#define CHECK(x)                                                 \
    do {                                                         \
        if (!(x)) {                                              \
            std::printf("%s, line %d: %s\n", what, __LINE__, #x); \
            return 1;                                            \
        }                                                        \
    } while (0)

// A status is read and cleared; nothing of a call that may be in flight on
// another stream is touched, whatever the code.
static int status()
{
    const char *what = "status";
    zp_cache c;
    int32_t words[64] = {};
    c.ws.sticky = words;
    c.ws.ca_arrived = reinterpret_cast<uint32_t *>(words + 8);
    c.num_sms = 4;
    for (const int32_t code : {ZP_OK, ZP_ERR_INVALID_ARG, ZP_ERR_DEVICE_CHECK, ZP_ERR_TIMEOUT}) {
        g_sticky = code;
        g_clears.clear();
        int32_t got = 1;
        CHECK(zp_cache_status(&c, nullptr, &got) == ZP_OK && got == code);
        CHECK(g_clears.size() == 1 && g_clears[0].p == c.ws.sticky && g_clears[0].n == 4);
    }
    return 0;
}

int main(int argc, char **argv)
{
    const char *what = argc > 1 ? argv[1] : "";
    int bad = 2;
    if (!std::strcmp(what, "status"))
        bad = status();
    if (!bad)
        std::printf("ok\n");
    return bad;
}
