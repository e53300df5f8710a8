// Chunk calls over an 8-bit cache whose kernels overlap, without a GPU: the first kernel says that
// the work before the call is visible, the ones behind it heed that and the last one clears the word;
// a call of one kernel has no word; where a launch behind the first fails, the host clears it.
#include <cuda_runtime.h>

#include <cstdio>
#include <string>
#include <vector>

static int g_cleared;
static cudaError_t fake_get_device(int *d)
{
    *d = 0;
    return cudaSuccess;
}
static cudaError_t fake_memset(void *, int value, size_t bytes, cudaStream_t)
{
    g_cleared += value == 0 && bytes == 4;
    return cudaSuccess;
}
#define cudaGetDevice fake_get_device
#define cudaMemsetAsync fake_memset
#include "zp_api.cu"

struct Launch {
    bool few, follows, last;
    const uint32_t *word;
};
static std::vector<Launch> g_launches;
static size_t g_fails;  // the launch that fails, from 1 on

static cudaError_t launched(const Launch &l)
{
    g_launches.push_back(l);
    return g_launches.size() == g_fails ? cudaErrorInvalidValue : cudaSuccess;
}

namespace zp {
cudaError_t launch_fp8_few_rows(const Fp8AttnArgs &a, int, int, cudaStream_t)
{
    return launched({true, a.follows != 0, a.last != 0, a.visible});
}
cudaError_t launch_fp8_widen(const Fp8WidenArgs &, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_fp8_chunk_attn(const ChunkAttnArgs &a, int, int, cudaStream_t)
{
    return launched({false, false, false, a.visible});
}
cudaError_t launch_chunk_attn(const ChunkAttnArgs &a, int, int, cudaStream_t)
{
    return launched({false, false, false, a.visible});
}
bool encode_chunk_q_map(CUtensorMap *, const void *, int, int64_t, int, int, int) { return true; }
}  // namespace zp

#define CHECK(x)                                                                     \
    do {                                                                             \
        if (!(x)) {                                                                  \
            std::printf("R %d, total %d, G %d, fails %zu: line %d: %s\n", R, total, G, \
                        g_fails, __LINE__, #x);                                      \
            return 1;                                                                \
        }                                                                            \
    } while (0)

int main()
{
    uintptr_t at = 1 << 20;  // addresses that nothing reads
    auto take = [&](size_t bytes) {
        const uintptr_t p = at;
        at += (bytes + 31) / 32 * 32;
        return reinterpret_cast<void *>(p);
    };
    int seen[4] = {};
    for (const int G : {1, 4, 7, 16})
        for (const int R : {1, 4, 38, 76, 256, 512})
            for (int total = 1; total <= 40 * R; total += 1 + total / 9)
                for (g_fails = 0; g_fails <= 3; ++g_fails) {
                    zp_cache c;
                    c.L = 1;
                    c.Hkv = 8;
                    c.Hq = 8 * G;
                    c.d = 64;
                    c.b = 16;
                    c.num_blocks = 8;
                    c.num_sms = 152;
                    c.max_requests = 512;
                    c.fp8 = true;
                    for (std::vector<void *> *v : {&c.kpools, &c.vpools})
                        v->push_back(take(8 * 8 * 16 * 64));
                    for (std::vector<float *> *v : {&c.kscales, &c.vscales})
                        v->push_back(static_cast<float *>(take(8 * 8 * 4)));
                    c.ws.ca_visible = static_cast<uint32_t *>(take(4));
                    const size_t row = 2ull * c.Hq * c.d;
                    g_launches.clear();
                    g_cleared = 0;
                    const zp_status st = zp_paged_chunk_attn(
                        &c, 0, take(total * row), c.Hq * c.d, static_cast<int32_t *>(take(4 * 513)),
                        total, static_cast<int32_t *>(take(4 * 512 * 128)), 128, 512,
                        static_cast<int32_t *>(take(4 * 512)), nullptr, R, 1.f, take(total * row),
                        nullptr);
                    const size_t n = g_launches.size();
                    CHECK(n >= 1 && n <= 3);
                    CHECK(st == (g_fails >= 1 && g_fails <= n ? ZP_ERR_CUDA : ZP_OK));
                    const bool overlap = g_launches.back().few && (n > 1 || g_launches[0].word);
                    for (size_t i = 0; i < n; ++i) {
                        const Launch &l = g_launches[i];
                        CHECK(l.word == (overlap ? c.ws.ca_visible : g_launches[0].word));
                        CHECK(l.few || i == 0 || !g_launches[i - 1].few);  // the few rows' come last
                        CHECK(l.follows == (l.few && i > 0));
                    }
                    if (st == ZP_OK) {
                        ++seen[n];
                        CHECK((g_launches[0].word != nullptr) == (n > 1 && g_launches.back().few));
                        for (size_t i = 0; i < n; ++i)
                            CHECK(!g_launches[i].few || g_launches[i].last == (i + 1 == n));
                        CHECK(g_cleared == 0);
                    } else {
                        CHECK(g_cleared == (g_launches.back().follows ? 1 : 0));
                    }
                }
    if (!seen[1] || !seen[2] || !seen[3])
        return 1;
    std::printf("ok\n");
    return 0;
}
