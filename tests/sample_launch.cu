// The draws' launches without a GPU: what shared memory is asked for once, at a handle's creation,
// holds for every call, and no call asks again (it is the kernels' state, which threads share).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>
#include <map>

static int g_sets;
static std::map<const void *, size_t> g_set;  // of a kernel
template <class F>
static cudaError_t fake_set(F *kernel, cudaFuncAttribute attr, int value)
{
    if (attr != cudaFuncAttributeMaxDynamicSharedMemorySize || value > 227 * 1024)
        return cudaErrorInvalidValue;
    ++g_sets;
    g_set[reinterpret_cast<const void *>(kernel)] = static_cast<size_t>(value);
    return cudaSuccess;
}
static cudaLaunchConfig_t g_cfg;
static unsigned g_ctas;
template <class F, class... A>
static cudaError_t fake_launch(const cudaLaunchConfig_t *cfg, F *kernel, A...)
{
    g_cfg = *cfg;
    if (cfg->dynamicSmemBytes > g_set[reinterpret_cast<const void *>(kernel)])
        return cudaErrorInvalidValue;
    g_ctas = cfg->attrs[1].val.clusterDim.x;
    return cudaSuccess;
}
#define cudaFuncSetAttribute fake_set
#define cudaLaunchKernelEx fake_launch
#include "zp_sample.cu"

int main()
{
    using namespace zp;
    if (prepare_sample() != cudaSuccess || g_sets != 2 || g_set.size() != 2)
        return 1;
    for (int vocab = 1; vocab <= kSampleMaxVocab;
         vocab = vocab == kSampleMaxVocab ? vocab + 1 : std::min(vocab + vocab / 37 + 1, kSampleMaxVocab))
        for (const int R : {1, 2, 5, 38, 76, 152, 304, 1280, 1 << 24})
            for (const bool bf16 : {false, true}) {
                SampleArgs a{};
                a.vocab = vocab;
                a.R = R;
                if (launch_sample(a, bf16, 152, nullptr) != cudaSuccess || g_ctas < 1 || g_ctas > 8 ||
                    g_cfg.gridDim.x != g_ctas * R) {
                    std::printf("vocab %d, %d rows: %zu bytes, %u CTAs\n", vocab, R,
                                g_cfg.dynamicSmemBytes, g_ctas);
                    return 1;
                }
            }
    if (g_sets != 2)
        return 1;
    std::printf("ok\n");
    return 0;
}
