// The launches of the compression at admission without a GPU: a kernel's limit of shared memory,
// which all threads share, is set to the same whatever the call's sizes.
#include <cuda_runtime.h>

#include <cstdio>
#include <map>

static std::map<const void *, int> g_set;  // of a kernel
static int g_changed;
template <class F>
static cudaError_t fake_set(F *kernel, cudaFuncAttribute, int value)
{
    const auto at = g_set.emplace(reinterpret_cast<const void *>(kernel), value).first;
    g_changed += at->second != value;
    return cudaSuccess;
}
static cudaError_t fake_last_error() { return cudaSuccess; }  // (no launch succeeds here)
#define cudaFuncSetAttribute fake_set
#define cudaGetLastError fake_last_error
#include "zp_prefill.cu"

int main()
{
    using namespace zp;
    for (const int d : {64, 128})
        for (const int mt : {1, 2, 4})
            for (int tokens = 64; tokens <= kPrefillMaxTokens; tokens *= 2) {
                PrefillArgs a{};
                a.T_cap = tokens;
                a.NC = 1;
                if (launch_prefill(a, d, mt, 1, nullptr) != cudaSuccess)
                    return 1;
            }
    for (const auto &s : g_set)
        if (s.second > 227 * 1024)
            return 1;
    std::printf(g_changed ? "%d changes\n" : "ok\n", g_changed);
    return g_changed != 0;
}
