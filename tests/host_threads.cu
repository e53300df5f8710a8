// Calls that two host threads make at once, each with its own handle and stream, of sizes that need
// different amounts of shared memory of the same kernel: every one is taken.  argv[1]: draws.
#include "zp.h"

#include <cuda_runtime.h>

#include <atomic>
#include <cstdio>
#include <cstring>
#include <thread>
#include <vector>

static void *zeros(size_t bytes)
{
    void *p = nullptr;
    if (cudaMalloc(&p, bytes) != cudaSuccess || cudaMemset(p, 0, bytes) != cudaSuccess)
        std::printf("no memory\n");
    return p;
}

static zp_cache *handle()
{
    const void *pools[2] = {zeros(16 * 64 * 2 * 8), zeros(16 * 64 * 2 * 8)};
    zp_cache_desc desc{};
    desc.num_layers = desc.num_kv_heads = desc.num_q_heads = desc.max_requests = 1;
    desc.head_dim = 64;
    desc.block_size = 16;
    desc.num_blocks = 8;
    desc.max_blocks_per_req = 2048;
    desc.k_pools = const_cast<void **>(pools);
    desc.v_pools = const_cast<void **>(pools + 1);
    zp_cache *c = nullptr;
    if (zp_cache_create(&desc, &c) != ZP_OK)
        std::printf("no handle\n");
    return c;
}

template <class Call>
static int at_once(Call first, Call second)
{
    std::atomic<int> refused{0};
    auto loop = [&](Call call) {
        cudaStream_t s;
        cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking);
        for (int k = 0; k < 20000; ++k) {
            refused += call(s) != ZP_OK;
            if (k % 500 == 499)
                cudaStreamSynchronize(s);
        }
        cudaStreamSynchronize(s);
    };
    cudaDeviceSynchronize();
    std::thread a(loop, first), b(loop, second);
    a.join();
    b.join();
    if (cudaDeviceSynchronize() != cudaSuccess)
        ++refused;
    return refused;
}

// One row of zeros: the token is floor(vocab / 2) at u = 0.5.
struct Draw {
    zp_cache *c;
    int32_t vocab, dtype;
    void *logits;
    float *u;
    int32_t *token;
    explicit Draw(int32_t v, int32_t t) : c(handle()), vocab(v), dtype(t)
    {
        logits = zeros(4 * static_cast<size_t>(v));
        u = static_cast<float *>(zeros(4));
        token = static_cast<int32_t *>(zeros(4));
        const float half = 0.5f;
        cudaMemcpy(u, &half, 4, cudaMemcpyHostToDevice);
    }
    zp_status operator()(cudaStream_t s) const
    {
        return zp_sample(c, logits, dtype, vocab, vocab, nullptr, nullptr, nullptr, nullptr, 1,
                         nullptr, u, 1, token, s);
    }
    int wrong() const
    {
        int32_t t = -1, st = -1;
        cudaMemcpy(&t, token, 4, cudaMemcpyDeviceToHost);
        return zp_cache_status(c, nullptr, &st) != ZP_OK || st != ZP_OK || t != vocab / 2;
    }
};

int main(int argc, char **argv)
{
    const char *what = argc > 1 ? argv[1] : "";
    int bad = 1;
    if (!std::strcmp(what, "draws")) {
        bad = 0;
        for (const int32_t type : {ZP_DTYPE_F32, ZP_DTYPE_BF16}) {
            const Draw small(500, type), large(300000, type);
            bad += at_once(small, large);
            bad += small.wrong() + large.wrong();
        }
    }
    if (!bad)
        std::printf("ok\n");
    else
        std::printf("%d calls refused or wrong\n", bad);
    return bad != 0;
}
