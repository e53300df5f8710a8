// The word by which a chunk call's first kernel says that the work before the call is visible: 0
// after every call, whichever kernels it had, and one left behind changes no output.
#include "zp_api.cu"

#include <cstdio>

#define CHECK(x)                                                      \
    do {                                                              \
        if (!(x)) {                                                   \
            std::printf("batch %d: line %d: %s\n", which, __LINE__, #x); \
            return 1;                                                 \
        }                                                             \
    } while (0)

int main()
{
    constexpr int Hkv = 8, Hq = 32, D = 128, R = 80, W = 20, NB = R * W;
    int which = -1;
    auto up = [](const void *p, size_t n) {
        void *d = nullptr;
        if (cudaMalloc(&d, n) != cudaSuccess ||
            cudaMemcpy(d, p, n, cudaMemcpyHostToDevice) != cudaSuccess)
            std::printf("no memory\n");
        return d;
    };
    unsigned long long seed = 1;
    auto rnd = [&](unsigned n) {
        seed = seed * 6364136223846793005ull + 1442695040888963407ull;
        return static_cast<unsigned>(seed >> 33) % n;
    };
    const size_t pool = static_cast<size_t>(NB) * Hkv * 16 * D;
    std::vector<uint8_t> kv(pool);
    for (auto &x : kv)
        x = static_cast<uint8_t>((rnd(2) << 7) | (40 + rnd(24)));  // e4m3 numbers of 2^-2 to 2^0
    std::vector<float> ones(static_cast<size_t>(NB) * Hkv, 1.f);
    void *k = up(kv.data(), pool), *v = up(kv.data(), pool);
    float *ks = static_cast<float *>(up(ones.data(), 4 * ones.size()));
    float *vs = static_cast<float *>(up(ones.data(), 4 * ones.size()));
    zp_cache_desc desc{};
    desc.num_layers = 1;
    desc.num_kv_heads = Hkv;
    desc.num_q_heads = Hq;
    desc.head_dim = D;
    desc.block_size = 16;
    desc.num_blocks = NB;
    desc.max_requests = R;
    desc.max_blocks_per_req = W;
    desc.k_pools = &k;
    desc.v_pools = &v;
    zp_cache *c = nullptr;
    CHECK(zp_cache_create_fp8(&desc, &ks, &vs, &c) == ZP_OK);
    std::vector<int32_t> table(NB), length(R, 300);
    for (int i = 0; i < NB; ++i)
        table[i] = NB - 1 - i;
    auto *dt = static_cast<int32_t *>(up(table.data(), 4 * NB));
    auto *dl = static_cast<int32_t *>(up(length.data(), 4 * R));
    // one kernel; two; three; the two of few rows alone
    const int sizes[4][2] = {{60, 60}, {60, 1}, {9, 2}, {1, 0}};
    for (which = 0; which < 4; ++which) {
        std::vector<int32_t> starts{0};
        for (int i = 0; i < R; ++i)
            starts.push_back(starts.back() +
                             (which == 3 ? i < 6 : i % 5 ? sizes[which][1] : sizes[which][0]));
        const int total = starts.back();
        const size_t rows = static_cast<size_t>(total) * Hq * D;
        std::vector<uint16_t> q(rows), first(rows), got(rows, 7);
        for (auto &x : q)
            x = static_cast<uint16_t>((rnd(2) << 15) | (0x3e80 + rnd(256)));  // bf16 of 2^-2 to 2^0
        void *dq = up(q.data(), 2 * rows), *out = up(got.data(), 2 * rows);
        auto *ds = static_cast<int32_t *>(up(starts.data(), 4 * (R + 1)));
        for (int rep = 0; rep < 6; ++rep) {
            const uint32_t left = rep == 3;
            if (rep == 2 || rep == 3)
                CHECK(cudaMemcpy(c->ws.ca_visible, &left, 4, cudaMemcpyHostToDevice) == cudaSuccess);
            CHECK(cudaMemset(out, 0, 2 * rows) == cudaSuccess);
            CHECK(zp_paged_chunk_attn(c, 0, dq, Hq * D, ds, total, dt, W, R, dl, nullptr, R, 0.0884f,
                                      out, nullptr) == ZP_OK);
            int32_t st = 1;
            CHECK(zp_cache_status(c, nullptr, &st) == ZP_OK && st == ZP_OK);
            uint32_t word = 7;
            CHECK(cudaMemcpy(&word, c->ws.ca_visible, 4, cudaMemcpyDeviceToHost) == cudaSuccess);
            const bool one = which == 0;  // no kernel has the word
            CHECK(word == (one && rep >= 3 ? 1u : 0u));
            CHECK(cudaMemcpy(got.data(), out, 2 * rows, cudaMemcpyDeviceToHost) == cudaSuccess);
            if (rep == 0)
                first = got;
            CHECK(got == first);
        }
        const uint32_t none = 0;
        CHECK(cudaMemcpy(c->ws.ca_visible, &none, 4, cudaMemcpyHostToDevice) == cudaSuccess);
        bool any = false;
        for (uint16_t x : first)
            any |= x != 0;
        CHECK(any);
    }
    zp_cache_destroy(c);
    std::printf("ok\n");
    return 0;
}
