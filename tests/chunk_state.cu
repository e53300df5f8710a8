// Chunk attention after a call of the handle that gave up a wait: such a call
// leaves some of its arrivals uncounted.  The test leaves them so itself, with
// another error recorded first, and the calls after it must give the first
// call's bits.  (One long row of few heads, cut over many CTAs.)
#include "zp_api.cu"

#include <cstdio>

#define CHECK(x)                                       \
    do {                                               \
        if (!(x)) {                                    \
            std::printf("line %d: %s\n", __LINE__, #x); \
            return 1;                                  \
        }                                              \
    } while (0)

int main()
{
    constexpr int Hkv = 2, Hq = 8, D = 128, N = 5, T = 6000, NB = (T + 15) / 16;
    const size_t pool = static_cast<size_t>(NB) * Hkv * 16 * D;
    const size_t rows = static_cast<size_t>(N) * Hq * D;
    auto values = [](size_t n, unsigned seed) {  // bf16 in about [-1, 1]
        std::vector<uint16_t> v(n);
        unsigned long long s = seed;
        for (auto &x : v) {
            s = s * 6364136223846793005ull + 1442695040888963407ull;
            const float f = static_cast<float>(static_cast<int>(s >> 40) - (1 << 23)) / (1 << 23);
            uint32_t u;
            std::memcpy(&u, &f, 4);
            x = static_cast<uint16_t>(u >> 16);
        }
        return v;
    };
    auto up = [](const void *p, size_t n) {
        void *d = nullptr;
        if (cudaMalloc(&d, n) != cudaSuccess ||
            cudaMemcpy(d, p, n, cudaMemcpyHostToDevice) != cudaSuccess)
            std::printf("no memory\n");
        return d;
    };
    const auto hk = values(pool, 1), hv = values(pool, 2), hq = values(rows, 3);
    void *k = up(hk.data(), 2 * pool), *v = up(hv.data(), 2 * pool), *q = up(hq.data(), 2 * rows);
    std::vector<int32_t> table(NB);
    for (int i = 0; i < NB; ++i)
        table[i] = NB - 1 - i;
    const int32_t len = T, offs[2] = {0, N};
    auto *dt = static_cast<int32_t *>(up(table.data(), 4 * NB));
    auto *dl = static_cast<int32_t *>(up(&len, 4)), *ds = static_cast<int32_t *>(up(offs, 8));
    std::vector<uint16_t> first(rows), got(rows, 7);
    void *out = up(got.data(), 2 * rows);

    zp_cache_desc desc{};
    desc.num_layers = 1;
    desc.num_kv_heads = Hkv;
    desc.num_q_heads = Hq;
    desc.head_dim = D;
    desc.block_size = 16;
    desc.num_blocks = NB;
    desc.max_requests = 1;
    desc.max_blocks_per_req = NB;
    desc.k_pools = &k;
    desc.v_pools = &v;
    zp_cache *c = nullptr;
    CHECK(zp_cache_create(&desc, &c) == ZP_OK);
    auto call = [&] {
        return zp_paged_chunk_attn(c, 0, q, Hq * D, ds, N, dt, NB, 1, dl, nullptr, 1, 0.0884f, out,
                                   nullptr);
    };
    auto status = [&] {
        int32_t st = 1;
        return zp_cache_status(c, nullptr, &st) == ZP_OK ? st : 1;
    };
    CHECK(call() == ZP_OK && status() == ZP_OK);
    CHECK(cudaMemcpy(first.data(), out, 2 * rows, cudaMemcpyDeviceToHost) == cudaSuccess);
    bool any = false;
    for (uint16_t x : first)
        any |= x != 0;
    CHECK(any);
    const std::vector<uint32_t> ones(2 * c->num_sms, 1);
    const int32_t code = ZP_ERR_DEVICE_CHECK;
    for (int rep = 0; rep < 6; ++rep) {
        uint32_t entered = 0;
        CHECK(cudaMemcpy(&entered, c->ws.ca_entered, 4, cudaMemcpyDeviceToHost) == cudaSuccess);
        CHECK(entered % c->num_sms == 0 && entered < 2u * c->num_sms);
        // the last call's set: the first when its numbers were below the CTAs of a call
        uint32_t *set = c->ws.ca_arrived + (entered == 0 ? 2 * c->num_sms : 0);
        CHECK(cudaMemcpy(set, ones.data(), 8 * c->num_sms, cudaMemcpyHostToDevice) == cudaSuccess);
        CHECK(cudaMemcpy(c->ws.sticky, &code, 4, cudaMemcpyHostToDevice) == cudaSuccess);
        CHECK(status() == ZP_ERR_DEVICE_CHECK);
        for (int i = 0; i <= rep; ++i) {
            CHECK(cudaMemset(out, 0, 2 * rows) == cudaSuccess);
            CHECK(call() == ZP_OK && status() == ZP_OK);
            CHECK(cudaMemcpy(got.data(), out, 2 * rows, cudaMemcpyDeviceToHost) == cudaSuccess);
            CHECK(got == first);
        }
    }
    zp_cache_destroy(c);
    std::printf("ok\n");
    return 0;
}
