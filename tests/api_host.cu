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

// Outputs that share memory with inputs or with each other are refused before
// any launch, those that lie right beside them are not.  Memory is a line of
// addresses that nothing reads.
struct Line {
    uintptr_t at = 1 << 20;
    template <class T>
    T *take(size_t bytes)
    {
        T *p = reinterpret_cast<T *>(at);
        at += (bytes + 31) / 32 * 32;
        return p;
    }
};

static int shared()
{
    const char *what = "shared";
    zp_cache c;
    c.L = 2;
    c.Hkv = 2;
    c.Hq = 4;
    c.d = 64;
    c.b = 16;
    c.num_blocks = 8;
    c.max_requests = 4;
    const size_t pool = 2ull * c.num_blocks * c.Hkv * c.b * c.d;
    Line m;
    for (int l = 0; l < 2; ++l) {
        c.kpools.push_back(m.take<void>(pool));
        c.vpools.push_back(m.take<void>(pool));
    }
    constexpr int R = 3, rows = 4, stride = 8, total = 16, V = 64;
    // every array of the three calls
    int32_t *starts = m.take<int32_t>(4 * (R + 1)), *tables = m.take<int32_t>(4 * rows * stride);
    int32_t *lengths = m.take<int32_t>(4 * rows), *req_idx = m.take<int32_t>(4 * 4);
    const size_t q_stride = 512, q_bytes = 2 * ((total - 1) * q_stride + c.Hq * c.d);
    uint8_t *q = m.take<uint8_t>(q_bytes);
    const size_t out_bytes = 2ull * total * c.Hq * c.d;
    uint8_t *out = m.take<uint8_t>(out_bytes);
    uint8_t *k = m.take<uint8_t>(2ull * total * c.Hkv * c.d);
    uint8_t *v = m.take<uint8_t>(2ull * total * c.Hkv * c.d);
    int32_t *tokens = m.take<int32_t>(4 * total), *acc = m.take<int32_t>(4 * 4);
    int32_t *next = m.take<int32_t>(4 * 4);
    float *p = m.take<float>(4 * total * V), *dp = m.take<float>(4 * total * V);
    float *au = m.take<float>(4 * total), *su = m.take<float>(4 * 4);

    auto refused = [](zp_status st) {
        const bool ok = st == ZP_ERR_INVALID_ARG && g_launches == 0;
        g_launches = 0;
        return ok;
    };
    auto launched = [](zp_status st) {
        const bool ok = st == ZP_OK && g_launches == 1;
        g_launches = 0;
        return ok;
    };
    auto attn = [&](void *o, const int32_t *s, const int32_t *t, const int32_t *l,
                    const int32_t *r, int layer = 0) {
        return zp_paged_chunk_attn(&c, layer, q, q_stride, s, total, t, stride, rows, l, r, R, 1.0f,
                                   o, nullptr);
    };
    auto at = [](void *base, size_t by) {
        return static_cast<void *>(static_cast<uint8_t *>(base) + by);
    };
    CHECK(launched(attn(out, starts, tables, lengths, req_idx)));
    CHECK(launched(attn(out, starts, tables, lengths, nullptr)));
    for (void *base : {c.kpools[0], c.vpools[0]}) {
        CHECK(refused(attn(base, starts, tables, lengths, req_idx)));
        CHECK(refused(attn(at(base, pool - 32), starts, tables, lengths, req_idx)));
    }
    CHECK(launched(attn(c.kpools[1], starts, tables, lengths, req_idx)));  // another layer's
    CHECK(refused(attn(c.kpools[1], starts, tables, lengths, req_idx, 1)));
    CHECK(refused(attn(q, starts, tables, lengths, req_idx)));
    CHECK(refused(attn(at(q, q_bytes / 32 * 32 - 32), starts, tables, lengths, req_idx)));
    // an index array whose first, or last, word lies in the output
    auto in = [&](size_t by) { return static_cast<int32_t *>(at(out, by)); };
    for (size_t by : {size_t(0), out_bytes - 4}) {
        CHECK(refused(attn(out, in(by), tables, lengths, req_idx)));
        CHECK(refused(attn(out, starts, in(by), lengths, req_idx)));
        CHECK(refused(attn(out, starts, tables, in(by), req_idx)));
        CHECK(refused(attn(out, starts, tables, lengths, in(by))));
    }
    CHECK(refused(attn(out, in(0) - R, tables, lengths, req_idx)));
    CHECK(refused(attn(out, starts, in(0) - rows * stride + 1, lengths, req_idx)));
    CHECK(refused(attn(out, starts, tables, in(0) - rows + 1, req_idx)));
    CHECK(refused(attn(out, starts, tables, lengths, in(0) - R + 1)));
    CHECK(launched(attn(out, in(0) - R - 1, in(0) - rows * stride, in(0) - rows, in(0) - R)));
    CHECK(launched(attn(out, in(out_bytes), in(out_bytes), in(out_bytes), in(out_bytes))));

    auto append = [&](const void *kn, const void *vn, const int32_t *s, const int32_t *t,
                      const int32_t *l, const int32_t *r) {
        return zp_append_kv_chunk(&c, 0, kn, 128, vn, 128, s, total, t, stride, rows, l, r, R,
                                  nullptr);
    };
    CHECK(launched(append(k, v, starts, tables, lengths, req_idx)));
    for (void *base : {c.kpools[0], c.vpools[0]})
        for (size_t by : {size_t(0), pool - 16}) {
            auto *w = static_cast<int32_t *>(at(base, by));
            CHECK(refused(append(w, v, starts, tables, lengths, req_idx)));
            CHECK(refused(append(k, w, starts, tables, lengths, req_idx)));
            CHECK(refused(append(k, v, w, tables, lengths, req_idx)));
            CHECK(refused(append(k, v, starts, w, lengths, req_idx)));
            CHECK(refused(append(k, v, starts, tables, w, req_idx)));
            CHECK(refused(append(k, v, starts, tables, lengths, w)));
        }
    CHECK(launched(append(c.kpools[1], c.vpools[1], starts, tables, lengths, nullptr)));

    auto verify = [&](int32_t *a_, int32_t *n_, int32_t *l_, const int32_t *r_) {
        return zp_verify_draft(&c, tokens, starts, total, p, dp, ZP_DTYPE_F32, V, V, au, su, l_,
                               rows, r_, R, a_, n_, nullptr);
    };
    CHECK(launched(verify(acc, next, lengths, req_idx)));
    CHECK(launched(verify(acc, next, nullptr, nullptr)));
    CHECK(refused(verify(acc, acc + 2, lengths, req_idx)));
    CHECK(launched(verify(acc, acc + 3, lengths, req_idx)));
    CHECK(refused(verify(acc, next, acc, req_idx)));
    CHECK(refused(verify(acc, next, lengths, acc)));
    CHECK(launched(verify(acc, next, nullptr, acc)));  // not read without lengths
    for (void *base : {static_cast<void *>(tokens + total - 1), static_cast<void *>(starts + R),
                       static_cast<void *>(p), static_cast<void *>(dp + total * V - 1),
                       static_cast<void *>(au), static_cast<void *>(su + R - 1)}) {
        CHECK(refused(verify(static_cast<int32_t *>(base), next, lengths, req_idx)));
        CHECK(refused(verify(acc, static_cast<int32_t *>(base), lengths, req_idx)));
        CHECK(refused(verify(acc, next, static_cast<int32_t *>(base), req_idx)));
    }
    return 0;
}

// Packed rows and vocabularies of a verification up to 2^30.
static int limits()
{
    const char *what = "limits";
    zp_cache c;
    c.max_requests = 4;
    auto array = [](int i) { return reinterpret_cast<int32_t *>(uintptr_t(i) << 48); };
    auto verify = [&](int32_t total, int32_t vocab) {
        g_launches = 0;
        return zp_verify_draft(&c, array(1), array(2), total, array(3), nullptr, ZP_DTYPE_F32,
                               vocab, vocab, reinterpret_cast<float *>(array(4)),
                               reinterpret_cast<float *>(array(5)), nullptr, 0, nullptr, 1,
                               array(6), array(7), nullptr);
    };
    const int32_t most = 1 << 30;
    CHECK(verify(most, 1) == ZP_OK && g_launches == 1);
    CHECK(verify(4, most) == ZP_OK && g_launches == 1);
    for (int32_t over : {most + 1, 0x7fffffff - 31, 0x7fffffff}) {
        CHECK(verify(over, 1) == ZP_ERR_UNSUPPORTED && g_launches == 0);
        CHECK(verify(4, over) == ZP_ERR_UNSUPPORTED && g_launches == 0);
    }
    return 0;
}

int main(int argc, char **argv)
{
    const char *what = argc > 1 ? argv[1] : "";
    int bad = 2;
    if (!std::strcmp(what, "status"))
        bad = status();
    else if (!std::strcmp(what, "shared"))
        bad = shared();
    else if (!std::strcmp(what, "limits"))
        bad = limits();
    if (!bad)
        std::printf("ok\n");
    return bad;
}
