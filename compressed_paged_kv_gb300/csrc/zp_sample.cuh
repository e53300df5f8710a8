// zp_sample.cuh -- launch arguments and the weights of zp_sample and
// zp_token_probs (zp_sample.cu).  Internal: not part of the C ABI.
#pragma once

#include "zp_internal.cuh"

namespace zp {

struct SampleArgs {
    const void *logits;
    int32_t vocab;
    int64_t stride;             // elements from a row to the next
    const float *temperature;   // these four of a table row, each nullable
    const int32_t *top_k;
    const float *top_p, *min_p;
    int32_t num_rows;
    const int32_t *req_idx;
    int32_t R;                  // rows of logits
    const float *u;             // tokens: random numbers
    int32_t *tokens;            // null: probabilities are wanted
    void *probs;
    int32_t prob_bf16;
    int64_t prob_stride;
    int32_t *sticky;
};

// Vocabulary limit: a row lies in the shared memory of eight CTAs.
constexpr int kSampleMaxVocab = 352 * 1024;

cudaError_t launch_sample(const SampleArgs &a, bool bf16, int sms, cudaStream_t s);

// ------------------------------------------------------------------ weights
// w = 2^-y, y = (M - l) log2(e) / T, as a whole number of 2^-44: sums of them are exact,
// whatever their order, up to 2^19 weights (M is the row's largest, w = 1).  Tokens are
// decided by sums of up to 10^5 weights, each a border that a random number may hit,
// so 2^-24 (fp32) gets several draws in a thousand wrong; and fp64 has a 64th of fp32's
// rate here.  So y is a pair of fp32 numbers, with
//     y = k / 1024 + g,  |g| <= 2^-11,     2^-y = 2^-(k / 1024) (1 - z + z^2/2 - z^3/6),
//     z = g ln 2, z^4/24 < 2^-50,
// the first factor from a table of the 1,024 fractions.  The error is below 2^-41.
constexpr int kWeightBits = 44;

struct WeightScale {
    float ch, cl;  // log2(e) / T as a pair
};

struct WeightTable {
    uint64_t v[1024];
    constexpr WeightTable() : v()
    {
        // roots[i] = 2^(-1 / 2^(i+1)) by Newton's iteration for the square root
        double roots[10] = {};
        double x = 0.5;
        for (int i = 0; i < 10; ++i) {
            double r = x;
            for (int n = 0; n < 40; ++n)
                r = 0.5 * (r + x / r);
            roots[i] = x = r;
        }
        for (int k = 0; k < 1024; ++k) {
            double p = 1.0;
            for (int i = 0; i < 10; ++i)
                if (k >> (9 - i) & 1)
                    p *= roots[i];
            v[k] = static_cast<uint64_t>(p * 17592186044416.0 + 0.5);  // 2^44
        }
    }
};

#ifdef __CUDACC__

__host__ __device__ __forceinline__ int nearest_int(float x)
{
#ifdef __CUDA_ARCH__
    return __float2int_rn(x);
#else
    return static_cast<int>(__builtin_rintf(x));
#endif
}

__host__ __device__ __forceinline__ int bits_of(float x)
{
#ifdef __CUDA_ARCH__
    return __float_as_int(x);
#else
    int v;
    __builtin_memcpy(&v, &x, 4);
    return v;
#endif
}

// M - l as a pair (D. E. Knuth's error-free sum); 0 at the maximum itself, even an
// infinite one.
__host__ __device__ __forceinline__ void gap(float M, float l, float &h, float &lo)
{
    h = M - l;
    const float b = h - M;
    lo = (M - (h - b)) - (l + b);
    if (l == M)
        h = lo = 0.f;
}

// The same for gap (h, lo).  0 past y = 48 and for what is no number.
__host__ __device__ __forceinline__ uint64_t weight(const uint64_t *table, const WeightScale &c,
                                                    float h, float lo)
{
    const float p = h * c.ch;
    if (!(p < 48.f))
        return 0;
    const float e = fmaf(lo, c.ch, fmaf(h, c.cl, fmaf(h, c.ch, -p)));
    const float t = p + 12288.f;  // 1.5 * 2^13: p to a multiple of 2^-10
    const int k = bits_of(t) - 0x46400000;
    const float g = p - (t - 12288.f), gs = g + e, ge = e - (gs - g);
    const float zh = gs * 0.693147182f;  // ln 2 = 0.693147182 - 1.90465421e-9
    const float zl = fmaf(ge, 0.693147182f, fmaf(gs, -1.90465421e-9f, fmaf(gs, 0.693147182f, -zh)));
    const float s = zl - zh * zh * fmaf(zh, -0.166666667f, 0.5f);
    const int z = nearest_int(zh * 4398046511104.f) + nearest_int(s * 4398046511104.f);  // 2^42
    const uint64_t v = table[k & 1023];
    const int n = k >> 10;
    const uint64_t w = v - static_cast<uint64_t>(
                               (static_cast<int64_t>(static_cast<int>(v >> 14)) * z) >> 28);
    return (w + ((1ull << n) >> 1)) >> n;
}

#endif  // __CUDACC__

}  // namespace zp
