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

// Once a device, before launch_sample: the most shared memory that any call needs.  (It is the
// kernels' own state, which calls from several threads share: a call does not set it.)
cudaError_t prepare_sample();
cudaError_t launch_sample(const SampleArgs &a, bool bf16, int sms, cudaStream_t s);

// ------------------------------------------------------------------ weights
// w = 2^-y, y = (M - l) log2(e) / T, as an odd whole number of 2^-44: sums of them are exact,
// whatever their order, up to 2^19 weights (M is the row's largest, w = 1).  Tokens are
// decided by sums of up to 10^5 weights, each a border that a random number may hit,
// so 2^-24 (fp32) gets several draws in a thousand wrong; and fp64 has a 64th of fp32's
// rate here.  So y is a pair of fp32 numbers, with
//     y = k / 1024 + g,  |g| <= 2^-11,     2^-y = 2^-(k / 1024) (1 - z + z^2/2 - z^3/6),
//     z = g ln 2, z^4/24 < 2^-50,
// the first factor from a table of the 1,024 fractions.  What is cut off below 2^-44 is
// half a unit in the mean, which the lowest bit, always set, makes up for.  The error is
// below 2^-40, 16 units: 5.6 from the table's number cut to 30 bits (2^-30 of |z| < 2^-11.5), 4
// from z in 2^-42 by two roundings, 2 from the shift and the lowest bit, 0.5 from the table, and
// less than 1 from the pair y.
constexpr int kWeightBits = 44;

struct WeightScale {
    float ch, cl;  // log2(e) / T as a pair
};

// The temperatures that are taken as they are: log2(e) / T, the range of gaps that have weight and
// the buckets over it, 64 T ln 2 and 8 log2(e) / T, are fp32 numbers.  Past 2^100 cl is a multiple of
// 2^-149, which puts y off by up to 2^-25 and a weight by 2^-24 of itself.
constexpr float kLeastTemp = 7.5231638452626401e-37f;  // 2^-120
constexpr float kMostTemp = 1.3292279957849159e36f;    // 2^120

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

constexpr float kSteps = 12288.f;   // 1.5 * 2^13: what added to p leaves multiples of 2^-10
constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: whole numbers
constexpr uint32_t kWholeBits = 0x4b400000u;
constexpr float kLn2 = 0.693147182f, kLn2Low = -1.90465421e-9f;

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

// The weight from p + (what follows 2^-11 of it as z): z in units of 2^-42.
__host__ __device__ __forceinline__ uint64_t weight_of_parts(const uint64_t *table, float p,
                                                             uint32_t t, int z)
{
    const uint64_t v = table[t & 1023];
    const int n = (t >> 10) & 63;
    const uint64_t w = v - static_cast<uint64_t>(
                               (static_cast<int64_t>(static_cast<int>(v >> 14)) * z) >> 28);
    return p < 48.f ? (w >> n) | 1 : 0;
}

// The weight at gap (h, lo).  0 past y = 48 and for what is no number.
__host__ __device__ __forceinline__ uint64_t weight(const uint64_t *table, const WeightScale &c,
                                                    float h, float lo)
{
    const float p = h * c.ch;
    const float e = fmaf(lo, c.ch, fmaf(h, c.cl, fmaf(h, c.ch, -p)));
    const float t = p + kSteps;
    const float g = p - (t - kSteps), gs = g + e, ge = e - (gs - g);
    const float zh = gs * kLn2;
    const float zl = fmaf(ge, kLn2, fmaf(gs, kLn2Low, fmaf(gs, kLn2, -zh)));
    const float s = fmaf(zh * zh, fmaf(zh, 0.166666667f, -0.5f), zl);
    // zh + s as a whole number of 2^-42, in two steps
    const float a = fmaf(zh, 8589934592.f, kWhole);  // 2^33
    const float b = fmaf(s + fmaf(a - kWhole, -1.16415322e-10f, zh), 4398046511104.f, kWhole);
    const uint32_t z = (static_cast<uint32_t>(bits_of(a)) << 9) + static_cast<uint32_t>(bits_of(b)) -
                       ((kWholeBits << 9) + kWholeBits);
    return weight_of_parts(table, p, static_cast<uint32_t>(bits_of(t)), static_cast<int>(z));
}

__host__ __device__ __forceinline__ float float_of(uint32_t x)
{
#ifdef __CUDA_ARCH__
    return __uint_as_float(x);
#else
    float v;
    __builtin_memcpy(&v, &x, 4);
    return v;
#endif
}

// Two fp32 numbers, each operation on both at once (on the host one after the other).
struct Two {
    uint64_t v;
};
__host__ __device__ __forceinline__ uint32_t low_bits(Two a) { return static_cast<uint32_t>(a.v); }
__host__ __device__ __forceinline__ uint32_t high_bits(Two a)
{
    return static_cast<uint32_t>(a.v >> 32);
}
__host__ __device__ __forceinline__ Two two(float x, float y)
{
    Two r;
#ifdef __CUDA_ARCH__
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
#else
    r.v = static_cast<uint64_t>(static_cast<uint32_t>(bits_of(y))) << 32 |
          static_cast<uint32_t>(bits_of(x));
#endif
    return r;
}
__host__ __device__ __forceinline__ Two two(float x) { return two(x, x); }
__host__ __device__ __forceinline__ Two operator+(Two a, Two b)
{
#ifdef __CUDA_ARCH__
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
#else
    return two(float_of(low_bits(a)) + float_of(low_bits(b)),
               float_of(high_bits(a)) + float_of(high_bits(b)));
#endif
}
__host__ __device__ __forceinline__ Two operator-(Two a, Two b)
{
#ifdef __CUDA_ARCH__
    Two r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
#else
    return two(float_of(low_bits(a)) - float_of(low_bits(b)),
               float_of(high_bits(a)) - float_of(high_bits(b)));
#endif
}
__host__ __device__ __forceinline__ Two operator*(Two a, Two b)
{
#ifdef __CUDA_ARCH__
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
#else
    return two(float_of(low_bits(a)) * float_of(low_bits(b)),
               float_of(high_bits(a)) * float_of(high_bits(b)));
#endif
}
__host__ __device__ __forceinline__ Two fma2(Two a, Two b, Two c)
{
#ifdef __CUDA_ARCH__
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
#else
    return two(fmaf(float_of(low_bits(a)), float_of(low_bits(b)), float_of(low_bits(c))),
               fmaf(float_of(high_bits(a)), float_of(high_bits(b)), float_of(high_bits(c))));
#endif
}

// y of two logits below a finite M: its fp32 value p and the rest e.
__host__ __device__ __forceinline__ void exponents(float M, const WeightScale &c, Two l, Two &p,
                                                   Two &e)
{
    const Two m = two(M), h = m - l, b = h - m, lo = (m - (h - b)) - (l + b);
    const Two ch = two(c.ch);
    p = h * ch;
    e = fma2(lo, ch, fma2(h, two(c.cl), fma2(h, ch, h * two(-c.ch))));
}

// The weights of two logits: weight() of each, to the bit.
__host__ __device__ __forceinline__ void weights(const uint64_t *table, const WeightScale &c,
                                                 float M, float l0, float l1, uint64_t &w0,
                                                 uint64_t &w1)
{
    if (fabsf(M) == INFINITY) {
        w0 = l0 == M ? (1ull << kWeightBits) | 1 : 0;
        w1 = l1 == M ? (1ull << kWeightBits) | 1 : 0;
        return;
    }
    Two p, e;
    exponents(M, c, two(l0, l1), p, e);
    const Two t = p + two(kSteps), g = p - (t - two(kSteps)), gs = g + e, ge = e - (gs - g);
    const Two ln2 = two(kLn2), zh = gs * ln2;
    const Two zl = fma2(ge, ln2, fma2(gs, two(kLn2Low), fma2(gs, ln2, gs * two(-kLn2))));
    const Two s = fma2(zh * zh, fma2(zh, two(0.166666667f), two(-0.5f)), zl);
    const Two whole = two(kWhole), a = fma2(zh, two(8589934592.f), whole);
    const Two b = fma2(s + fma2(a - whole, two(-1.16415322e-10f), zh), two(4398046511104.f), whole);
    constexpr uint32_t off = (kWholeBits << 9) + kWholeBits;
    w0 = weight_of_parts(table, float_of(low_bits(p)), low_bits(t),
                         static_cast<int>((low_bits(a) << 9) + low_bits(b) - off));
    w1 = weight_of_parts(table, float_of(high_bits(p)), high_bits(t),
                         static_cast<int>((high_bits(a) << 9) + high_bits(b) - off));
}

#endif  // __CUDACC__

}  // namespace zp
