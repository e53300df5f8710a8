// The weights of the draws as the kernels form them, two at a time (weights()): to the bit those of
// weight(), and within 2^-40 of exp((l - M) / T).  argv[1]: host, or gpu for the device's.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <vector>

#include "zp_sample.cuh"

using namespace zp;

struct Case {
    WeightScale c;
    float M, l[2], T;
};

static unsigned long long g_state = 7;
static double rnd()  // [0, 1), the same on every machine
{
    g_state = g_state * 6364136223846793005ull + 1442695040888963407ull;
    return static_cast<double>(g_state >> 11) * 0x1p-53;
}

static std::vector<Case> cases()
{
    std::vector<Case> v;
    for (int n = 0; n < 400000; ++n) {
        Case x;
        // temperatures of all sizes, and those in use
        x.T = static_cast<float>(std::exp2(n % 3 ? 12 * rnd() - 6 : 200 * rnd() - 100));
        const double d = 1.4426950408889634 / static_cast<double>(x.T);
        x.c.ch = static_cast<float>(d);
        x.c.cl = static_cast<float>(d - static_cast<double>(x.c.ch));
        // a maximum up to a million times the temperature (but 2^126), or none, infinite ones
        x.M = static_cast<float>(std::min(x.T * std::exp2(40 * rnd() - 20), 0x1p126) *
                                 (rnd() < 0.5 ? -1 : 1));
        if (n % 50 == 0)
            x.M = 0.f;
        for (int k = 0; k < 2; ++k) {
            const double far = rnd() < 0.2 ? std::exp2(-40 * rnd()) : 60 * rnd();
            x.l[k] = static_cast<float>(x.M - x.T * far * 0.6931471805599453);
            const double what = rnd();
            x.l[k] = what < 0.01 ? x.M : what < 0.02 ? -INFINITY : what < 0.03 ? -3e38f : x.l[k];
            x.l[k] = std::min(x.l[k], x.M);
        }
        if (n % 97 == 0)
            x.M = x.l[n & 1] = INFINITY;
        v.push_back(x);
    }
    return v;
}

__global__ void weigh(const Case *v, int n, const uint64_t *table, uint64_t *w)
{
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n)
        weights(table, v[i].c, v[i].M, v[i].l[0], v[i].l[1], w[2 * i], w[2 * i + 1]);
}

int main(int argc, char **argv)
{
    static const WeightTable table;
    const std::vector<Case> v = cases();
    const int n = static_cast<int>(v.size());
    std::vector<uint64_t> w(2 * v.size());
    if (argc > 1 && !std::strcmp(argv[1], "gpu")) {
        Case *dv = nullptr;
        uint64_t *dt = nullptr, *dw = nullptr;
        if (cudaMalloc(&dv, sizeof(Case) * n) != cudaSuccess ||
            cudaMalloc(&dt, sizeof(table)) != cudaSuccess ||
            cudaMalloc(&dw, 16ull * n) != cudaSuccess ||
            cudaMemcpy(dv, v.data(), sizeof(Case) * n, cudaMemcpyHostToDevice) != cudaSuccess ||
            cudaMemcpy(dt, table.v, sizeof(table), cudaMemcpyHostToDevice) != cudaSuccess)
            return 2;
        weigh<<<(n + 255) / 256, 256>>>(dv, n, dt, dw);
        if (cudaMemcpy(w.data(), dw, 16ull * n, cudaMemcpyDeviceToHost) != cudaSuccess)
            return 2;
    } else {
        for (int i = 0; i < n; ++i)
            weights(table.v, v[i].c, v[i].M, v[i].l[0], v[i].l[1], w[2 * i], w[2 * i + 1]);
    }
    double worst = 0;
    long long positive = 0;
    for (int i = 0; i < 2 * n; ++i) {
        const Case &x = v[i / 2];
        const float l = x.l[i & 1];
        uint64_t same = l == x.M ? (1ull << kWeightBits) | 1 : 0;
        if (std::fabs(x.M) < INFINITY) {
            float h, lo;
            gap(x.M, l, h, lo);
            same = weight(table.v, x.c, h, lo);
            const long double y = (static_cast<long double>(x.M) - l) / x.T;
            worst = std::max(worst, static_cast<double>(fabsl(static_cast<long double>(w[i]) * 0x1p-44L -
                                                              expl(-y))));
        }
        positive += w[i] > 0;
        if (w[i] != same) {
            std::printf("M %a, l %a, T %a: %llx, not %llx\n", x.M, l, x.T,
                        static_cast<unsigned long long>(w[i]), static_cast<unsigned long long>(same));
            return 1;
        }
    }
    if (!(worst < 0x1p-40) || positive < n) {
        std::printf("off by %g, %lld above 0\n", worst, positive);
        return 1;
    }
    std::printf("ok\n");
    return 0;
}
