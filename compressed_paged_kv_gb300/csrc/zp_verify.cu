// zp_verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers.
//
// Row first + j of the packed rows judges the chunk's token j + 1 (token 0 is
// the last accepted one).  With x that token, it is accepted when every token
// before it is and u * q(x) < p(x) (q = 1 when the draft has no
// probabilities).  The next token is drawn from the weights of the row the
// run ends at: max(p - q, 0) (p with x left out when there is no q) at a
// rejection, p after the last token; it is the lowest index whose running sum
// exceeds sample_u times the sum of all.  u * q is exact in 64 bits, and the
// sums are held in 64 bits, so that neither a border nor the order of the
// additions decides a token.
#include "zp_chunk.cuh"

namespace zp {

namespace {

constexpr int kVfThreads = 1024;

__device__ __forceinline__ double prob(const float *p, size_t i) { return p[i]; }
__device__ __forceinline__ double prob(const __nv_bfloat16 *p, size_t i)
{
    return __bfloat162float(p[i]);
}

}  // namespace

template <class T>
__global__ void __launch_bounds__(kVfThreads) zp_verify_kernel(const VerifyArgs a)
{
    const int i = blockIdx.x, tid = threadIdx.x;
    const int first = a.starts[i], end = a.starts[i + 1];
    if (first == end)
        return;
    if (first < 0 || end < first || end > a.total) {
        if (tid == 0)
            set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
        return;
    }
    const T *target = static_cast<const T *>(a.target), *draft = static_cast<const T *>(a.draft);
    const int drafts = end - first - 1;
    int j = 0;
    bool bad = false;
    int x = -1;  // the rejected token
    for (; j < drafts; ++j) {
        x = a.tokens[first + j + 1];
        if (x < 0 || x >= a.vocab) {
            bad = true;
            break;
        }
        const size_t at = (size_t)(first + j) * a.prob_stride + x;
        const double q = draft ? prob(draft, at) : 1.0;
        if (!(static_cast<double>(a.accept_u[first + j]) * q < prob(target, at)))
            break;
        x = -1;
    }
    const T *prow = target + (size_t)(first + j) * a.prob_stride;
    const T *qrow = draft && j < drafts ? draft + (size_t)(first + j) * a.prob_stride : nullptr;
    bool skip_x = !draft && x >= 0;
    auto weight = [&](int v) {
        double w = prob(prow, v);
        if (qrow)
            w -= prob(qrow, v);
        if (skip_x && v == x)
            w = 0.0;
        return w > 0.0 && w < INFINITY ? w : 0.0;
    };
    // thread t sums a contiguous piece; an exclusive scan over the pieces
    __shared__ double sums[kVfThreads];
    __shared__ int found;
    const int per = (a.vocab + kVfThreads - 1) / kVfThreads;
    const int lo = min(a.vocab, tid * per), hi = min(a.vocab, lo + per);
    double before, all;
    for (;;) {
        double s = 0.0;
        for (int v = lo; v < hi; ++v)
            s += weight(v);
        sums[tid] = s;
        if (tid == 0)
            found = 0x7fffffff;
        __syncthreads();
        before = all = 0.0;
        for (int t = 0; t < kVfThreads; ++t) {
            if (t == tid)
                before = all;
            all += sums[t];
        }
        if (all > 0.0 || (!qrow && !skip_x))
            break;
        qrow = nullptr;  // p <= q everywhere: drawn from p
        skip_x = false;
        __syncthreads();
    }
    const double level = static_cast<double>(a.sample_u[i]) * all;
    for (int v = lo; v < hi; ++v) {
        const double w = weight(v);
        before += w;
        if (w > 0.0 && before > level) {
            atomicMin(&found, v);
            break;
        }
    }
    __syncthreads();
    if (tid == 0) {
        const bool ok = !bad && found != 0x7fffffff;
        a.accepted[i] = j;
        a.next[i] = ok ? found : -1;
        if (!ok)
            set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
        if (a.lengths) {
            const int row = a.req_idx ? a.req_idx[i] : i;
            if (row < 0 || row >= a.num_rows || a.lengths[row] < drafts + 1)
                set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
            else
                a.lengths[row] -= drafts - j;
        }
    }
}

cudaError_t launch_verify_draft(const VerifyArgs &a, bool bf16, cudaStream_t s)
{
    if (bf16)
        zp_verify_kernel<__nv_bfloat16><<<a.R, kVfThreads, 0, s>>>(a);
    else
        zp_verify_kernel<float><<<a.R, kVfThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace zp
