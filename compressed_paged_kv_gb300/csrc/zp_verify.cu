// zp_verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers.
//
// Row first + j of the packed rows judges the chunk's token j + 1 (token 0 is
// the last accepted one).  With x that token, it is accepted when every token
// before it is and u * q(x) < p(x) (q = 1 when the draft has no
// probabilities).  The next token is drawn from the weights of the row the
// run ends at: max(p - q, 0) (p with x left out when there is no q) at a
// rejection, p after the last token; it is the lowest index whose running sum
// exceeds sample_u times the sum of all.
//
// u * q is exact in 64 bits.  The running sums decide between neighbouring
// tokens, of which there are as many as the vocabulary: an error of 2^-25 of
// the sum at every border gets about V * 2^-25 of the draws wrong (0.5 % at
// 150,000), so 32-bit sums will not do, and 64-bit additions run at a 64th of
// the 32-bit rate here.  p - q is therefore taken with its rounding error
// (both are fp32, the error is one too), and a thread adds up pairs of a
// 32-bit sum and the sum of its rounding errors (T. J. Dekker's and D. E.
// Knuth's error-free sums): about 46 bits.  The warps' sums are joined in 64
// bits.
//
// One cluster of kVfCtas CTAs a request.  A warp owns a contiguous run of the
// deciding row and reads it (of p and q) once, 16 bytes a lane; every CTA gets
// every warp's sum through distributed shared memory, and the warp that the
// level falls into goes through its own run a second time (out of L2) for the
// token.  Bound by the bytes of the deciding rows for large batches, and by
// the chain of dependent reads (offsets -> tokens -> their probabilities ->
// row -> sums -> run) for small ones.
#include "zp_chunk.cuh"

namespace zp {

namespace {

constexpr int kVfCtas = 8;    // of a cluster: the portable most
constexpr int kVfBatch = 4;   // vectors of p and of q a lane has in flight

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// 16 bytes as floats.
__device__ __forceinline__ void unpack(const uint4 &u, float (&v)[4])
{
    v[0] = __uint_as_float(u.x);
    v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z);
    v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack(const uint4 &u, float (&v)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// A row as 16-byte vectors of p: vector i holds elements first + i * VE ..; the
// first and the last one may lie partly outside.
template <class T>
struct Row {
    static constexpr int VE = 16 / sizeof(T);
    const T *p, *q;  // q: null when nothing is taken off
    int skip;        // a token left out, or -1
    int vocab, first, count;
    bool alike;      // q (if any) lies in its 16-byte vectors as p does

    __device__ __forceinline__ Row(const T *p_, const T *q_, int skip_, int vocab_)
        : p(p_), q(q_), skip(skip_), vocab(vocab_)
    {
        const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
        first = -mis;
        count = (mis + vocab + VE - 1) / VE;
        alike = !q || ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0;
    }

    // Weights w + e, exactly, of the elements e0 .. from p (in w) and q (in b).
    __device__ __forceinline__ void weigh(int e0, float (&w)[VE], const float (&b)[VE],
                                          float (&e)[VE]) const
    {
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            float d = w[k], r = 0.f;
            if (q) {
                d = w[k] - b[k];
                const float t = d - w[k];
                r = (w[k] - (d - t)) - (b[k] + t);
            }
            const bool some = d > 0.f && d < INFINITY && e0 + k != skip;
            w[k] = some ? d : 0.f;
            e[k] = some ? r : 0.f;
        }
    }

    // The same of vector i, element by element; 0 outside the row.
    __device__ __forceinline__ void weights(int i, float (&w)[VE], float (&e)[VE]) const
    {
        const int e0 = first + i * VE;
        float b[VE];
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            const bool in = e0 + k >= 0 && e0 + k < vocab;
            w[k] = in ? to_f32(p[e0 + k]) : 0.f;
            b[k] = in && q ? to_f32(q[e0 + k]) : 0.f;
        }
        weigh(e0, w, b, e);
    }
};

// (s, c) += w + e.
__device__ __forceinline__ void add_exact(float &s, float &c, float w, float e)
{
    const float t = s + w;
    const float z = t - s;
    c += ((s - (t - z)) + (w - z)) + e;
    s = t;
}

__device__ __forceinline__ double shfl_up(double v, int o)
{
    return __shfl_up_sync(0xffffffffu, v, o);
}

__device__ __forceinline__ double warp_scan(double v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = shfl_up(v, o);
        if (lane >= o)
            v += y;
    }
    return v;
}

__device__ __forceinline__ void st_dsmem_f64(uint32_t addr, double v)
{
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

}  // namespace

// NT threads a CTA.  Many requests: 128, so that the chains of many clusters
// run beside each other (1,024 threads an SM are 19 requests' CTAs of 8 warps
// ... 76 of 4); few: 512, so that one row has as many loads in flight.
template <class T, int NT>
__global__ void __cluster_dims__(kVfCtas, 1, 1) __launch_bounds__(NT, 1024 / NT)
    zp_verify_kernel(const VerifyArgs a)
{
    constexpr int VE = Row<T>::VE, kVfWarps = NT / 32;
    constexpr int kVfRuns = kVfCtas * kVfWarps;  // of a row, a warp each
    __shared__ double sums[2][kVfRuns];  // every run's, by the row's order; one set a pass
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, wi = threadIdx.x >> 5;
    const int rank = static_cast<int>(cluster_ctarank());
    const int i = blockIdx.x / kVfCtas;
    const int first = a.starts[i], end = a.starts[i + 1];
    const bool ok = first >= 0 && end >= first && end <= a.total;
    if (!ok || first == end) {  // the whole cluster alike
        if (!ok && rank == 0 && threadIdx.x == 0)
            set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
        return;
    }
    const T *target = static_cast<const T *>(a.target), *draft = static_cast<const T *>(a.draft);

    // the accepted run, 32 tokens at a time; every warp finds it for itself
    const int drafts = end - first - 1;
    int j = 0, x = -1;
    bool bad = false;
    for (; j < drafts; j += 32) {
        const int k = j + lane;
        bool stop = false, out = false;
        int tok = -1;
        if (k < drafts) {
            tok = a.tokens[first + k + 1];
            out = tok < 0 || tok >= a.vocab;
            stop = out;
            if (!out) {
                const size_t at = static_cast<size_t>(first + k) * a.prob_stride + tok;
                const double q = draft ? static_cast<double>(to_f32(draft[at])) : 1.0;
                stop = !(static_cast<double>(a.accept_u[first + k]) * q <
                         static_cast<double>(to_f32(target[at])));
            }
        }
        const unsigned m = __ballot_sync(0xffffffffu, stop);
        if (m) {
            const int l = __ffs(m) - 1;
            x = __shfl_sync(0xffffffffu, tok, l);
            bad = __shfl_sync(0xffffffffu, out, l);
            j += l;
            break;
        }
    }
    j = min(j, drafts);
    const size_t row_at = static_cast<size_t>(first + j) * a.prob_stride;
    const bool reject = j < drafts;

    if (rank == 0 && threadIdx.x == 0) {
        a.accepted[i] = j;
        if (bad) {
            a.next[i] = -1;
            set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
        }
        if (a.lengths) {
            const int row = a.req_idx ? a.req_idx[i] : i;
            if (row < 0 || row >= a.num_rows || a.lengths[row] < drafts + 1)
                set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
            else
                a.lengths[row] -= drafts - j;
        }
    }
    if (bad)
        return;
    cluster_arrive();  // paired below: the sums go to CTAs that have started

    for (int pass = 0; pass < 2; ++pass) {
        const bool left = pass == 0 && reject;  // what a rejection leaves; else p itself
        const Row<T> row(target + row_at, left && draft ? draft + row_at : nullptr,
                         left && !draft ? x : -1, a.vocab);
        // this warp's run of vectors
        const int per = (row.count + kVfRuns - 1) / kVfRuns;
        const int run = rank * kVfWarps + wi;
        const int v0 = min(row.count, run * per), v1 = min(row.count, v0 + per);
        float s = 0.f, c = 0.f;
        auto take = [&](float (&w)[VE], const float (&e)[VE]) {
#pragma unroll
            for (int k = 0; k < VE; ++k)
                add_exact(s, c, w[k], e[k]);
        };
        // the vectors that lie whole in the row, kVfBatch a lane at a time
        const int i0 = max(v0, 1), i1 = row.alike ? min(v1, row.count - 1) : i0;
        int v = i0 + lane;
        for (; v - lane + kVfBatch * 32 <= i1; v += kVfBatch * 32) {
            uint4 up[kVfBatch], uq[kVfBatch];
            const int e0 = row.first + v * VE;
#pragma unroll
            for (int u = 0; u < kVfBatch; ++u) {
                up[u] = ld_global_nc_v4(row.p + e0 + u * 32 * VE);
                if (row.q)
                    uq[u] = ld_global_nc_v4(row.q + e0 + u * 32 * VE);
            }
#pragma unroll
            for (int u = 0; u < kVfBatch; ++u) {
                float w[VE], b[VE], e[VE];
                unpack(up[u], w);
                unpack(uq[u], b);
                row.weigh(e0 + u * 32 * VE, w, b, e);
                take(w, e);
            }
        }
        for (; v < i1; v += 32) {
            float w[VE], b[VE], e[VE];
            const int e0 = row.first + v * VE;
            unpack(ld_global_nc_v4(row.p + e0), w);
            if (row.q)
                unpack(ld_global_nc_v4(row.q + e0), b);
            row.weigh(e0, w, b, e);
            take(w, e);
        }
        // and the others: the row's ends, or all of it
        if (row.alike) {
            if (lane == 0 && v0 == 0 && v1 > 0) {
                float w[VE], e[VE];
                row.weights(0, w, e);
                take(w, e);
            }
            if (lane == 1 && v0 < v1 && v1 == row.count && row.count > 1) {
                float w[VE], e[VE];
                row.weights(row.count - 1, w, e);
                take(w, e);
            }
        } else {
            for (v = v0 + lane; v < v1; v += 32) {
                float w[VE], e[VE];
                row.weights(v, w, e);
                take(w, e);
            }
        }
        double mine = static_cast<double>(s) + static_cast<double>(c);
#pragma unroll
        for (int o = 16; o; o >>= 1)
            mine += __shfl_xor_sync(0xffffffffu, mine, o);
        if (pass == 0)
            cluster_wait();
        if (lane < kVfCtas)
            st_dsmem_f64(dsmem_addr(&sums[pass][run], lane), mine);
        cluster_sync();
        // every warp: the runs' sums, kVfRuns / 32 a lane, and the level's run
        constexpr int PL = kVfRuns / 32;
        double part[PL], local = 0.0;
#pragma unroll
        for (int k = 0; k < PL; ++k) {
            part[k] = sums[pass][lane * PL + k];
            local += part[k];
        }
        const double upto = warp_scan(local, lane);
        const double all = __shfl_sync(0xffffffffu, upto, 31);
        if (!(all > 0.0)) {
            if (left)
                continue;  // p <= q everywhere: drawn from p
            if (rank == 0 && threadIdx.x == 0) {
                a.next[i] = -1;
                set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
            }
            return;
        }
        const double level = static_cast<double>(a.sample_u[i]) * all;
        double before = upto - local;
        int hit = -1, tail = -1;  // the run that passes the level; the last with any weight
        double hit_before = 0.0;
#pragma unroll
        for (int k = 0; k < PL; ++k) {
            if (part[k] > 0.0) {
                tail = lane * PL + k;
                if (hit < 0 && before + part[k] > level) {
                    hit = tail;
                    hit_before = before;
                }
            }
            before += part[k];
        }
        const unsigned m = __ballot_sync(0xffffffffu, hit >= 0);
        int target_run;
        if (m) {
            target_run = __shfl_sync(0xffffffffu, hit, __ffs(m) - 1);
            hit_before = __shfl_sync(0xffffffffu, hit_before, __ffs(m) - 1);
        } else {  // sample_u not below 1: the last token with weight
            target_run = __reduce_max_sync(0xffffffffu, tail);
            hit_before = -INFINITY;
        }
        if (target_run != run)
            return;
        // the token within this warp's run
        int last = -1;
        for (int vb = v0; vb < v1; vb += 32) {
            const int v = vb + lane;
            float w[VE], e[VE];
            double sum = 0.0;
            int top = -1;
            if (v < v1) {
                row.weights(v, w, e);
#pragma unroll
                for (int k = 0; k < VE; ++k) {
                    sum += static_cast<double>(w[k]) + static_cast<double>(e[k]);
                    if (w[k] > 0.f)
                        top = row.first + v * VE + k;
                }
            }
            const double incl = hit_before + warp_scan(sum, lane);
            const unsigned got = __ballot_sync(0xffffffffu, top >= 0 && incl > level);
            if (got) {
                const int l = __ffs(got) - 1;
                if (lane == l) {
                    double at = incl - sum;
                    int tok = top;
#pragma unroll
                    for (int k = 0; k < VE; ++k) {
                        at += static_cast<double>(w[k]) + static_cast<double>(e[k]);
                        if (w[k] > 0.f && at > level) {
                            tok = row.first + v * VE + k;
                            break;
                        }
                    }
                    a.next[i] = tok;
                }
                return;
            }
            last = max(last, __reduce_max_sync(0xffffffffu, top));
            hit_before = __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0)  // the level lies at the run's very end
            a.next[i] = last;
        return;
    }
}

template <class T, int NT>
static cudaError_t launch_verify_t(const VerifyArgs &a, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.R) * kVfCtas, 1, 1);
    cfg.blockDim = dim3(NT, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, zp_verify_kernel<T, NT>, a);
}

cudaError_t launch_verify_draft(const VerifyArgs &a, bool bf16, int sms, cudaStream_t s)
{
    // 512 threads a CTA while all clusters then run at once, two CTAs an SM
    const bool few = static_cast<long long>(a.R) * kVfCtas <= 2ll * sms;
    if (bf16)
        return few ? launch_verify_t<__nv_bfloat16, 512>(a, s)
                   : launch_verify_t<__nv_bfloat16, 128>(a, s);
    return few ? launch_verify_t<float, 512>(a, s) : launch_verify_t<float, 128>(a, s);
}

}  // namespace zp
