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
// (both are fp32, the error is one too), and every sum is a pair of fp32 numbers,
// the second one what the first has lost (T. J. Dekker's and D. E. Knuth's
// error-free sums): about 46 bits.  (With the sums of warps and CTAs joined in 64
// bits the joins alone took 10 us of a call.)
//
// One cluster of CTAs a request.  A warp owns a contiguous run of the deciding
// row and reads it (of p and q) once, 16 bytes a lane and 2 kVfBatch of them under
// way, leaving its lanes' sums in shared memory now and then; every CTA gets
// every warp's sum through distributed shared memory, and the warp that the
// level falls into finds the stretch of its run from the sums it left, reads
// that a second time (out of L2) and finds the token.  Bound by the bytes of
// the deciding rows for large batches (256 requests of 151,936 fp32 p and q: 218
// MB in 48.7 us = 4.5 TB/s, 0.66 of the copy peak; of bf16 38.8 us; the clusters
// of rejected tokens read twice as much as the others), and by the chain of
// dependent reads (offsets -> tokens -> their probabilities -> row -> sums ->
// stretch) for small ones (one request of 32,000: 6.7 us).
#include "zp_chunk.cuh"

namespace zp {

namespace {

constexpr int kVfCtas = 8;    // of a cluster, at most: the portable most
constexpr int kVfBatch = 4;   // vectors of p and of q a lane has in flight
constexpr int kVfMarks = 32;  // sums left by the warps of a CTA, together

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

// Two fp32 numbers, added or subtracted at once.
__device__ __forceinline__ uint64_t pack2(float x, float y)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b)
{
    uint64_t v;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ float low2(uint64_t v)
{
    return __uint_as_float(static_cast<uint32_t>(v));
}
__device__ __forceinline__ float high2(uint64_t v)
{
    return __uint_as_float(static_cast<uint32_t>(v >> 32));
}

__device__ __forceinline__ void cp_async16(uint32_t to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A row as 16-byte vectors of p: vector i holds elements first + i * VE ..; the
// first and the last one may lie partly outside.
template <class T>
struct Row {
    static constexpr int VE = 16 / sizeof(T);
    const T *p, *q;  // q: null when nothing is taken off
    int skip;        // a token left out, or -1
    int vocab, first, count;
    int lo, hi;      // the vectors that lie whole in the row and that q (if any) has alike

    __device__ __forceinline__ Row(const T *p_, const T *q_, int skip_, int vocab_)
        : p(p_), q(q_), skip(skip_), vocab(vocab_)
    {
        const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
        first = -mis;
        count = (mis + vocab + VE - 1) / VE;
        lo = mis ? 1 : 0;
        hi = first + count * VE == vocab ? count : count - 1;
        if (q && ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15))
            hi = 0;
    }

    // Weights w + e, exactly, of the elements e0 .. from p (in w) and, with Q, q
    // (in b).  Only p > q counts, where (p - d) - q is the error of d = p - q.
    template <bool Q>
    __device__ __forceinline__ void weigh(int e0, float (&w)[VE], const float (&b)[VE],
                                          float (&e)[VE]) const
    {
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            const float d = Q ? w[k] - b[k] : w[k];
            const bool some = d > 0.f && d < INFINITY && (Q || e0 + k != skip);
            e[k] = Q && some ? (w[k] - d) - b[k] : 0.f;
            w[k] = some ? d : 0.f;
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
        if (q)
            weigh<true>(e0, w, b, e);
        else
            weigh<false>(e0, w, b, e);
    }

    // The vectors v, v + 32, .. (kVfBatch of them) of a row with lo < hi, zeros
    // outside lo .. hi - 1: `take` gets each one's number and bits of p and q.
    template <bool Q, class F>
    __device__ __forceinline__ void batch(int v, F take) const
    {
        uint4 up[kVfBatch], uq[kVfBatch];
#pragma unroll
        for (int u = 0; u < kVfBatch; ++u) {
            const int at = first + min(max(v + u * 32, lo), hi - 1) * VE;
            up[u] = ld_global_nc_v4(p + at);
            uq[u] = Q ? ld_global_nc_v4(q + at) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < kVfBatch; ++u) {
            const int i = v + u * 32;
            if (i < lo || i >= hi)
                up[u] = uq[u] = make_uint4(0u, 0u, 0u, 0u);
            take(u, up[u], uq[u]);
        }
    }

    // The weights of vector i from its bits, every one tested.
    template <bool Q>
    __device__ __forceinline__ void weights_of(int i, const uint4 &up, const uint4 &uq,
                                               float (&w)[VE], float (&e)[VE]) const
    {
        float b[VE];
        unpack(up, w);
        if (Q)
            unpack(uq, b);
        weigh<Q>(first + i * VE, w, b, e);
    }

    // Adds the weights of vector i, from its bits, to the two sums (s, c).  For
    // finite numbers: others make the sums infinite or NaN.
    template <bool Q>
    __device__ __forceinline__ void add_fast(int i, const uint4 &up, const uint4 &uq, uint64_t &s,
                                             uint64_t &c) const
    {
        float w[VE], b[VE];
        unpack(up, w);
        if (Q) {
            unpack(uq, b);
#pragma unroll
            for (int k = 0; k < VE; ++k)  // q where p exceeds it, else p: nothing left
                b[k] = fminf(b[k], w[k]);
        } else {
#pragma unroll
            for (int k = 0; k < VE; ++k)
                w[k] = fmaxf(w[k], 0.f);
            const unsigned at = static_cast<unsigned>(skip - (first + i * VE));
            if (at < static_cast<unsigned>(VE) && skip >= 0) {
#pragma unroll
                for (int k = 0; k < VE; ++k)
                    w[k] = k == static_cast<int>(at) ? 0.f : w[k];
            }
        }
#pragma unroll
        for (int k = 0; k < VE; k += 2) {
            uint64_t d = pack2(w[k], w[k + 1]);
            if (Q) {
                const uint64_t pq = d, b2 = pack2(b[k], b[k + 1]);
                d = sub2(pq, b2);
                c = add2(c, sub2(sub2(pq, d), b2));
            }
            const uint64_t t = add2(s, d), z = sub2(t, s);
            c = add2(c, add2(sub2(s, sub2(t, z)), sub2(d, z)));
            s = t;
        }
    }

    // The same of the vectors v0 + lane, + 32, .. below v1, through this lane's ring
    // of 2 kVfBatch vectors, of p or of p and q: a copy is always under way, where a
    // batch's loads wait for its additions (256 requests 51.3 -> 48.7 us).  `ends` and
    // `mark` are called after each kVfBatch vectors.  A lane reads what it copied
    // itself, so its own waits are enough.
    template <bool Q, class E, class M>
    __device__ __forceinline__ void stream(uint4 *ring, int v0, int v1, int lane, uint64_t &s,
                                           uint64_t &c, E ends, M mark) const
    {
        constexpr int DEPTH = Q ? kVfBatch : 2 * kVfBatch;
        const uint32_t at = smem_u32(ring);
        auto fetch = [&](int k, int stage) {  // vector k of the lane
            const int v = v0 + lane + k * 32;
            if (v >= lo && v < hi && v < v1) {
                const int e0 = first + v * VE;
                cp_async16(at + stage * 512, p + e0);
                if (Q)
                    cp_async16(at + (DEPTH + stage) * 512, q + e0);
            }
            cp_async_commit();
        };
#pragma unroll
        for (int k = 0; k < DEPTH; ++k)
            fetch(k, k);
        int n = 0;
#pragma unroll 1
        for (int v = v0; v < v1; v += kVfBatch * 32, ++n) {
            const int half = Q ? 0 : (n & 1) * kVfBatch;
#pragma unroll
            for (int u = 0; u < kVfBatch; ++u) {
                cp_async_wait<DEPTH - 1>();
                const int i = v + u * 32 + lane;
                uint4 up = make_uint4(0u, 0u, 0u, 0u), uq = up;
                if (i >= lo && i < hi) {
                    up = ring[(half + u) * 32];
                    if (Q)
                        uq = ring[(DEPTH + half + u) * 32];
                }
                add_fast<Q>(i, up, uq, s, c);
                fetch(n * kVfBatch + u + DEPTH, half + u);
            }
            ends(v);
            mark(n);
        }
        cp_async_wait<0>();
    }

    // The same of any vectors below `end`, those outside with weight 0.
    template <class F>
    __device__ __forceinline__ void ragged(int v, int end, F take) const
    {
#pragma unroll 1
        for (int u = 0; u < kVfBatch; ++u, v += 32) {
            float w[VE], e[VE];
            if (v < end) {
                weights(v, w, e);
            } else {
#pragma unroll
                for (int k = 0; k < VE; ++k)
                    w[k] = e[k] = 0.f;
            }
            take(u, w, e);
        }
    }
};

// (s, c) += w + e, none of them below 0 but e.
__device__ __forceinline__ void add_exact(float &s, float &c, float w, float e)
{
    const float t = s + w;
    c += (fminf(s, w) - (t - fmaxf(s, w))) + e;
    s = t;
}

// h + l, h the nearest fp32 number to it.
struct Pair {
    float h, l;
};

__device__ __forceinline__ Pair normal(float h, float l)  // |l| well below |h|, or h = 0
{
    const float t = h + l;
    return {t, l - (t - h)};
}

__device__ __forceinline__ Pair operator+(const Pair &a, const Pair &b)
{
    const float t = a.h + b.h, z = t - a.h;
    return normal(t, ((a.h - (t - z)) + (b.h - z)) + (a.l + b.l));
}

__device__ __forceinline__ bool operator>(const Pair &a, const Pair &b)
{
    return a.h > b.h || (a.h == b.h && a.l > b.l);
}

__device__ __forceinline__ Pair shfl_xor(const Pair &v, int o)
{
    return {__shfl_xor_sync(0xffffffffu, v.h, o), __shfl_xor_sync(0xffffffffu, v.l, o)};
}

__device__ __forceinline__ Pair shfl(const Pair &v, int src)
{
    return {__shfl_sync(0xffffffffu, v.h, src), __shfl_sync(0xffffffffu, v.l, src)};
}

__device__ __forceinline__ Pair warp_sum(Pair v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = v + shfl_xor(v, o);
    return v;
}

__device__ __forceinline__ Pair warp_scan(Pair v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair y = {__shfl_up_sync(0xffffffffu, v.h, o), __shfl_up_sync(0xffffffffu, v.l, o)};
        if (lane >= o)
            v = y + v;
    }
    return v;
}

__device__ __forceinline__ void st_dsmem_pair(uint32_t addr, const Pair &v)
{
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.h), "f"(v.l)
                 : "memory");
}

}  // namespace

// NT threads a CTA: see launch_verify_draft.
template <class T, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) zp_verify_kernel(const VerifyArgs a, int ctas)
{
    constexpr int VE = Row<T>::VE, WARPS = NT / 32, MARKS = kVfMarks / WARPS;
    constexpr int STEP = kVfBatch * 32;           // vectors of a batch
    __shared__ __align__(8) Pair sums[4][kVfCtas * WARPS];  // every run's, in the row's order, a pass
    __shared__ Pair marks[WARPS][MARKS][32];  // the lanes' sums after a stretch of the run
    __shared__ uint4 ring[WARPS][2 * kVfBatch][32];  // the lanes' vectors on their way
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, wi = threadIdx.x >> 5;
    const int rank = static_cast<int>(cluster_ctarank());
    const int i = blockIdx.x / ctas, runs = ctas * WARPS;
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

    bool left = reject;   // what a rejection leaves; else p itself
    bool strict = false;  // every weight tested
    for (int pass = 0; pass < 4; ++pass) {
        const Row<T> row(target + row_at, left && draft ? draft + row_at : nullptr,
                         left && !draft ? x : -1, a.vocab);
        // this warp's run: whole batches, `stretch` of them to a mark
        const int per = ((row.count + runs - 1) / runs + STEP - 1) / STEP;
        const int stretch = (per + MARKS - 1) / MARKS;
        const int run = rank * WARPS + wi;
        const int v0 = min(row.count, run * per * STEP), v1 = min(row.count, v0 + per * STEP);
        uint64_t s2 = 0, c2 = 0;  // two sums and what they lost
        float s = 0.f, c = 0.f;   // and one of tested weights
        auto add = [&](int, const float (&w)[VE], const float (&e)[VE]) {
#pragma unroll
            for (int k = 0; k < VE; ++k)
                add_exact(s, c, w[k], e[k]);
        };
        auto total = [&] {
            return (normal(low2(s2), low2(c2)) + normal(high2(s2), high2(c2))) + normal(s, c);
        };
        auto mark = [&](int n) {
            if ((n + 1) % stretch == 0)
                marks[wi][n / stretch][lane] = total();
        };
        auto ends = [&](int v) {  // the row's, where they lie in this batch
            const int edge = lane == 0 ? (row.lo ? 0 : -1)
                                       : (row.hi < row.count ? row.count - 1 : -1);
            if (lane < 2 && edge >= v && edge < v + STEP) {
                float w[VE], e[VE];
                row.weights(edge, w, e);
                add(0, w, e);
            }
        };
        if (strict || row.lo >= row.hi) {
            for (int v = v0, n = 0; v < v1; v += STEP, ++n) {
                row.ragged(v + lane, v1, add);
                mark(n);
            }
        } else if (row.q) {
            row.template stream<true>(&ring[wi][0][lane], v0, v1, lane, s2, c2, ends, mark);
        } else if (sizeof(T) == 4) {  // (not where a vector holds eight weights to add:
            // 128 requests of 128,000 without q 19.1 us this way, 18.3 by batches)
            row.template stream<false>(&ring[wi][0][lane], v0, v1, lane, s2, c2, ends, mark);
        } else {
            for (int v = v0, n = 0; v < v1; v += STEP, ++n) {
                row.template batch<false>(v + lane, [&](int u, const uint4 &up, const uint4 &uq) {
                    row.template add_fast<false>(v + u * 32 + lane, up, uq, s2, c2);
                });
                ends(v);
                mark(n);
            }
        }
        const Pair mine = warp_sum(total());
        if (pass == 0)
            cluster_wait();
        if (lane < ctas)
            st_dsmem_pair(dsmem_addr(&sums[pass][run], lane), mine);
        cluster_sync();
        // every warp: the runs' sums, PL a lane, and the level's run
        constexpr int PL = (kVfCtas * WARPS + 31) / 32;
        Pair part[PL], local = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < PL; ++k) {
            part[k] = lane * PL + k < runs ? sums[pass][lane * PL + k] : Pair{0.f, 0.f};
            local = local + part[k];
        }
        const Pair upto = warp_scan(local, lane);
        const Pair all = shfl(upto, 31);
        if (!(all.h < INFINITY) && !strict) {
            strict = true;
            continue;
        }
        if (!(all.h > 0.f)) {
            if (left) {  // p <= q everywhere: drawn from p
                left = strict = false;
                continue;
            }
            if (rank == 0 && threadIdx.x == 0) {
                a.next[i] = -1;
                set_error(a.sticky, ZP_ERR_DEVICE_CHECK);
            }
            return;
        }
        const float r = a.sample_u[i], rh = r * all.h;
        const Pair level = normal(rh, fmaf(r, all.h, -rh) + r * all.l);
        Pair before = {__shfl_up_sync(0xffffffffu, upto.h, 1), __shfl_up_sync(0xffffffffu, upto.l, 1)};
        if (lane == 0)
            before = {0.f, 0.f};
        int hit = -1, tail = -1;  // the run that passes the level; the last with any weight
        Pair hit_before = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < PL; ++k) {
            const Pair after = before + part[k];
            if (part[k].h > 0.f) {
                tail = lane * PL + k;
                if (hit < 0 && after > level) {
                    hit = tail;
                    hit_before = before;
                }
            }
            before = after;
        }
        const unsigned m = __ballot_sync(0xffffffffu, hit >= 0);
        int target_run;
        if (m) {
            target_run = __shfl_sync(0xffffffffu, hit, __ffs(m) - 1);
            hit_before = shfl(hit_before, __ffs(m) - 1);
        } else {  // sample_u not below 1: the last token with weight
            target_run = __reduce_max_sync(0xffffffffu, tail);
        }
        const bool at_end = m == 0;
        if (target_run != run)
            return;
        // the stretch, by the marks; then the step of 32 vectors, the lane and the
        // element that pass the level
        int from = 0;  // batches before the stretch
        if (!at_end) {
            Pair skipped = {0.f, 0.f};
            int k0 = 0, k1 = (v1 - v0 + STEP - 1) / STEP / stretch;  // marks left
            while (k0 < k1) {  // the first mark past the level
                const int k = (k0 + k1) / 2;
                const Pair upto_k = warp_sum(marks[wi][k][lane]);
                if (hit_before + upto_k > level) {
                    k1 = k;
                } else {
                    k0 = k + 1;
                    skipped = upto_k;
                }
            }
            from = k0 * stretch;
            hit_before = hit_before + skipped;
        }
        int last = -1, low = -1;
        for (int vb = v0 + from * STEP; vb < v1; vb += STEP) {
            Pair sum[kVfBatch], step[kVfBatch];
            int top = -1;
            auto one = [&](int u, const float (&w)[VE], const float (&e)[VE]) {
                float ps = 0.f, pc = 0.f;
#pragma unroll
                for (int k = 0; k < VE; ++k) {
                    add_exact(ps, pc, w[k], e[k]);
                    if (w[k] > 0.f)
                        top = row.first + (vb + u * 32 + lane) * VE + k;
                }
                const Pair d = normal(ps, pc);
#pragma unroll
                for (int z = 0; z < kVfBatch; ++z)
                    if (z == u)
                        sum[z] = step[z] = d;
            };
            if (vb < row.lo || vb + STEP > row.hi)
                row.ragged(vb + lane, v1, one);
            else if (row.q)
                row.template batch<true>(vb + lane, [&](int u, const uint4 &up, const uint4 &uq) {
                    float w[VE], e[VE];
                    row.template weights_of<true>(vb + u * 32 + lane, up, uq, w, e);
                    one(u, w, e);
                });
            else
                row.template batch<false>(vb + lane, [&](int u, const uint4 &up, const uint4 &uq) {
                    float w[VE], e[VE];
                    row.template weights_of<false>(vb + u * 32 + lane, up, uq, w, e);
                    one(u, w, e);
                });
#pragma unroll
            for (int o = 16; o; o >>= 1)
#pragma unroll
                for (int u = 0; u < kVfBatch; ++u)
                    step[u] = step[u] + shfl_xor(step[u], o);
#pragma unroll
            for (int u = 0; u < kVfBatch; ++u) {
                if (at_end || !(step[u].h > 0.f && hit_before + step[u] > level)) {
                    hit_before = hit_before + step[u];
                    continue;
                }
                const Pair incl = hit_before + warp_scan(sum[u], lane);
                unsigned got = __ballot_sync(0xffffffffu, sum[u].h > 0.f && incl > level);
                if (!got)  // the level lies at the step's very end
                    got = 0x80000000u >> __clz(__ballot_sync(0xffffffffu, sum[u].h > 0.f));
                const int src = __ffs(got) - 1;
                Pair at = {__shfl_up_sync(0xffffffffu, incl.h, 1),
                           __shfl_up_sync(0xffffffffu, incl.l, 1)};
                if (lane == 0)
                    at = hit_before;
                if (lane == src) {
                    const int v = vb + u * 32 + lane;
                    float w[VE], e[VE];
                    row.weights(v, w, e);
                    int tok = -1;
#pragma unroll
                    for (int k = 0; k < VE; ++k) {
                        if (!(w[k] > 0.f))
                            continue;
                        if (tok < 0 || !(at > level))
                            tok = row.first + v * VE + k;
                        at = at + Pair{w[k], e[k]};
                    }
                    a.next[i] = tok;
                }
                return;
            }
            last = max(last, __reduce_max_sync(0xffffffffu, top));
        }
        // the level lies at the run's very end: its last token with weight
        for (int vb = v0; vb < v0 + from * STEP && last < 0; vb += 32) {
            int top = -1;
            if (vb + lane < v1) {
                float w[VE], e[VE];
                row.weights(vb + lane, w, e);
#pragma unroll
                for (int k = 0; k < VE; ++k)
                    if (w[k] > 0.f)
                        top = row.first + (vb + lane) * VE + k;
            }
            low = max(low, __reduce_max_sync(0xffffffffu, top));
        }
        if (lane == 0)
            a.next[i] = max(last, low);
        return;
    }
}

template <class T, int NT>
static cudaError_t launch_verify_t(const VerifyArgs &a, int ctas, cudaStream_t s)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.R) * static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(NT, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, zp_verify_kernel<T, NT>, a, ctas);
}

cudaError_t launch_verify_draft(const VerifyArgs &a, bool bf16, int sms, cudaStream_t s)
{
    // Small CTAs, as many as give every warp of theirs a batch, up to eight a
    // request (256 requests of a vocabulary of 2,000: 7.7 us with one, 15.8 with
    // eight) and up to what the SMs hold at once, 1,024 threads each (256 of
    // 151,936: 48.4 us with four, 52.8 with two, 46.5 with eight, 77 with one).  Up
    // to two CTAs an SM and long rows: CTAs of twice the threads, for twice the loads
    // in flight (32 requests of 151,936: 14.2 us, not 15.9; but 48 of 50,257: 12.3,
    // not 10.5).
    constexpr int kSmall = 128, kLarge = 256;
    const long long R = a.R, vectors = (static_cast<long long>(a.vocab) * (bf16 ? 2 : 4) + 15) / 16;
    const int step = kSmall * kVfBatch;  // vectors of a batch of every warp of a small CTA
    if (R * kVfCtas <= 2ll * sms && vectors > 2 * kVfCtas * step)
        return bf16 ? launch_verify_t<__nv_bfloat16, kLarge>(a, kVfCtas, s)
                    : launch_verify_t<float, kLarge>(a, kVfCtas, s);
    int ctas = 1;
    while (ctas < kVfCtas && ctas * step < vectors &&
           (ctas == 1 || R * 2 * ctas <= 1024 / kSmall * static_cast<long long>(sms)))
        ctas *= 2;
    return bf16 ? launch_verify_t<__nv_bfloat16, kSmall>(a, ctas, s)
                : launch_verify_t<float, kSmall>(a, ctas, s);
}

}  // namespace zp
