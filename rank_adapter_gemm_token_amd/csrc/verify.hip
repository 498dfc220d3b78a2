// verify.hip -- drafted tokens accepted or replaced against the target's
// probabilities, from given random numbers.
//
// For a sequence with drafted tokens d_0 .. d_{n-1}, the draft's
// distributions q_i, the target's p_i and numbers u_i of [0, 1):  d_i is kept
// while u_i q_i(d_i) < p_i(d_i), exactly (a product of two fp32 values is
// exact in fp64).  At the first i that is not, the token is drawn from
// w = max(0, p_i - q_i) -- p_i itself if nothing of that is left -- and after
// the last kept one from w = p_n:  the first index at which the running sum
// of w passes u times the whole.  The sums are held in fp64: with fp32 ones a
// vocabulary of 10^5 would move the chosen index in some per cent of calls.
#include "dtype.hpp"
#include "kv_internal.hpp"

namespace lora {

namespace {

constexpr int THREADS = 256;
constexpr int STEP = 8;  // elements a thread takes at a time
constexpr int NONE = 0x7FFFFFFF;

template <int DT>
struct Wide {
    typename Elem<DT>::raw w[STEP];
};

// Eight neighbouring probabilities; rows start at any element, so the load is
// as wide as the hardware makes of an unaligned one.
template <int DT>
__device__ __forceinline__ void load_p(const typename Elem<DT>::raw *p, float (&x)[STEP]) {
    Wide<DT> t;
    __builtin_memcpy(&t, p, sizeof t);
#pragma unroll
    for (int i = 0; i < STEP; ++i) x[i] = Elem<DT>::to_f(t.w[i]);
}

// A weight: what is not above zero (NaN among it) counts as nothing.
__device__ __forceinline__ double weight(float p, float q) {
    const double d = static_cast<double>(p) - static_cast<double>(q);
    return d > 0.0 ? d : 0.0;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// Sum over the workgroup's threads, to all of them.
__device__ __forceinline__ double block_sum(double v, double *s) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// Inclusive running sum over the workgroup's threads.
__device__ __forceinline__ double block_scan(double v, double *s) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_up(v, d, 64);
        if (lane >= d) v += o;
    }
    __syncthreads();
    if (lane == 63) s[wave] = v;
    __syncthreads();
    for (int w = 0; w < wave; ++w) v += s[w];
    return v;
}

// The sum of eight neighbouring weights, index i .. i + 7, those below hi.
template <int DT>
__device__ __forceinline__ double weights(const typename Elem<DT>::raw *p, const typename Elem<DT>::raw *q, int i,
                                          int hi) {
    float x[STEP] = {}, y[STEP] = {};
    if (i + STEP <= hi) {
        load_p<DT>(p + i, x);
        if (q != nullptr) load_p<DT>(q + i, y);
    } else {
#pragma unroll
        for (int j = 0; j < STEP; ++j)
            if (i + j < hi) {
                x[j] = Elem<DT>::to_f(p[i + j]);
                if (q != nullptr) y[j] = Elem<DT>::to_f(q[i + j]);
            }
    }
    double v = 0.0;
#pragma unroll
    for (int j = 0; j < STEP; ++j) v += weight(x[j], y[j]);
    return v;
}

// The row that a sequence's new token is drawn from is cut into up to
// VERIFY_PARTS parts.  Workgroup (c, b) finds that row of sequence b itself (a
// handful of reads), adds up `group` of its parts, and the last of a
// sequence's workgroups to finish picks the part, reads it once more and picks
// the token.
template <int DT>
__global__ __launch_bounds__(THREADS) void k_verify(VerifyArgs a) {
    using raw = typename Elem<DT>::raw;
    const raw *p = static_cast<const raw *>(a.p), *q = static_cast<const raw *>(a.q);
    const int b = blockIdx.y, c = blockIdx.x, t = threadIdx.x, V = a.vocab;
    __shared__ double s[VERIFY_PARTS][THREADS / 64];
    __shared__ int found;
    __shared__ unsigned arrived;

    const int r0 = a.row0[b], r1 = a.row0[b + 1];
    const int n = r1 - r0 - 1;
    // Every sequence has a row at least: b rows come before, n_seqs - 1 - b
    // after.  A list that says otherwise is not followed.
    if (r0 < b || n < 0 || n > VERIFY_MAX_DRAFTS || r1 > a.n_rows - (a.n_seqs - 1 - b)) {
        if (c == 0 && t == 0) a.accepted[b] = -1;
        return;
    }
    // Lane i looks at drafted token i.
    const int lane = t & 63, wave = t >> 6;
    bool keep = false, bad = false;
    int d = -1;
    if (lane < n) {
        d = a.draft[r0 - b + lane];
        bad = d < 0 || d >= V;
        if (!bad) {
            const double pv = Elem<DT>::to_f(p[static_cast<long>(r0 + lane) * V + d]);
            const double qv = Elem<DT>::to_f(q[static_cast<long>(r0 - b + lane) * V + d]);
            keep = static_cast<double>(a.u[r0 + lane]) * qv < pv;
        }
    }
    const bool any_bad = __ballot(bad) != 0;
    const int kept = uniform(__builtin_ctzll(~__ballot(keep)));  // n <= 63: a bit is left
    if (any_bad) {
        // A drafted token that is none: no answer for the sequence.
        if (c == 0) {
            if (t <= n) a.tokens[r0 + t] = -1;
            if (t == 0) a.accepted[b] = -1;
        }
        return;
    }
    const raw *pr = p + static_cast<long>(r0 + kept) * V;
    const raw *qr = kept < n ? q + static_cast<long>(r0 - b + kept) * V : nullptr;

    const int p0 = c * a.group, p1 = p0 + a.group < a.parts ? p0 + a.group : a.parts;
#pragma unroll 2
    for (int part = p0; part < p1; ++part) {
        const int lo = part * a.part, hi = lo + a.part < V ? lo + a.part : V;
        double v = 0.0;
        for (int i = lo + t * STEP; i < hi; i += THREADS * STEP) v += weights<DT>(pr, qr, i, hi);
        v = wave_sum(v);
        if (lane == 0) s[part - p0][wave] = v;
    }
    __syncthreads();
    double *sums = a.sums + static_cast<long>(b) * VERIFY_PARTS;
    if (wave == 0) {
        if (lane < p1 - p0)
            __hip_atomic_store(sums + p0 + lane, (s[lane][0] + s[lane][1]) + (s[lane][2] + s[lane][3]),
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        // The sums are at the agent's coherence point before the workgroup is
        // counted (a release at agent scope would write the whole L2 back:
        // 480 us instead of 40 for 256 sequences).
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if (lane == 0) {
            arrived = __hip_atomic_fetch_add(a.count + b, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            found = NONE;
        }
    }
    __syncthreads();
    if (arrived != gridDim.x - 1) return;
    if (t == 0) __hip_atomic_store(a.count + b, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);

    // Lane i holds part i's sum (VERIFY_PARTS is a wave's width).
    double part_sum = 0.0;
    if (lane < a.parts) part_sum = __hip_atomic_load(sums + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    double run = part_sum;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        const double o = __shfl_up(run, k, 64);
        if (lane >= k) run += o;
    }
    double total = __shfl(run, 63, 64);
    // The part to look in, and the running sum before it.
    int from = 0, to = V;
    double base = 0.0;
    if (!(total > 0.0) && qr != nullptr) {
        // Nothing of the difference is left: the target's row, as a whole.
        qr = nullptr;
        double v = 0.0;
        for (int i = t * STEP; i < V; i += THREADS * STEP) v += weights<DT>(pr, qr, i, V);
        total = block_sum(v, s[0]);
    } else {
        const double aim = static_cast<double>(a.u[r0 + kept]) * total;
        // The first part whose running sum passes, or the last with any weight.
        const unsigned long long passes = __ballot(run > aim), some = __ballot(part_sum > 0.0);
        const int pick = uniform(passes ? __builtin_ctzll(passes) : some ? 63 - __builtin_clzll(some) : 0);
        if (pick > 0) base = __shfl(run, pick - 1, 64);
        from = pick * a.part;
        to = from + a.part < V ? from + a.part : V;
    }
    int token = -1;
    if (total > 0.0 && total <= 1.7976931348623157e308) {
        const double aim = static_cast<double>(a.u[r0 + kept]) * total;
        int last = -1;  // the last index with any weight, if none passes
        for (int at = from; at < to; at += THREADS * STEP) {
            double w[STEP], mine = 0.0;
            const int i = at + t * STEP;
#pragma unroll
            for (int j = 0; j < STEP; ++j) {
                w[j] = i + j < to ? weight(Elem<DT>::to_f(pr[i + j]), qr != nullptr ? Elem<DT>::to_f(qr[i + j]) : 0.0f)
                                  : 0.0;
                mine += w[j];
            }
            const double incl = block_scan(mine, s[0]);
            double r = base + (incl - mine);
            int hit = NONE;
#pragma unroll
            for (int j = 0; j < STEP; ++j) {
                r += w[j];
                if (w[j] > 0.0) last = i + j;
                if (hit == NONE && w[j] > 0.0 && r > aim) hit = i + j;
            }
            if (hit != NONE) atomicMin(&found, hit);
            __syncthreads();
            if (found != NONE) break;
            if (t == THREADS - 1) s[0][0] = base + incl;
            __syncthreads();
            base = s[0][0];
        }
        token = found;
        if (token == NONE) {
            // Rounding kept the running sum at or below the aim.
            __syncthreads();
            if (t == 0) found = -1;
            __syncthreads();
            atomicMax(&found, last);
            __syncthreads();
            token = found;
        }
    }
    // Nothing to draw from (no weight, or not finite): no answer for the sequence.
    if (t == 0) a.accepted[b] = token >= 0 ? kept : -1;
    if (t <= n) a.tokens[r0 + t] = token < 0 ? -1 : t < kept ? d : t == kept ? token : -1;
}

}  // namespace

hipError_t launch_verify(const VerifyArgs &a, int dtype, hipStream_t st) {
    const dim3 grid((a.parts + a.group - 1) / a.group, a.n_seqs);
    switch (dtype) {
        case DT_F32: k_verify<DT_F32><<<grid, THREADS, 0, st>>>(a); break;
        case DT_F16: k_verify<DT_F16><<<grid, THREADS, 0, st>>>(a); break;
        default: k_verify<DT_BF16><<<grid, THREADS, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace lora
