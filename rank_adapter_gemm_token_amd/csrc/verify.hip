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
//
// Bound by the chain of dependent reads for few sequences (7 us for one, 9 us
// for 64 of 32000 entries), by memory for many (256 of 131072 entries in 16
// bits: 134 MB in 33 us, 4.1 TB/s).
#include "dtype.hpp"
#include "kv_internal.hpp"

namespace lora {

namespace {

constexpr int THREADS = 1024;
constexpr int WAVES = THREADS / 64;
constexpr int STEP = 8;    // neighbouring elements of a thread
constexpr int ROUNDS = 4;  // of these, asked for together
constexpr int SEGS = ROUNDS * WAVES;  // runs of 64 * STEP elements in a part
static_assert(THREADS * STEP * ROUNDS == VERIFY_PART && SEGS == 64, "a lane for each segment of a part");

template <int DT>
struct Wide {
    typename Elem<DT>::raw w[STEP];
};

// A weight: what is not above zero (NaN among it) counts as nothing.
__device__ __forceinline__ double weight(float p, float q) {
    const double d = static_cast<double>(p) - static_cast<double>(q);
    return d > 0.0 ? d : 0.0;
}

// v plus what lane data-parallel move CTRL brings to the lanes of the rows in
// MASK (nothing to the others).
template <int CTRL, int MASK>
__device__ __forceinline__ double add_moved(double v) {
    const uint64_t w = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(w), CTRL, MASK, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(w >> 32), CTRL, MASK, 0xf, false);
    return v + __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// Inclusive running sum over the wave's lanes, in registers: a sequence's
// answer waits for five of these one after the other, and by way of LDS each
// would take 0.3 us.
__device__ __forceinline__ double wave_scan(double v) {
    v = add_moved<0x111, 0xf>(v);  // row_shr:1
    v = add_moved<0x112, 0xf>(v);
    v = add_moved<0x114, 0xf>(v);
    v = add_moved<0x118, 0xf>(v);
    v = add_moved<0x142, 0xa>(v);     // lane 15 to the second and fourth row of 16
    return add_moved<0x143, 0xc>(v);  // lane 31 to the third and fourth
}

// Lane `l` of v, to all lanes.
__device__ __forceinline__ double lane_of(double v, int l) {
    const uint64_t w = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(w), l);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(w >> 32), l);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ double wave_sum(double v) { return lane_of(wave_scan(v), 63); }

// Of lanes that hold neighbouring runs' sums v, running r: the first with any
// weight whose running sum passes `aim`, or else the last with any weight.  (A
// lane of none may be the first to pass: the scan adds the same weights in
// another order for each lane, so its sum may stand a rounding above its left
// neighbour's.)
__device__ __forceinline__ int pick_lane(double v, double r, double aim) {
    const unsigned long long some = __ballot(v > 0.0), passes = __ballot(r > aim) & some;
    return uniform(passes ? __builtin_ctzll(passes) : some ? 63 - __builtin_clzll(some) : 0);
}

// The weights of one part of a row, in the workgroup's registers: thread t has
// elements (round * 1024 + t) * 8 .. + 7 of the part.
template <int DT>
struct Part {
    Wide<DT> p[ROUNDS], q[ROUNDS];

    __device__ __forceinline__ void load(const typename Elem<DT>::raw *pr, const typename Elem<DT>::raw *qr, int part,
                                         int V) {
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
            const int i = part * VERIFY_PART + (k * THREADS + static_cast<int>(threadIdx.x)) * STEP;
            p[k] = q[k] = Wide<DT>{};
            // Rows start at any element, so the load is as wide as the
            // hardware makes of an unaligned one.
            if (i + STEP <= V) {
                __builtin_memcpy(&p[k], pr + i, sizeof p[k]);
                if (qr != nullptr) __builtin_memcpy(&q[k], qr + i, sizeof q[k]);
            } else {
#pragma unroll
                for (int j = 0; j < STEP; ++j)
                    if (i + j < V) {
                        p[k].w[j] = pr[i + j];
                        if (qr != nullptr) q[k].w[j] = qr[i + j];
                    }
            }
        }
    }
    __device__ __forceinline__ double at(int k, int j) const {
        return weight(Elem<DT>::to_f(p[k].w[j]), Elem<DT>::to_f(q[k].w[j]));
    }
    __device__ __forceinline__ double sum(int k) const {
        double v = 0.0;
#pragma unroll
        for (int j = 0; j < STEP; ++j) v += at(k, j);
        return v;
    }
};

// Workgroup (c, b) finds the row that sequence b's new token is drawn from (a
// handful of reads), adds up `group` of the row's parts, and the last of a
// sequence's workgroups to finish picks the part, in it the segment, the lane
// and the token.  A part's 32768 elements are in flight at once in one
// workgroup: a row of that much needs no second workgroup and no second read
// (64 sequences, 32000 entries, fp32: 9 us; with 16 workgroups a sequence that
// count each other 18.6 us).
template <int DT>
__global__ __launch_bounds__(THREADS) void k_verify(VerifyArgs a) {
    using raw = typename Elem<DT>::raw;
    const raw *p = static_cast<const raw *>(a.p), *q = static_cast<const raw *>(a.q);
    const int b = blockIdx.y, c = blockIdx.x, t = threadIdx.x, V = a.vocab;
    __shared__ double seg[SEGS];
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
    const int lane = t & 63, wave = uniform(t >> 6);
    bool keep = false, bad = false;
    int d = -1;
    const float u = lane <= n ? a.u[r0 + lane] : 0.0f;
    if (lane < n) {
        d = a.draft[r0 - b + lane];
        bad = d < 0 || d >= V;
        if (!bad) {
            const double pv = Elem<DT>::to_f(p[static_cast<long>(r0 + lane) * V + d]);
            const double qv = Elem<DT>::to_f(q[static_cast<long>(r0 - b + lane) * V + d]);
            keep = static_cast<double>(u) * qv < pv;
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
    const double u_new = static_cast<double>(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(u), kept)));

    // Lane i of part_sum: the sum of part i.
    Part<DT> held;
    double part_sum = 0.0;
    auto add_parts = [&](int p0, int p1) {
        for (int part = p0; part < p1; ++part) {
            held.load(pr, qr, part, V);
            __syncthreads();  // the segments of the part before have been read
#pragma unroll
            for (int k = 0; k < ROUNDS; ++k) {
                const double v = wave_sum(held.sum(k));
                if (lane == 0) seg[k * WAVES + wave] = v;
            }
            __syncthreads();
            const double all = wave_sum(seg[lane]);
            if (lane == part) part_sum = all;
        }
    };
    const int p0 = c * a.group, p1 = p0 + a.group < a.parts ? p0 + a.group : a.parts;
    add_parts(p0, p1);
    int at = p1 - 1;  // the part in `held`
    if (gridDim.x > 1) {
        double *sums = a.sums + static_cast<long>(b) * VERIFY_PARTS;
        if (wave == 0) {
            if (lane >= p0 && lane < p1)
                __hip_atomic_store(sums + lane, part_sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            // The sums are at the agent's coherence point before the workgroup
            // is counted (a release at agent scope would write the whole L2
            // back: 480 us instead of 40 for 256 sequences of 64 workgroups).
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            if (lane == 0)
                arrived = __hip_atomic_fetch_add(a.count + b, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (arrived != gridDim.x - 1) return;
        if (t == 0) __hip_atomic_store(a.count + b, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (lane < a.parts) part_sum = __hip_atomic_load(sums + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (!(wave_sum(part_sum) > 0.0) && qr != nullptr) {
        // Nothing of the difference is left: the target's row, as a whole.
        qr = nullptr;
        part_sum = 0.0;
        add_parts(0, a.parts);
        at = a.parts - 1;
    }
    double run = wave_scan(part_sum);
    const double total = lane_of(run, 63), aim = u_new * total;
    int token = -1;
    if (total > 0.0 && total <= 1.7976931348623157e308) {
        const int part = pick_lane(part_sum, run, aim);
        double base = part > 0 ? lane_of(run, part - 1) : 0.0;
        if (part != at) add_parts(part, part + 1);
        // The segment, by every wave; the rest by the wave that has it.
        const double v = seg[lane];
        run = base + wave_scan(v);
        const int s = pick_lane(v, run, aim);
        if (s > 0) base = lane_of(run, s - 1);
        if (wave == s % WAVES) {
#pragma unroll
            for (int k = 0; k < ROUNDS; ++k) {
                if (k != s / WAVES) continue;
                const double mine = held.sum(k), upto = base + wave_scan(mine);
                const int l = pick_lane(mine, upto, aim);
                if (l > 0) base = lane_of(upto, l - 1);
                if (lane == l) {
                    const int i = part * VERIFY_PART + (k * THREADS + t) * STEP;
                    int hit = -1, last = -1;
#pragma unroll
                    for (int j = 0; j < STEP; ++j) {
                        const double w = held.at(k, j);
                        base += w;
                        if (w > 0.0) last = i + j;
                        if (hit < 0 && w > 0.0 && base > aim) hit = i + j;
                    }
                    found = hit >= 0 ? hit : last;  // last: rounding kept the sum at or below the aim
                }
            }
        }
        __syncthreads();
        token = found;
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
