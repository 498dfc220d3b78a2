// logprobs.hip -- log probabilities of given tokens, the entropy and the
// likeliest alternatives of rows of logits, each logit read once.
//
// With c = scale * log2(e), the row's largest logit M and y_i = c (z_i - M):
//     l = sum 2^y_i,   s = sum y_i 2^y_i,
//     log p_i = ln 2 * (y_i - log2 l),   entropy = ln 2 * (log2 l - s / l).
// A part of a row stands in the registers of one workgroup.  Every wave makes
// l and s against its own largest logit, and they are joined once.
//
// Alternatives are ordered by (logit descending, index ascending), one 64-bit
// key an entry.  The k-th largest of the largest logits of 64 groups of lanes
// is a bound that k entries reach, and few more do: these are listed, and each
// entry's place is the number of those above it.  Where the list runs over (equal
// logits, a vocabulary of a few hundred), the k-th largest of all lanes'
// largest entries, with the index to tell equal ones apart, is a bound that
// only k lanes reach.
#include "dtype.hpp"
#include "kv_internal.hpp"

namespace lora {

namespace {

constexpr int STEP = 8;          // neighbouring logits of a thread
constexpr int ROUNDS = 4;        // of these
constexpr int GROUPS = 64;       // of lanes, whose largest logits give the first bound
constexpr int LIST = 256;        // entries that the first bound may leave
constexpr int ROOM = LOGPROBS_MAX_PARTS * LOGPROBS_MAX_TOP;  // and that there is room for
static_assert(ROOM >= LOGPROBS_MAX_TOP * (STEP * ROUNDS + 1), "the entries of as many lanes, and those of the parts before");

template <int DT>
struct Wide {
    typename Elem<DT>::raw w[STEP];
};

// The bits of a float that 16-bit logits leave 0.
template <int DT>
constexpr int low_bits() {
    return DT == DT_F32 ? 0 : DT == DT_BF16 ? 16 : 13;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Whole numbers in the order of the logits (-0 is 0).
__device__ __forceinline__ uint32_t order_of(float z) {
    const uint32_t u = __float_as_uint(z + 0.0f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float of_order(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}

__device__ __forceinline__ uint64_t key_of(float z, int index) {
    return static_cast<uint64_t>(order_of(z)) << 32 | ~static_cast<uint32_t>(index);
}

// v and what lane data-parallel move CTRL brings, joined.
template <int CTRL, typename Op>
__device__ __forceinline__ float moved(float v, Op op) {
    return op(v, __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(v), __float_as_uint(v), CTRL, 0xf, 0xf, false)));
}

// Over the 4, 16 and 64 lanes about each.
template <typename Op>
__device__ __forceinline__ float over4(float v, Op op) {
    v = moved<0xB1>(v, op);   // quad_perm: lanes 1 0 3 2
    return moved<0x4E>(v, op);  // 2 3 0 1
}
template <typename Op>
__device__ __forceinline__ float over16(float v, Op op) {
    v = over4(v, op);
    v = moved<0x124>(v, op);  // row_ror:4
    return moved<0x128>(v, op);
}
template <typename Op>
__device__ __forceinline__ float over64(float v, Op op) {
    v = over16(v, op);
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return op(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

struct Max {
    __device__ __forceinline__ float operator()(float x, float y) const { return fmaxf(x, y); }
};
struct Sum {
    __device__ __forceinline__ float operator()(float x, float y) const { return x + y; }
};

// Against the largest logit m: l and s.
struct Stats {
    float m, l, s;
};

// A term 0 * -inf counts as nothing.
__device__ __forceinline__ float product(float e, float y) { return e * fmaxf(y, -256.0f); }

// Brings l and s to the larger of two largest logits.
__device__ __forceinline__ Stats join(const Stats &a, const Stats &b, float c) {
    const float m = fmaxf(a.m, b.m), ref = m == -INFINITY ? 0.0f : m;
    const float ya = (a.m - ref) * c, yb = (b.m - ref) * c, ea = exp2_fast(ya), eb = exp2_fast(yb);
    // l is 0 where nothing is above -inf, NaN where something is no number.
    return Stats{m, a.l * ea + b.l * eb, a.s * ea + product(a.l * ea, ya) + b.s * eb + product(b.l * eb, yb)};
}

template <int THREADS>
struct Shared {
    uint64_t list[ROOM];                // entries; those of the parts before come first
    uint64_t best[LOGPROBS_MAX_TOP];    // the largest so far, in order
    uint64_t bound;
    uint32_t group[GROUPS];             // largest logits of the lanes' groups, as order_of
    Stats wave[THREADS / 64];
    int n;                              // entries in the list
    unsigned arrived;
};

// The k-th largest of 64 lanes' values, of which the lowest LOW bits are alike.
template <int LOW>
__device__ __forceinline__ uint32_t kth_of_lanes(uint32_t v, int k) {
    uint32_t bound = 0;
    for (int bit = 31; bit >= LOW; --bit) {
        const uint32_t up = bound | 1u << bit;
        if (__popcll(__ballot(v >= up)) >= k) bound = up;
    }
    // A negative number's low bits are ones here.
    return bound & 0x80000000u ? bound : bound | ((1u << LOW) - 1u);
}

// Each entry's place among the n of the list: put(place, entry) for the first k.
template <int THREADS, typename Put>
__device__ __forceinline__ void rank(const uint64_t *list, int n, int k, Put put) {
    for (int t = threadIdx.x; t < n; t += THREADS) {
        const uint64_t mine = list[t];
        int place = 0;
        for (int j = 0; j < n; ++j) place += list[j] > mine;
        if (place < k) put(place, mine);
    }
}

// The logits of one part of a row, in the workgroup's registers: thread t has
// entries (round * THREADS + t) * 8 .. + 7 of the part.
template <int DT, int THREADS>
struct Part {
    Wide<DT> z[ROUNDS];
    int base, V;

    __device__ __forceinline__ int index(int k) const {
        return base + (k * THREADS + static_cast<int>(threadIdx.x)) * STEP;
    }
    // Whether all lanes of the wave hold 8 logits of round k.
    __device__ __forceinline__ bool whole(int k) const {
        return uniform(base + (k * THREADS + static_cast<int>(threadIdx.x | 63)) * STEP + STEP) <= V;
    }
    __device__ __forceinline__ void load(const typename Elem<DT>::raw *row, int part, int vocab) {
        base = part * THREADS * STEP * ROUNDS;
        V = vocab;
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
            const int i = index(k);
            // Rows start at any element, so the load is as wide as the
            // hardware makes of an unaligned one.  Past the end: NaN, which no
            // comparison takes.
            if (i + STEP <= V) {
                __builtin_memcpy(&z[k], row + i, sizeof z[k]);
            } else {
#pragma unroll
                for (int j = 0; j < STEP; ++j) z[k].w[j] = i + j < V ? row[i + j] : Elem<DT>::qnan;
            }
        }
    }
    // What was made of the logits is made anew: kept, it would take more
    // registers than two workgroups a CU have.
    __device__ __forceinline__ void forget() {
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
            uint32_t w[sizeof z[k] / 4];
            __builtin_memcpy(w, &z[k], sizeof w);
#pragma unroll
            for (uint32_t &x : w) asm volatile("" : "+v"(x));
            __builtin_memcpy(&z[k], w, sizeof w);
        }
    }
    __device__ __forceinline__ float at(int k, int j) const { return Elem<DT>::to_f(z[k].w[j]); }
    // -inf where there is none.
    __device__ __forceinline__ float at_or_none(int k, int j) const { return index(k) + j < V ? at(k, j) : -INFINITY; }

    __device__ __forceinline__ float largest() const {
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
            if (whole(k)) {
#pragma unroll
                for (int j = 0; j < STEP; ++j) m = fmaxf(m, at(k, j));
            } else {
#pragma unroll
                for (int j = 0; j < STEP; ++j) m = fmaxf(m, at_or_none(k, j));
            }
        }
        return m;
    }

    // The wave's l and s against its largest logit m.
    __device__ __forceinline__ Stats stats(float m, float c) const {
        float l = 0.0f, s = 0.0f;
        const float mc = m * c;
        if (fabsf(mc) < 1048576.0f) {
            // y against mc, which is off m c by `off`: one rounding a logit.
            const float off = fmaf(m, c, -mc);
#pragma unroll
            for (int k = 0; k < ROUNDS; ++k) {
                if (whole(k)) {
#pragma unroll
                    for (int j = 0; j < STEP; ++j) {
                        const float y = fmaf(at(k, j), c, -mc), e = exp2_fast(y);
                        l += e;
                        s = fmaf(e, y, s);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < STEP; ++j) {
                        const float y = fmaf(at_or_none(k, j), c, -mc), e = exp2_fast(y);
                        l += e;
                        s += product(e, y);
                    }
                }
            }
            s -= off * l;
            const float less = exp2_fast(-off);
            l *= less;
            s *= less;
            // A logit of -inf makes s NaN, and not l.
            if (!__any(s != s)) return Stats{m, over64(l, Sum()), over64(s, Sum())};
            l = s = 0.0f;
        }
        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k)
#pragma unroll
            for (int j = 0; j < STEP; ++j) {
                const float y = (at_or_none(k, j) - ref) * c, e = exp2_fast(y);
                l += e;
                s += product(e, y);
            }
        return Stats{m, over64(l, Sum()), over64(s, Sum())};
    }

    // Adds the thread's entries of at least `bound` (none of them is below the
    // logit `low`) to the list, as far as there is room.
    __device__ __forceinline__ void list_those(uint64_t *list, int *n, float low, uint64_t bound) const {
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k)
#pragma unroll
            for (int j = 0; j < STEP; ++j) {
                const float v = at(k, j);
                if (v >= low) {
                    const uint64_t key = key_of(v, index(k) + j);
                    const int to = key >= bound ? atomicAdd(n, 1) : ROOM;
                    if (to < ROOM) list[to] = key;
                }
            }
    }

    // The first of the thread's logits that are its largest, m.
    __device__ __forceinline__ int first_of(float m) const {
        int i = V;
#pragma unroll
        for (int k = ROUNDS - 1; k >= 0; --k)
#pragma unroll
            for (int j = STEP - 1; j >= 0; --j) i = at(k, j) == m ? index(k) + j : i;
        return i;
    }
};

// Workgroup (row, c) takes parts c * group .. of the row, one after the other;
// the last of a row's workgroups to finish joins what they found.
template <int DT, int THREADS>
__global__ __launch_bounds__(THREADS, 8) void k_logprobs(LogprobsArgs a) {
    using raw = typename Elem<DT>::raw;
    constexpr int WAVES = THREADS / 64, LOW = low_bits<DT>();
    __shared__ Shared<THREADS> sh;
    const int row = blockIdx.x, t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
    const raw *z = static_cast<const raw *>(a.z) + row * a.stride;
    const int top = a.top;
    const int token = a.tokens != nullptr ? a.tokens[row] : -1;
    const bool known = token >= 0 && token < a.vocab;
    const float zt = known ? Elem<DT>::to_f(z[token]) : 0.0f;

    Stats all{-INFINITY, 0.0f, 0.0f};
    int n_best = 0;  // entries of sh.best
    const int p0 = blockIdx.y * a.group, p1 = p0 + a.group < a.parts ? p0 + a.group : a.parts;
    Part<DT, THREADS> part;
    for (int p = p0; p < p1; ++p) {
        part.load(z, p, a.vocab);
        if (t < n_best) sh.list[t] = sh.best[t];
        if (t == 0) sh.n = n_best;
        const float mine = part.largest();
        const float of_group = THREADS == 1024 ? over16(mine, Max()) : over4(mine, Max());
        if (t % (THREADS / GROUPS) == 0) sh.group[t / (THREADS / GROUPS)] = order_of(of_group);
        part.forget();
        const Stats st = part.stats(over64(of_group, Max()), a.c);
        part.forget();
        if (lane == 0) sh.wave[wave] = st;
        __syncthreads();
#pragma unroll 1
        for (int w = 0; w < WAVES; ++w) all = join(all, sh.wave[w], a.c);
        if (top > 0) {
            // At least `top` entries of the part reach the bound, if it has as many.
            const float low = of_order(kth_of_lanes<LOW>(sh.group[lane], top));
            if (mine >= low) part.list_those(sh.list, &sh.n, low, 0);
            __syncthreads();
            if (sh.n > LIST) {
                __syncthreads();
                if (t == 0) sh.n = n_best, sh.bound = 0;
                __syncthreads();
                part.forget();
                const int first = mine >= low ? part.first_of(mine) : a.vocab;
                const uint64_t entry = first < a.vocab ? key_of(mine, first) : 0;
                if (entry != 0) sh.list[atomicAdd(&sh.n, 1)] = entry;
                __syncthreads();
                rank<THREADS>(sh.list, sh.n, top, [&](int place, uint64_t key) {
                    if (place == top - 1) sh.bound = key;
                });
                __syncthreads();
                const uint64_t bound = sh.bound;
                if (t == 0) sh.n = n_best;
                __syncthreads();
                part.forget();
                if (entry >= bound && entry != 0) part.list_those(sh.list, &sh.n, low, bound);
                __syncthreads();
            }
            const int n = sh.n;
            rank<THREADS>(sh.list, n, top, [&](int place, uint64_t key) { sh.best[place] = key; });
            n_best = n < top ? n : top;
        }
        __syncthreads();
    }

    if (gridDim.y > 1) {
        // What this workgroup found, to the agent's coherence point; then it is counted.
        const int wgs = gridDim.y;
        uint64_t *keys = a.keys + (static_cast<long>(row) * wgs + blockIdx.y) * LOGPROBS_MAX_TOP;
        float *stats = a.stats + (static_cast<long>(row) * wgs + blockIdx.y) * 4;
        if (wave == 0) {
            if (lane < top)
                __hip_atomic_store(keys + lane, lane < n_best ? sh.best[lane] : 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (lane < 3)
                __hip_atomic_store(stats + lane, lane == 0 ? all.m : lane == 1 ? all.l : all.s, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            if (lane == 0)
                sh.arrived = __hip_atomic_fetch_add(a.count + row, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (sh.arrived != static_cast<unsigned>(wgs) - 1) return;
        if (t == 0) {
            __hip_atomic_store(a.count + row, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            sh.n = 0;
        }
        all = Stats{-INFINITY, 0.0f, 0.0f};
        const float *from = a.stats + static_cast<long>(row) * wgs * 4;
        for (int w = 0; w < wgs; ++w) {
            auto get = [&](int i) { return __hip_atomic_load(from + w * 4 + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
            all = join(all, Stats{get(0), get(1), get(2)}, a.c);
        }
        if (top > 0) {
            __syncthreads();
            for (int i = t; i < wgs * top; i += THREADS) {
                const uint64_t key = __hip_atomic_load(
                    a.keys + (static_cast<long>(row) * wgs + i / top) * LOGPROBS_MAX_TOP + i % top, __ATOMIC_RELAXED,
                    __HIP_MEMORY_SCOPE_AGENT);
                if (key != 0) sh.list[atomicAdd(&sh.n, 1)] = key;
            }
            __syncthreads();
            rank<THREADS>(sh.list, sh.n, top, [&](int place, uint64_t key) { sh.best[place] = key; });
            __syncthreads();
        }
    }

    // No distribution: something is no number, or nothing is above -inf.
    const bool none = !(all.l > 0.0f && all.l < INFINITY) || !(fabsf(all.m) < INFINITY);
    constexpr double LN2 = 0.69314718055994530942;
    const float nan = __uint_as_float(Elem<DT_F32>::qnan);
    // log2 l: the exponent is exact, and the logarithm of what is left below 1.
    int exponent;
    const float left = frexpf(all.l, &exponent);
    const double log_l = static_cast<double>(exponent) + static_cast<double>(__log2f(left));
    auto log_p = [&](float v) {
        const double y = (static_cast<double>(v) - static_cast<double>(all.m)) * static_cast<double>(a.c);
        return none ? nan : static_cast<float>(LN2 * (y - log_l));
    };
    if (t == 0) {
        if (a.logprob != nullptr) a.logprob[row] = known ? log_p(zt) : nan;
        if (a.entropy != nullptr)
            a.entropy[row] = none ? nan : static_cast<float>(LN2 * (log_l - static_cast<double>(all.s) / static_cast<double>(all.l)));
    }
    if (t < top) {
        const uint64_t key = sh.best[t];
        const long at = static_cast<long>(row) * top + t;
        a.top_ids[at] = none ? -1 : static_cast<int32_t>(~static_cast<uint32_t>(key));
        a.top_logprobs[at] = log_p(of_order(static_cast<uint32_t>(key >> 32)));
    }
}

template <int DT>
hipError_t run(const LogprobsArgs &a, hipStream_t st) {
    const dim3 grid(a.n_rows, (a.parts + a.group - 1) / a.group);
    if (a.threads == 256)
        k_logprobs<DT, 256><<<grid, 256, 0, st>>>(a);
    else
        k_logprobs<DT, 1024><<<grid, 1024, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_logprobs(const LogprobsArgs &args, int dtype, hipStream_t st) {
    LogprobsArgs a = args;
    // A vocabulary that four waves hold needs no more of them.
    a.threads = a.vocab <= 256 * STEP * ROUNDS ? 256 : 1024;
    const int held = a.threads * STEP * ROUNDS;
    a.parts = (a.vocab + held - 1) / held;
    // As many workgroups to a row as there are CUs for it.
    const int wgs = LOGPROBS_WGS / a.n_rows;
    a.group = wgs < 1 ? a.parts : (a.parts + wgs - 1) / wgs;
    switch (dtype) {
        case DT_F32: return run<DT_F32>(a, st);
        case DT_F16: return run<DT_F16>(a, st);
        default: return run<DT_BF16>(a, st);
    }
}

}  // namespace lora
