// logprobs.hip -- log probabilities of given tokens, the entropy and the
// likeliest alternatives of rows of logits.
//
// With c = scale * log2(e), the row's largest logit M and y_i = c (z_i - M):
//     l = sum 2^y_i,   s = sum y_i 2^y_i,
//     log p_i = ln 2 * (y_i - log2 l),   entropy = ln 2 * (log2 l - s / l).
// A row streams through a workgroup's waves once; every lane keeps its largest
// logit, and l and s against it, and the lanes' are joined at the end.
//
// Alternatives are ordered by (logit descending, index ascending), one 64-bit
// key an entry.  The k-th largest of the largest logits of 64 groups of lanes
// is a bound that k entries reach, and few more do: the lanes that hold any look
// for them once more, and each entry's place in their list is the number of
// those above it.  Where the list runs over (equal logits, a vocabulary of a
// few hundred), the k-th largest of what it holds is the next bound, and the
// lanes are looked through again (64 rows of 131072 equal logits, fp32, 20
// alternatives: 42 us; of logits that differ: 12).
// Where fewer than k groups hold anything above -inf, what is above -inf is
// listed, and the lowest indices follow (with -inf as the bound the list ran
// over with masked entries: such rows, of which 200 neighbours are left, 43 us
// instead of 16).
//
// Bound by vector instructions beside memory where there are many rows (2048 of
// 32000, 16 bits: 131 MB in 32 us, 4.1 TB/s), by the chain row -> bound -> list
// -> places where there are few (one of 32000, fp32: 7.5 us; 64 of 131072, fp32,
// four workgroups each: 15 us).
#include "dtype.hpp"
#include "kv_internal.hpp"
#include "row_eight.hpp"

namespace lora {

namespace {

constexpr int STEP = 8;          // neighbouring logits of a lane
constexpr int SEGMENT = 64 * STEP;
constexpr int AHEAD = 4;         // segments that a wave asks for together
constexpr int GROUPS = 64;       // of lanes, whose largest logits give the first bound
constexpr int LIST = 256;        // entries that a bound may leave
constexpr int ROOM = 2 * LIST;   // entries listed of those that are too many
constexpr uint32_t LEAST = 0x00800000u;  // order_of the lowest finite logit, the next above -inf
static_assert(LIST > LOGPROBS_MAX_TOP, "the next bound is above the one before");
static_assert(LOGPROBS_MAX_TOP <= 64, "a lane for each of the first");

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

// Over the 4, 16 and 64 lanes about each.  In every step two lanes that are
// joined give the same result to both, so that a sum is rounded alike in all
// lanes: a token has one log probability, whichever lane writes it.
template <typename Op>
__device__ __forceinline__ float over4(float v, Op op) {
    v = moved<0xB1>(v, op);   // quad_perm: lanes 1 0 3 2
    return moved<0x4E>(v, op);  // 2 3 0 1
}
template <typename Op>
__device__ __forceinline__ float over16(float v, Op op) {
    v = over4(v, op);
    v = moved<0x128>(v, op);  // row_ror:8
    return moved<0x124>(v, op);  // row_ror:4, of lanes alike 8 apart
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

// The same of all lanes' (a lane without any: -inf, 0, 0), alike in all of them:
// the products are rounded before they are added, not fused into one lane's sum.
__device__ __forceinline__ Stats join_lanes(const Stats &a, float c) {
#pragma clang fp contract(off)
    const float m = over64(a.m, Max()), ref = m == -INFINITY ? 0.0f : m;
    const float y = (a.m - ref) * c, e = exp2_fast(y), l = a.l * e;
    return Stats{m, over64(l, Sum()), over64(a.s * e + product(l, y), Sum())};
}

// What a workgroup's waves tell each other.
template <int N>
struct Shared {
    // Entries, ROOM of them, or of all workgroups of the row; 0 where there is none.
    uint64_t list[LOGPROBS_MAX_PARTS * LOGPROBS_MAX_TOP];
    uint64_t best[LOGPROBS_MAX_TOP];                       // the largest, in order
    uint64_t bound;
    uint32_t group[GROUPS];  // largest logits of the lanes' groups, as order_of
    Stats wave[N / 64];
    uint8_t lane[N / 64][64];  // of each wave: the lanes that hold entries to list
    int n;                   // entries in the list
    unsigned arrived;
};
static_assert(ROOM <= LOGPROBS_MAX_PARTS * LOGPROBS_MAX_TOP, "one array serves both");

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

// Each entry's place among the n of the list (zeros among them, and up to a
// multiple of 8, do no harm): put(place, entry) for the first k.
template <int N, typename Put>
__device__ __forceinline__ void rank(const uint64_t *list, int n, int k, Put put) {
    for (int t = threadIdx.x; t < n; t += N) {
        const uint64_t mine = list[t];
        int place = 0;
        for (int j = 0; j < n; j += 8) {  // read together: one by one, 80 entries took 3 us
            uint64_t other[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) other[i] = list[j + i];
#pragma unroll
            for (int i = 0; i < 8; ++i) place += other[i] > mine;
        }
        if (mine != 0 && place < k) put(place, mine);
    }
}

// Segments s0 .. s1 - 1 of a row of V logits, of which wave w has every N / 64th
// from s0 + w on.
template <int DT, int N>
struct Row {
    using raw = typename Elem<DT>::raw;
    static constexpr int WAVES = N / 64;
    static constexpr raw NONE = DT == DT_F32 ? 0xFF800000u : DT == DT_F16 ? 0xFC00u : 0xFF80u;  // -inf
    const raw *z;
    int V, s0, s1;

    using Batch = Eight<DT>[AHEAD];

    // The lane's logits of AHEAD of the wave's segments from s on; -inf past the end.
    __device__ __forceinline__ void load(Batch &e, int s) const {
        const unsigned lane = threadIdx.x & 63;
        const int last = s + (AHEAD - 1) * WAVES;
        if (last < s1 && (last + 1) * SEGMENT <= V) {  // uniform
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                __builtin_memcpy(e[k].w, z + (s + k * WAVES) * SEGMENT + lane * STEP, sizeof e[k].w);
            asm volatile("");  // a branch
        } else {
            auto index = [&](int k) {
                return s + k * WAVES < s1 ? (s + k * WAVES) * SEGMENT + static_cast<int>(lane) * STEP : V;
            };
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) e[k].load(z, index(k), V);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) e[k].clear(index(k), V, NONE);
        }
    }

    // The lane's l and s of a batch, against its largest logit m.
    static __device__ __forceinline__ Stats stats(const Batch &e, float c) {
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
#pragma unroll
            for (int j = 0; j < STEP; ++j) m = fmaxf(m, e[k].at(j));
        const float mc = m * c;
        float l = 0.0f, s = 0.0f;
        if (__all(fabsf(mc) < 1048576.0f)) {
            // y against mc, which is off m c by `off`: one rounding a logit.
            const float off = fmaf(m, c, -mc), less = exp2_fast(-off);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
#pragma unroll
                for (int j = 0; j < STEP; ++j) {
                    const float y = fmaf(e[k].at(j), c, -mc), x = exp2_fast(y);
                    l += x;
                    s = fmaf(x, y, s);
                }
            s = (s - off * l) * less;
            l *= less;
            // A logit of -inf makes s NaN, and not l.
            if (!__any(s != s)) return Stats{m, l, s};
            l = s = 0.0f;
        }
        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
#pragma unroll
            for (int j = 0; j < STEP; ++j) {
                const float y = (e[k].at(j) - ref) * c, x = exp2_fast(y);
                l += x;
                s += product(x, y);
            }
        return Stats{m, l, s};
    }

    // The lane's l and s of all its logits.
    __device__ __forceinline__ Stats read(float c) const {
        Stats all{-INFINITY, 0.0f, 0.0f};
        for (int s = s0 + uniform(threadIdx.x >> 6); s < s1; s += AHEAD * WAVES) {
            Batch e;
            load(e, s);
            all = join(all, stats(e, c), c);
        }
        return all;
    }

    // Adds the entries of at least `bound` that the wave's lanes with `mine` hold
    // to the list, as long as there are not too many.  The wave looks through
    // these lanes' logits together, LOOK of them a lane at a time (every lane
    // through its own: 2048 rows of 32000 took 44 us).
    __device__ __forceinline__ void list(bool mine, uint64_t bound, uint8_t *whose, uint64_t *to, int *n) const {
        constexpr int LOOK = 4;
        const int lane = threadIdx.x & 63, from = s0 + uniform(threadIdx.x >> 6);
        const unsigned long long some = __ballot(mine);
        if (some == 0 || from >= s1) return;
        if (mine) whose[__popcll(some & ((1ull << lane) - 1))] = static_cast<uint8_t>(lane);
        const int segments = (s1 - 1 - from) / WAVES + 1, all = __popcll(some) * segments * STEP;
        for (int q = lane; q - lane < all; q += LOOK * 64) {
            int i[LOOK];
            float v[LOOK];
#pragma unroll
            for (int k = 0; k < LOOK; ++k) {
                const int at = q + k * 64, c = at / STEP / segments, s = at / STEP - c * segments;
                i[k] = at < all ? (from + s * WAVES) * SEGMENT + whose[c & 63] * STEP + at % STEP : V;
                v[k] = Elem<DT>::to_f(z[i[k] < V ? i[k] : V - 1]);
            }
#pragma unroll
            for (int k = 0; k < LOOK; ++k)
                if (i[k] < V && v[k] == v[k] && key_of(v[k], i[k]) >= bound) {
                    const int place = atomicAdd(n, 1);
                    if (place < ROOM) to[place] = key_of(v[k], i[k]);
                }
            if (__hip_atomic_load(n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) > ROOM) break;
        }
    }
};

// What workgroup blockIdx.y of a row found, to the agent's coherence point; the
// workgroup that is counted last joins all of them, in sh.best and (first wave)
// in `all`.
template <int N>
__device__ __forceinline__ bool last_of_row(const LogprobsArgs &a, Shared<N> &sh, int row, int n_best, Stats &all) {
    const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6), wgs = gridDim.y, top = a.top;
    uint64_t *keys = a.keys + static_cast<long>(row) * wgs * LOGPROBS_MAX_TOP;
    float *stats = a.stats + static_cast<long>(row) * wgs * 4;
    if (wave == 0) {
        if (lane < top)
            __hip_atomic_store(keys + blockIdx.y * LOGPROBS_MAX_TOP + lane, lane < n_best ? sh.best[lane] : 0,
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (lane < 3)
            __hip_atomic_store(stats + blockIdx.y * 4 + lane, lane == 0 ? all.m : lane == 1 ? all.l : all.s,
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if (lane == 0)
            sh.arrived = __hip_atomic_fetch_add(a.count + row, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (sh.arrived != static_cast<unsigned>(wgs) - 1) return false;
    if (t == 0) __hip_atomic_store(a.count + row, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (wave == 0) {
        const float *from = stats + (lane < wgs ? lane : 0) * 4;
        auto get = [&](int i) { return __hip_atomic_load(from + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
        const Stats there{get(0), get(1), get(2)};
        all = join_lanes(lane < wgs ? there : Stats{-INFINITY, 0.0f, 0.0f}, a.c);
    }
    if (top > 0) {
        for (int i = t; i < ((wgs * top + 7) & ~7); i += N)
            sh.list[i] = i < wgs * top ? __hip_atomic_load(keys + i / top * LOGPROBS_MAX_TOP + i % top, __ATOMIC_RELAXED,
                                                           __HIP_MEMORY_SCOPE_AGENT)
                                       : 0;
        __syncthreads();
        rank<N>(sh.list, wgs * top, top, [&](int place, uint64_t key) { sh.best[place] = key; });
        __syncthreads();
    }
    return true;
}

// A row's results, by one wave.
template <int DT>
__device__ __forceinline__ void put(const LogprobsArgs &a, int row, const Stats &all, const uint64_t *best, bool known,
                                    float zt) {
    const int lane = threadIdx.x & 63;
    // No distribution: something is no number, or nothing is above -inf.
    const bool none = !(all.l > 0.0f && all.l < INFINITY) || !(fabsf(all.m) < INFINITY);
    constexpr double LN2 = 0.69314718055994530942;
    const float nan = __uint_as_float(Elem<DT_F32>::qnan);
    // log2 l: the exponent is exact, and the logarithm of what is left below 1.
    // The largest logit's own term makes l 1 at least, but the term's two
    // exponentials (Row::stats) and the logarithm are rounded: without the bounds
    // here and below a sure row's log probability came out as +6e-8 and its
    // entropy as -6e-8.
    int exponent;
    const float left = frexpf(all.l, &exponent);
    const double log_l = fmax(static_cast<double>(exponent) + static_cast<double>(__log2f(left)), 0.0);
    // Lane `top` has the given token.
    const uint64_t key = lane < a.top ? best[lane] : 0;
    const float v = lane < a.top ? of_order(static_cast<uint32_t>(key >> 32)) : zt;
    const double y = (static_cast<double>(v) - static_cast<double>(all.m)) * static_cast<double>(a.c);
    const float log_p = none ? nan : static_cast<float>(LN2 * (y - log_l));
    if (lane < a.top) {
        const long at = static_cast<long>(row) * a.top + lane;
        a.top_ids[at] = none ? -1 : static_cast<int32_t>(~static_cast<uint32_t>(key));
        a.top_logprobs[at] = log_p;
    } else if (lane == a.top) {
        if (a.logprob != nullptr) a.logprob[row] = known ? log_p : nan;
        if (a.entropy != nullptr)
            a.entropy[row] = none ? nan : static_cast<float>(LN2 * fmax(log_l - static_cast<double>(all.s) / static_cast<double>(all.l), 0.0));
    }
}

// Workgroup (row, c) reads `group` segments of a row from c * group on; the last
// of a row's workgroups to finish joins what they found.
template <int DT, int N>
__global__ __launch_bounds__(N, 8) void k_logprobs(LogprobsArgs a) {
    constexpr int WAVES = N / 64, LANES = N / GROUPS, LOW = low_bits<DT>();
    static_assert(LANES == 4 || LANES == 16, "what the lanes are joined over");
    __shared__ Shared<N> sh;
    const int row = blockIdx.x, t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6), top = a.top;
    Row<DT, N> r;
    r.z = static_cast<const typename Elem<DT>::raw *>(a.z) + row * a.stride;
    r.V = a.vocab;
    r.s0 = blockIdx.y * a.group;
    r.s1 = r.s0 + a.group < a.segments ? r.s0 + a.group : a.segments;
    const int token = a.tokens != nullptr ? a.tokens[row] : -1;
    const bool known = token >= 0 && token < a.vocab;
    const float zt = known ? Elem<DT>::to_f(r.z[token]) : 0.0f;
    if (t == 0) sh.n = 0;
    for (int i = t; i < ROOM; i += N) sh.list[i] = 0;

    const Stats mine = r.read(a.c);
    const float of_group = LANES == 16 ? over16(mine.m, Max()) : over4(mine.m, Max());
    if (t % LANES == 0) sh.group[t / LANES] = order_of(of_group);
    const Stats of_wave = join_lanes(mine, a.c);
    if (lane == 0) sh.wave[wave] = of_wave;
    __syncthreads();
    int n_best = 0;
    if (top > 0) {
        // At least `top` entries reach the bound, if there are as many above -inf.
        const uint32_t kth = kth_of_lanes<LOW>(sh.group[lane], top);
        uint64_t bound = static_cast<uint64_t>(kth > LEAST ? kth : LEAST) << 32;
        for (;;) {
            r.list(order_of(mine.m) >= static_cast<uint32_t>(bound >> 32), bound, sh.lane[wave], sh.list, &sh.n);
            __syncthreads();
            const int n = sh.n;
            if (n <= LIST) break;
            // Too many: as many entries reach the `top`-th of those listed.
            rank<N>(sh.list, n < ROOM ? n : ROOM, top, [&](int place, uint64_t key) {
                if (place == top - 1) sh.bound = key;
            });
            __syncthreads();
            bound = sh.bound;
            if (t == 0) sh.n = 0;
            for (int i = t; i < ROOM; i += N) sh.list[i] = 0;
            __syncthreads();
        }
        const int n = sh.n;
        rank<N>(sh.list, n, top, [&](int place, uint64_t key) { sh.best[place] = key; });
        n_best = n < top ? n : top;
        if (n < top) {
            // All that is above -inf, so the first of the others are among the
            // first 64.
            const int index = r.s0 * SEGMENT + lane, end = r.s1 * SEGMENT < r.V ? r.s1 * SEGMENT : r.V;
            const bool masked = index < end && Elem<DT>::to_f(r.z[index]) == -INFINITY;
            const unsigned long long all_masked = __ballot(masked);
            const int place = n + __popcll(all_masked & ((1ull << lane) - 1));
            if (wave == 0 && masked && place < top) sh.best[place] = key_of(-INFINITY, index);
            n_best = n + __popcll(all_masked) < top ? n + __popcll(all_masked) : top;
        }
        __syncthreads();
    }
    Stats all{-INFINITY, 0.0f, 0.0f};
    if (wave == 0) all = join_lanes(lane < WAVES ? sh.wave[lane] : all, a.c);
    if (gridDim.y > 1 && !last_of_row<N>(a, sh, row, n_best, all)) return;
    if (wave == 0) put<DT>(a, row, all, sh.best, known, zt);
}

template <int DT>
hipError_t run(const LogprobsArgs &a, bool few, hipStream_t st) {
    const dim3 grid(a.n_rows, (a.segments + a.group - 1) / a.group);
    if (few)
        k_logprobs<DT, 256><<<grid, 256, 0, st>>>(a);
    else
        k_logprobs<DT, 1024><<<grid, 1024, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_logprobs(const LogprobsArgs &args, int dtype, hipStream_t st) {
    LogprobsArgs a = args;
    a.segments = (a.vocab + SEGMENT - 1) / SEGMENT;
    const bool few = a.vocab <= 8192 || (a.n_rows >= 512 && a.vocab <= 1 << 18);
    // As many workgroups to a row as there are CUs for it, of 64 segments each at least.
    int wgs = LOGPROBS_WGS / a.n_rows, parts = (a.segments + 63) / 64;
    if (few || wgs < 1) wgs = 1;
    if (wgs > parts) wgs = parts;
    a.group = (a.segments + wgs - 1) / wgs;
    switch (dtype) {
        case DT_F32: return run<DT_F32>(a, few, st);
        case DT_F16: return run<DT_F16>(a, few, st);
        default: return run<DT_BF16>(a, few, st);
    }
}

}  // namespace lora
