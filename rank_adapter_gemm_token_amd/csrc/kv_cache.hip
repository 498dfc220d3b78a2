// kv_cache.hip -- keys and values quantised into the paged cache as they are
// written, keys turned by their positions on the way, and rows of it read back.
//
// A row x of D values (one token, one head) is held as e4m3 elements e and
// one exponent s:  s the least whole number >= KV_MIN_EXP with
// max|x| <= 448 * 2^s,  e = x * 2^-s rounded to e4m3, ties to even.  Scaling
// by a power of two is exact, so the one rounding is the element's.
//
// Bound by memory for long runs (4096 tokens of 32 heads of 128: 101 MB in 23
// us, 4.4 TB/s, and back 101 MB in 18 us, 5.6 TB/s), by the chain slot -> row
// -> store for a decode step (64 tokens: 6 and 5 us).
//
// An appended key is turned first: pair i of its elements, (x, y), by the angle
// a = position * freq_i:  x cos a - y sin a,  x sin a + y cos a.  The turned
// key has no 16-bit form in between; it is computed in fp64 from a cosine and a
// sine of 48 bits and brought to fp32 with the last bit odd where it is not
// exact, so that the one rounding to e4m3 falls as it does on the turned key
// itself.  (In fp32 an element now and then falls on the other side; with an
// error bound, and fp64 for rows in doubt, it took as long.)  Queries are turned
// in fp32 beside it, by workgroups of their own.  Bound by the chain slot ->
// position -> angle -> store: 4096 tokens in eight runs, 32 and 8 heads of 128,
// 31 us, of which the keys and values alone take 21 (12 where none is turned);
// 64 tokens of 32 and 32 heads 8 us.  A workgroup's 38 KB of LDS, 32 of them
// angles, leave four a CU, so that of those 4096 tokens the queries' workgroups
// follow the keys' rather than run beside them.
#include "dtype.hpp"
#include "kv_internal.hpp"

namespace lora {

namespace {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));

constexpr int TOKENS = 16;   // tokens of a workgroup: 16 lanes each
constexpr int LANES = 16;
constexpr int VT_LD = 20;    // bytes of one element's 16 tokens in LDS, padded
constexpr long FULL_WGS = 2048;  // workgroups that run at once
// Heads of a workgroup that turns keys, and of one that turns queries, at most.
constexpr int APPEND_HEADS = 4, QUERY_HEADS = 8;

// Two values rounded to 16 bits, nearest even.
template <int DT>
__device__ __forceinline__ uint32_t pack(float x, float y) {
    if constexpr (DT == DT_F16) {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, h2{static_cast<_Float16>(x), static_cast<_Float16>(y)});
    } else {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, b2{static_cast<__bf16>(x), static_cast<__bf16>(y)});
    }
}

__device__ __forceinline__ float max16(float v) {
    // Over the 16 lanes of a token (a DPP row).
    v = fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x128, 0xf, 0xf, false)));  // ror 8
    v = fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x124, 0xf, 0xf, false)));
    v = fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x122, 0xf, 0xf, false)));
    v = fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x121, 0xf, 0xf, false)));
    return v;
}

// Exponent byte of a row with largest magnitude amax (finite).
__device__ __forceinline__ int exp_byte(float amax) {
    const uint32_t u = __float_as_uint(amax);
    // amax = m * 2^x, 1 <= m < 2; 448 = 1.75 * 2^8.
    int s = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    s = s < KV_MIN_EXP ? KV_MIN_EXP : s;
    return s + KV_EXP_BIAS;
}

// N neighbouring 16-bit elements of a row, N / 2 words.
template <int N>
struct Words {
    uint32_t w[N / 2];
    __device__ __forceinline__ void load(const uint16_t *p) {
        if constexpr (N == 8)
            *reinterpret_cast<u32x4_t *>(w) = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(p));
        else
            *reinterpret_cast<u32x2_t *>(w) = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t *>(p));
    }
    __device__ __forceinline__ void store(uint16_t *p) const {
        if constexpr (N == 8)
            *reinterpret_cast<u32x4_t *>(p) = *reinterpret_cast<const u32x4_t *>(w);
        else
            *reinterpret_cast<u32x2_t *>(p) = *reinterpret_cast<const u32x2_t *>(w);
    }
    template <int DT>
    __device__ __forceinline__ float at(int i) const {
        return Elem<DT>::to_f(static_cast<uint16_t>(w[i / 2] >> (16 * (i % 2))));
    }
};

// Elements x(0) .. x(N - 1) of a row as bytes in N / 4 words.
template <int N, typename X>
__device__ __forceinline__ void quantise(X x, int byte, uint32_t (&w)[N / 4]) {
    const float inv = __uint_as_float(static_cast<uint32_t>(2 * KV_EXP_BIAS - byte) << 23);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(x(4 * i) * inv, x(4 * i + 1) * inv, 0, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(x(4 * i + 2) * inv, x(4 * i + 3) * inv, v, true);
        w[i] = static_cast<uint32_t>(v);
    }
}

// How the elements of a head are paired to be turned.
enum : int { TURN_NONE = 0, TURN_HALVES = 1, TURN_PAIRS = 2 };

// Tokens that a workgroup may look at: its own and the 15 after them.
constexpr int SIGHT = 2 * TOKENS - 1;

struct Positions {
    int at[ROPE_MAX_AXES][SIGHT];
};

// The positions of tokens first .. first + SIGHT - 1, for all threads after the
// next barrier.
__device__ __forceinline__ void load_positions(const TurnArgs &a, int n_tokens, int first, Positions &p) {
    const int axis = threadIdx.x / SIGHT, i = threadIdx.x % SIGHT;
    static_assert(ROPE_MAX_AXES * SIGHT <= 256, "a thread for each");
    if (axis < a.t.n_axes)
        p.at[axis][i] = first + i < n_tokens ? a.positions[static_cast<long>(axis) * n_tokens + first + i] : 0;
}

// Whether a token has a position outside the table.
__device__ __forceinline__ bool outside(const RopeTable &t, const Positions &p, int token) {
    bool bad = false;
    for (int a = 0; a < t.n_axes; ++a) bad |= static_cast<unsigned>(p.at[a][token]) >= static_cast<unsigned>(t.n_positions);
    return bad;
}

// A pair's cosine and sine.
template <typename T>
struct __align__(2 * sizeof(T)) Angle {
    T c, s;
};

// Looks up the angles of the first `tokens` tokens with positions `p` (a barrier
// is to follow), each once for all of a workgroup's heads.  A lane that turns M
// pairs of a head, pairs q M .. q M + M - 1, finds the j-th of token i at i n +
// j n / M + q: neighbouring lanes read neighbouring places.  (Every lane with its
// own pairs' in registers, 4096 tokens of 8 key heads took 34 us.)
template <typename T, int M>
__device__ __forceinline__ void look_up(const RopeTable &t, const Positions &p, int tokens, Angle<T> *to) {
    for (int at = threadIdx.x; at < tokens * t.n; at += 256) {
        const int token = at / t.n, i = at - token * t.n;
        const int pos = p.at[t.n_axes > 1 ? t.axis[i] : 0][token];
        const long from = (static_cast<unsigned>(pos) < static_cast<unsigned>(t.n_positions) ? static_cast<long>(pos) : 0) * t.n + i;
        const float2 h = t.hi[from];
        float2 l{};
        if constexpr (sizeof(T) == 8) l = t.lo[from];
        to[token * t.n + i % M * (t.n / M) + i / M] = {static_cast<T>(h.x) + static_cast<T>(l.x),
                                                       static_cast<T>(h.y) + static_cast<T>(l.y)};
    }
}

// Pairs of a lane's N elements.
template <int N, int STYLE>
constexpr int pairs_of() { return STYLE == TURN_PAIRS ? N / 2 : N; }

// Lane l's first pair, if its elements turn.
template <int N, int STYLE>
__device__ __forceinline__ int first_pair(int n, int l) {
    return STYLE == TURN_PAIRS ? l * (N / 2) : l * N >= n ? l * N - n : l * N;
}

// The words of the row that hold the partners of lane l's elements (halves:
// another lane's of the same 16; pairs: its own).
template <int N, int STYLE>
__device__ __forceinline__ Words<N> partners(const Words<N> &x, int n, int l) {
    if constexpr (STYLE == TURN_PAIRS) return x;
    const int away = n / N, lane = threadIdx.x & 63;
    const int from = l * N >= 2 * n ? lane : l * N < n ? lane + away : lane - away;
    Words<N> y;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) y.w[i] = __shfl(x.w[i], from);
    return y;
}

// fp64 to fp32, to the neighbour with the odd last bit where it is not exact:
// any later rounding to two bits fewer falls as that of d itself would.
__device__ __forceinline__ float to_odd(double d) {
    const float f = static_cast<float>(d);
    const double back = static_cast<double>(f);
    uint32_t u = __float_as_uint(f);
    if (back != d && fabsf(f) < INFINITY) u = (u - (fabs(back) > fabs(d) ? 1u : 0u)) | 1u;
    return __uint_as_float(u);
}

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

// Element i of a row's N (of which y holds the partners), turned by its pair's
// angle: x c - y s of the first of a pair, x c + y s of the second.
template <int DT, typename T, int N, int STYLE>
__device__ __forceinline__ T turned(const Words<N> &x, const Words<N> &y, int i, Angle<T> a, bool second) {
    const float v = y.template at<DT>(STYLE == TURN_PAIRS ? i ^ 1 : i);
    if (STYLE == TURN_PAIRS) second = (i & 1) != 0;
    return fma(static_cast<T>(x.template at<DT>(i)), a.c, static_cast<T>(second ? v : -v) * a.s);
}

// The tokens a workgroup deals with.  It owns 16 neighbouring tokens of the
// call.  Where most of 16 neighbours of the call lie in order in one block of
// 16 rows (at least MOST; the others are padding, or of another block), the
// block's values are turned in LDS and move as words; the workgroup that owns
// the neighbours' first place takes all of them.  The other tokens it owns
// move four to a word or a byte at a time.  4096 tokens of 32 heads of 128: one
// run 23 us (and 18 to read); with 2% padding among them 24; eight runs that
// begin and end inside a block, with 2% padding, 30 (25); scattered, where
// every byte has a word of its own, 147 (51).
constexpr int MOST = 9;  // more than half: no two blocks have the same first place

struct Tile {
    int slot;        // of the lane's own token, or -1
    bool single;     // not moved with a block
    bool word;       // single, one of four neighbours that fill a word of a block
    int leads;       // bit i: a block is moved from the workgroup's place i (uniform)
    bool any_word;   // of the workgroup's tokens (uniform)
};

// The call's slots about the workgroup: tokens first - 15 .. first + 30, and
// for each place that a block is moved from, the block's first slot.
struct Window {
    int s[46];
    int leads, any_word;
    int block[TOKENS];
};

__device__ __forceinline__ Tile find_tile(const int32_t *slots, int n_tokens, int first, int n_rows, Window &w) {
    const int t = threadIdx.x;
    if (t < 46) {
        const int at = first - 15 + t;
        w.s[t] = at >= 0 && at < n_tokens ? slots[at] : -1;
    }
    if (t == 0) w.leads = w.any_word = 0;
    __syncthreads();
    const int me = t / LANES, l = t % LANES;  // the lane's token: w.s[15 + me]
    Tile r;
    const int mine = w.s[15 + me];
    r.slot = mine >= 0 && mine < n_rows ? mine : -1;
    // How many of the 16 neighbours from `place` of the window lie in order in
    // the block from slot0.
    auto moved = [&](int place, int slot0) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < KV_BLOCK; ++i) n += w.s[place + i] == slot0 + i;
        return n >= MOST;
    };
    // A token's block begins slot % 16 places before it.
    const int place = 15 + me - (r.slot & 15);
    r.single = r.slot >= 0 && !(first - 15 + place >= 0 && moved(place, r.slot & ~15));
    const int w0 = me - (r.slot & 3);
    r.word = r.single && w0 >= 0 && w0 + 3 < TOKENS;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.word = r.word && w.s[15 + w0 + i] == (r.slot & ~3) + i;
    if (r.word) w.any_word = 1;
    // Place `me` as a first one: lane l asks for the block of the token l after it.
    const int other = w.s[15 + me + l], slot0 = other >= l ? other - l : -1;
    if (slot0 >= 0 && (slot0 & 15) == 0 && slot0 < n_rows && moved(15 + me, slot0)) {
        w.block[me] = slot0;
        atomicOr(&w.leads, 1 << me);
    }
    __syncthreads();
    r.leads = uniform(w.leads);
    r.any_word = uniform(w.any_word) != 0;
    return r;
}

__device__ __forceinline__ long row_of(const KvCache &c, int slot, int head) {
    const int page = slot >> c.page_shift, off = slot & ((1 << c.page_shift) - 1);
    return ((static_cast<long>(page) * c.heads + head) << c.page_shift) + off;
}

// Workgroup: one tile of tokens and `per` neighbouring heads, one after the
// other, the next head's rows asked for before this one's are turned.
template <int DT, int D, int STYLE>
__device__ __forceinline__ void write_tile(const KvCache &c, const TurnArgs &turn, Angle<double> *angles,
                                           const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride,
                                           const int32_t *slots, int n_tokens, int b, int per, int groups) {
    constexpr int N = D / LANES;
    __shared__ Window w;
    __shared__ Positions pos;
    __shared__ __align__(16) uint8_t by_element[2][D * VT_LD];
    const int first = b / groups * TOKENS, h0 = b % groups * per;
    const int h1 = h0 + per < c.heads ? h0 + per : c.heads;
    const int me = threadIdx.x / LANES, l = threadIdx.x % LANES;
    if constexpr (STYLE != TURN_NONE) load_positions(turn, n_tokens, first, pos);
    const Tile tile = find_tile(slots, n_tokens, first, c.n_pages << c.page_shift, w);
    if constexpr (STYLE != TURN_NONE) {
        // Of its own tokens, and of those after them in a block that it moves.
        look_up<double, pairs_of<N, STYLE>()>(turn.t, pos, TOKENS + (tile.leads != 0 ? 31 - __builtin_clz(tile.leads) : 0), angles);
        __syncthreads();
    }
    if (h0 == 0 && l == 0) {
        const int mine = w.s[15 + me];
        const bool lost = STYLE != TURN_NONE && first + me < n_tokens && outside(turn.t, pos, me);
        if (first + me < n_tokens && mine != -1 && (tile.slot < 0 || lost)) atomicAdd(c.err, 1ull);
    }

    // One row's share of a lane: its key's and value's elements.
    struct Pair {
        Words<N> k, v;
    };
    auto load = [&](int token, int head) {
        Pair x;
        x.k.load(k + token * k_stride + static_cast<long>(head) * D + l * N);
        x.v.load(v + token * v_stride + static_cast<long>(head) * D + l * N);
        return x;
    };
    // Writes the key and both exponents of a token, the i-th from `first` on, and
    // leaves the value's bytes in vw.
    auto put = [&](const Pair &x, int i, long R, uint32_t (&vw)[N / 4]) {
        float kx[N], vx[N], ka = 0.0f, va = 0.0f;
        bool fin = true;
        if constexpr (STYLE != TURN_NONE) {
#pragma unroll
            for (int e = 0; e < N; ++e) kx[e] = x.k.template at<DT>(e), vx[e] = x.v.template at<DT>(e);
            constexpr int M = pairs_of<N, STYLE>();
            const int n = turn.t.n;
            const Words<N> y = partners<N, STYLE>(x.k, n, l);
            fin = !outside(turn.t, pos, i);
            if (l * N < 2 * n) {
                const Angle<double> *a = angles + i * n + first_pair<N, STYLE>(n, l) / M;
#pragma unroll
                for (int e = 0; e < N; ++e)
                    kx[e] = to_odd(turned<DT, double, N, STYLE>(x.k, y, e, a[(STYLE == TURN_PAIRS ? e / 2 : e) * (n / M)], l * N >= n));
            }
        }
        // What was not turned is widened anew where it is used: in registers it
        // would leave fewer workgroups a CU.
        auto key = [&](int e) {
            if constexpr (STYLE == TURN_NONE) return x.k.template at<DT>(e);
            else return kx[e];
        };
        auto value = [&](int e) {
            if constexpr (STYLE == TURN_NONE) return x.v.template at<DT>(e);
            else return vx[e];
        };
#pragma unroll
        for (int e = 0; e < N; ++e) {
            // A value that is not finite has the exponent bits all set (and
            // turns into one that is not); fmax drops NaN.
            fin &= finite(key(e));
            fin &= finite(value(e));
            ka = fmaxf(ka, fabsf(key(e)));
            va = fmaxf(va, fabsf(value(e)));
        }
        ka = max16(ka);
        va = max16(va);
        const bool poison = max16(fin ? 0.0f : 1.0f) != 0.0f;
        const int kb = poison ? KV_EXP_BIAS : exp_byte(ka), vb = poison ? KV_EXP_BIAS : exp_byte(va);
        uint32_t kw[N / 4];
        quantise<N>(key, kb, kw);
        quantise<N>(value, vb, vw);
        if (poison) {
#pragma unroll
            for (int e = 0; e < N / 4; ++e) kw[e] = 0x7F7F7F7Fu, vw[e] = 0u;
        }
        uint32_t *kd = reinterpret_cast<uint32_t *>(c.k + (R & ~15L) * D + key_byte<D>(R & 15, l * N));
#pragma unroll
        for (int i = 0; i < N / 4; ++i) kd[i] = kw[i];
        if (l == 0) {
            c.kexp[R] = static_cast<uint8_t>(kb);
            c.vinv[R] = static_cast<uint8_t>(poison ? KV_POISON : 2 * KV_EXP_BIAS - vb);
        }
    };

    // The cross-lane maxima stay within a token's 16 lanes, which go the same way.
    // Of the single ones, four neighbours that fill a word of the block move as
    // words, each of the four tokens' lanes a quarter of the elements.
    if (tile.single || tile.any_word) {
        const int q = tile.slot & 3, w0 = me - q;
        const bool word = tile.word;
        Pair x{};
        if (tile.single) x = load(first + me, h0);
        for (int head = h0; head < h1; ++head) {
            Pair next{};
            uint8_t *by = by_element[(head - h0) & 1];
            uint32_t vw[N / 4] = {};
            long R = 0;
            if (tile.single) {
                next = load(first + me, head + 1 < h1 ? head + 1 : head);
                R = row_of(c, tile.slot, head);
                put(x, me, R, vw);
            }
            if (word) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    by[(l * N + i) * VT_LD + me] = static_cast<uint8_t>(vw[i / 4] >> (8 * (i % 4)));
            }
            if (tile.any_word) __syncthreads();
            uint8_t *vd = c.v + (R & ~15L) * D + (R & 15);
            if (word) {
#pragma unroll
                for (int i = 0; i < N / 4; ++i) {
                    const int d = l * N + q * (N / 4) + i;
                    uint32_t four;
                    __builtin_memcpy(&four, by + d * VT_LD + w0, 4);
                    *reinterpret_cast<uint32_t *>(vd - q + d * KV_BLOCK) = four;
                }
            } else if (tile.single) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    vd[(l * N + i) * KV_BLOCK] = static_cast<uint8_t>(vw[i / 4] >> (8 * (i % 4)));
            }
            x = next;
        }
        if (tile.any_word) __syncthreads();  // `by_element` is written again
    }
    for (int leads = tile.leads; leads != 0; leads &= leads - 1) {
        const int place = __builtin_ctz(leads), slot0 = w.block[place], token = first + place + me;
        int have = 0;  // bit i: row i of the block is among the tokens
#pragma unroll
        for (int i = 0; i < KV_BLOCK; ++i) have |= (w.s[15 + place + i] == slot0 + i) << i;
        const bool there = (have >> me) & 1;
        Pair x{};
        if (there) x = load(token, h0);
        for (int head = h0; head < h1; ++head) {
            Pair next{};
            uint8_t *by = by_element[(head - h0) & 1];
            uint32_t vw[N / 4] = {};
            const long R = row_of(c, slot0, head);
            if (there) {
                next = load(token, head + 1 < h1 ? head + 1 : head);
                put(x, place + me, R + me, vw);
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
                by[(l * N + i) * VT_LD + me] = static_cast<uint8_t>(vw[i / 4] >> (8 * (i % 4)));
            __syncthreads();
            // 256 threads x N bytes: the block's D x 16 bytes in order.
            const int at = threadIdx.x * N, d = at / KV_BLOCK, part = at % KV_BLOCK;
            uint8_t *vd = c.v + R * D + at;
            const uint8_t *from = by + d * VT_LD + part;
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const int four = (have >> (part + i)) & 15;
                if (four == 15) {
                    *reinterpret_cast<uint32_t *>(vd + i) = *reinterpret_cast<const uint32_t *>(from + i);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if ((four >> j) & 1) vd[i + j] = from[i + j];
                }
            }
            x = next;
        }
        __syncthreads();  // `by_element` is written again
    }
}

template <int DT, int D>
__global__ __launch_bounds__(256) void k_kv_write(KvCache c, const uint16_t *k, int64_t k_stride, const uint16_t *v,
                                                  int64_t v_stride, const int32_t *slots, int n_tokens, int per,
                                                  int groups) {
    write_tile<DT, D, TURN_NONE>(c, TurnArgs{}, nullptr, k, k_stride, v, v_stride, slots, n_tokens, static_cast<int>(blockIdx.x),
                                 per, groups);
}

// Workgroup b of the queries': 16 tokens and `per` neighbouring heads, QUERIES
// rows of a lane in flight.  A row's lanes read all of it before any writes, so
// it may be turned in place.
constexpr int QUERIES = 4;

template <int DT, int D, int STYLE>
__device__ __forceinline__ void turn_queries(const TurnArgs &a, Angle<float> *angles, int n_tokens, int b, int per,
                                             int groups) {
    constexpr int N = D / LANES, M = pairs_of<N, STYLE>();
    __shared__ Positions pos;
    const int first = b / groups * TOKENS, h0 = b % groups * per;
    const int h1 = h0 + per < a.n_heads ? h0 + per : a.n_heads;
    const int me = threadIdx.x / LANES, l = threadIdx.x % LANES;
    const int token = first + me < n_tokens ? first + me : n_tokens - 1;
    const uint16_t *from = a.q + token * a.q_stride + l * N;
    uint16_t *to = a.q_out + token * a.out_stride + l * N;
    Words<N> x[QUERIES];
    auto load = [&](int head) {
#pragma unroll
        for (int j = 0; j < QUERIES; ++j) x[j].load(from + static_cast<long>(head + j < h1 ? head + j : h1 - 1) * D);
    };
    load(h0);
    load_positions(a, n_tokens, first, pos);
    __syncthreads();
    look_up<float, M>(a.t, pos, TOKENS, angles);
    const bool bad = outside(a.t, pos, me), turns = l * N < 2 * a.t.n;
    __syncthreads();
    if (first + me >= n_tokens) return;
    Angle<float> angle[M];
#pragma unroll
    for (int j = 0; j < M; ++j) angle[j] = angles[me * a.t.n + first_pair<N, STYLE>(a.t.n, turns ? l : 0) / M + j * (a.t.n / M)];
    for (int head = h0; head < h1; head += QUERIES) {
#pragma unroll
        for (int j = 0; j < QUERIES; ++j) {
            if (head + j >= h1) break;
            const Words<N> y = partners<N, STYLE>(x[j], a.t.n, l);
            Words<N> o;
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const int k = STYLE == TURN_PAIRS ? i / 2 : i, k1 = STYLE == TURN_PAIRS ? k : i + 1;
                const bool second = l * N >= a.t.n;
                const uint32_t both = pack<DT>(turned<DT, float, N, STYLE>(x[j], y, i, angle[k], second),
                                               turned<DT, float, N, STYLE>(x[j], y, i + 1, angle[k1], second));
                o.w[i / 2] = bad ? Elem<DT>::qnan * 0x10001u : turns ? both : x[j].w[i / 2];
            }
            o.store(to + static_cast<long>(head + j) * D);
        }
        if (head + QUERIES < h1) load(head + QUERIES);
    }
}

// The first write_wgs workgroups write keys and values, the others turn queries.
// (In turn over the launch, four workgroups a CU there too: 35 us instead of 31
// for 4096 tokens of 32 and 8 heads.)
template <int DT, int D, int STYLE>
__global__ __launch_bounds__(256) void k_kv_append(KvCache c, TurnArgs turn, const uint16_t *k, int64_t k_stride,
                                                   const uint16_t *v, int64_t v_stride, const int32_t *slots,
                                                   int n_tokens, int per, int groups, unsigned write_wgs, int q_per,
                                                   int q_groups) {
    __shared__ Angle<double> angles[SIGHT * (D / 2)];
    const unsigned b = blockIdx.x;
    if (b < write_wgs)
        write_tile<DT, D, STYLE>(c, turn, angles, k, k_stride, v, v_stride, slots, n_tokens, static_cast<int>(b), per, groups);
    else
        turn_queries<DT, D, STYLE>(turn, reinterpret_cast<Angle<float> *>(angles), n_tokens,
                                   static_cast<int>(b - write_wgs), q_per, q_groups);
}

// A position's row of the table, in fp64 and cut in two.
__global__ __launch_bounds__(256) void k_rope_table(const double *freq, double scale, int n_positions, int n,
                                                    float2 *hi, float2 *lo) {
    const long all = static_cast<long>(n_positions) * n;
    for (long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x; i < all; i += static_cast<long>(gridDim.x) * 256) {
        const long p = i / n;
        double sn, cs;
        sincos(static_cast<double>(p) * freq[i - p * n], &sn, &cs);
        cs *= scale;
        sn *= scale;
        const float2 h{static_cast<float>(cs), static_cast<float>(sn)};
        hi[i] = h;
        lo[i] = float2{static_cast<float>(cs - h.x), static_cast<float>(sn - h.y)};
    }
}

template <int DT, int D>
__global__ __launch_bounds__(256) void k_kv_read(KvCache c, const int32_t *slots, int n_tokens, uint16_t *k,
                                                 uint16_t *v, int per, int groups) {
    constexpr int N = D / LANES;
    __shared__ Window w;
    __shared__ __align__(16) uint8_t turned[2][D * VT_LD];
    const int first = static_cast<int>(blockIdx.x) / groups * TOKENS, h0 = static_cast<int>(blockIdx.x) % groups * per;
    const int h1 = h0 + per < c.heads ? h0 + per : c.heads;
    const int me = threadIdx.x / LANES, l = threadIdx.x % LANES;
    const Tile tile = find_tile(slots, n_tokens, first, c.n_pages << c.page_shift, w);

    // N values of a row: their elements in words w, all scaled by 2^(byte - 127).
    auto put = [&](uint16_t *to, int token, int head, const uint32_t (&w)[N / 4], int byte, bool poison) {
        const float f = __uint_as_float(static_cast<uint32_t>(byte) << 23);
        Words<N> o;
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), false);
            const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), true);
            const uint32_t nan = Elem<DT>::qnan * 0x10001u;
            o.w[2 * i] = poison ? nan : pack<DT>(lo.x * f, lo.y * f);
            o.w[2 * i + 1] = poison ? nan : pack<DT>(hi.x * f, hi.y * f);
        }
        o.store(to + (static_cast<long>(token) * c.heads + head) * D + l * N);
    };
    // What a lane reads of a row: its key's elements, N bytes of the value's
    // (at vp), and the exponents.
    struct Held {
        uint32_t k[N / 4], v[N / 4];
        int kb, vi;
    };
    auto load = [&](long R) {
        Held x;
        const uint32_t *kp = reinterpret_cast<const uint32_t *>(c.k + (R & ~15L) * D + key_byte<D>(R & 15, l * N));
        const uint32_t *vp = reinterpret_cast<const uint32_t *>(c.v + (R & ~15L) * D + threadIdx.x * N);
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            x.k[i] = kp[i];
            x.v[i] = vp[i];
        }
        x.kb = c.kexp[R];
        x.vi = c.vinv[R];
        return x;
    };

    if (first + me < n_tokens && (tile.single || tile.slot < 0)) {
        const int token = first + me;
        if (tile.slot < 0) {
            // Nothing is held for this token: an explicit NaN row.
            if (h0 == 0 && l == 0) atomicAdd(c.err, 1ull);
            const uint32_t none[N / 4] = {};
            for (int head = h0; head < h1; ++head) {
                put(k, token, head, none, 0, true);
                put(v, token, head, none, 0, true);
            }
        } else {
#pragma unroll 2
            for (int head = h0; head < h1; ++head) {
                const long R = row_of(c, tile.slot, head);
                const Held x = load(R);
                put(k, token, head, x.k, x.kb, x.vi == KV_POISON);
                const uint8_t *vs = c.v + (R & ~15L) * D + (R & 15) + l * N * KV_BLOCK;
                uint32_t e[N / 4] = {};
#pragma unroll
                for (int i = 0; i < N; ++i) e[i / 4] |= static_cast<uint32_t>(vs[i * KV_BLOCK]) << (8 * (i % 4));
                put(v, token, head, e, 2 * KV_EXP_BIAS - x.vi, x.vi == KV_POISON);
            }
        }
    }
    for (int leads = tile.leads; leads != 0; leads &= leads - 1) {
        const int place = __builtin_ctz(leads), slot0 = w.block[place], token = first + place + me;
        const bool there = w.s[15 + place + me] == slot0 + me;
        const int at = threadIdx.x * N, d = at / KV_BLOCK, part = at % KV_BLOCK;
        Held x = load(row_of(c, slot0, h0) + me);
        for (int head = h0; head < h1; ++head) {
            const Held next = load(row_of(c, slot0, head + 1 < h1 ? head + 1 : head) + me);
            uint8_t *turn = turned[(head - h0) & 1];
#pragma unroll
            for (int i = 0; i < N / 4; ++i) *reinterpret_cast<uint32_t *>(turn + d * VT_LD + part + 4 * i) = x.v[i];
            if (there) put(k, token, head, x.k, x.kb, x.vi == KV_POISON);
            __syncthreads();
            uint32_t e[N / 4] = {};
#pragma unroll
            for (int i = 0; i < N; ++i)
                e[i / 4] |= static_cast<uint32_t>(turn[(l * N + i) * VT_LD + me]) << (8 * (i % 4));
            if (there) put(v, token, head, e, 2 * KV_EXP_BIAS - x.vi, x.vi == KV_POISON);
            x = next;
        }
        __syncthreads();  // `turned` is written again
    }
}

// Heads of a workgroup: one until the workgroups fill the device several times
// over, then up to four, which share the look at the slots and keep more rows
// in flight.  Those that look angles up share that too, from fewer workgroups on.
struct Cut {
    int per, groups;
    unsigned grid;
    Cut(int heads, int T, int most = 0) {
        const int tiles = (T + TOKENS - 1) / TOKENS;
        const long all = tiles * static_cast<long>(heads);
        per = all >= 4 * FULL_WGS ? 4 : 1;
        if (most != 0) {
            per = static_cast<int>(all / 1024);
            per = per < 1 ? 1 : per > most ? most : per;
        }
        groups = (heads + per - 1) / per;
        grid = static_cast<unsigned>(tiles) * static_cast<unsigned>(groups);
    }
};

template <int DT, int D>
hipError_t write(const KvCache &c, const void *k, int64_t ks, const void *v, int64_t vs, const int32_t *slots, int T,
                 hipStream_t st) {
    const Cut cut(c.heads, T);
    k_kv_write<DT, D><<<cut.grid, 256, 0, st>>>(c, static_cast<const uint16_t *>(k), ks,
                                                static_cast<const uint16_t *>(v), vs, slots, T, cut.per, cut.groups);
    return hipGetLastError();
}

template <int DT, int D>
hipError_t append(const KvCache &c, const TurnArgs &a, const void *k, int64_t ks, const void *v, int64_t vs,
                  const int32_t *slots, int T, hipStream_t st) {
    const Cut cut(c.heads, T, APPEND_HEADS), q(a.q == nullptr ? 1 : a.n_heads, T, QUERY_HEADS);
    auto *kernel = a.t.pairs ? k_kv_append<DT, D, TURN_PAIRS> : k_kv_append<DT, D, TURN_HALVES>;
    kernel<<<cut.grid + (a.q == nullptr ? 0 : q.grid), 256, 0, st>>>(
        c, a, static_cast<const uint16_t *>(k), ks, static_cast<const uint16_t *>(v), vs, slots, T, cut.per, cut.groups,
        cut.grid, q.per, q.groups);
    return hipGetLastError();
}

template <int DT, int D>
hipError_t read(const KvCache &c, const int32_t *slots, int T, void *k, void *v, hipStream_t st) {
    const Cut cut(c.heads, T);
    k_kv_read<DT, D><<<cut.grid, 256, 0, st>>>(c, slots, T, static_cast<uint16_t *>(k), static_cast<uint16_t *>(v),
                                               cut.per, cut.groups);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_write(const KvCache &c, const void *k, int64_t ks, const void *v, int64_t vs,
                           const int32_t *slots, int T, hipStream_t st) {
    if (c.dtype == DT_F16)
        return c.dim == 128 ? write<DT_F16, 128>(c, k, ks, v, vs, slots, T, st)
                            : write<DT_F16, 64>(c, k, ks, v, vs, slots, T, st);
    return c.dim == 128 ? write<DT_BF16, 128>(c, k, ks, v, vs, slots, T, st)
                        : write<DT_BF16, 64>(c, k, ks, v, vs, slots, T, st);
}

hipError_t launch_kv_append(const KvCache &c, const TurnArgs &turn, const void *k, int64_t ks, const void *v,
                            int64_t vs, const int32_t *slots, int T, hipStream_t st) {
    if (c.dtype == DT_F16)
        return c.dim == 128 ? append<DT_F16, 128>(c, turn, k, ks, v, vs, slots, T, st)
                            : append<DT_F16, 64>(c, turn, k, ks, v, vs, slots, T, st);
    return c.dim == 128 ? append<DT_BF16, 128>(c, turn, k, ks, v, vs, slots, T, st)
                        : append<DT_BF16, 64>(c, turn, k, ks, v, vs, slots, T, st);
}

hipError_t launch_rope_table(const double *freq, double scale, int n_positions, int n, float2 *hi, float2 *lo,
                             hipStream_t st) {
    const long blocks = (static_cast<long>(n_positions) * n + 255) / 256;
    k_rope_table<<<static_cast<unsigned>(blocks < 65536 ? blocks : 65536), 256, 0, st>>>(freq, scale, n_positions, n, hi, lo);
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache &c, const int32_t *slots, int T, void *k, void *v, hipStream_t st) {
    if (c.dtype == DT_F16)
        return c.dim == 128 ? read<DT_F16, 128>(c, slots, T, k, v, st) : read<DT_F16, 64>(c, slots, T, k, v, st);
    return c.dim == 128 ? read<DT_BF16, 128>(c, slots, T, k, v, st) : read<DT_BF16, 64>(c, slots, T, k, v, st);
}

}  // namespace lora
