// kv_cache.hip -- keys and values quantised into the paged cache as they are
// written, and rows of it read back.
//
// A row x of D values (one token, one head) is held as e4m3 elements e and
// one exponent s:  s the least whole number >= KV_MIN_EXP with
// max|x| <= 448 * 2^s,  e = x * 2^-s rounded to e4m3, ties to even.  Scaling
// by a power of two is exact, so the one rounding is the element's.
//
// Bound by memory for long runs (4096 tokens of 32 heads of 128: 101 MB in 23
// us, 4.4 TB/s, and back 101 MB in 18 us, 5.6 TB/s), by the chain slot -> row
// -> store for a decode step (64 tokens: 6 and 5 us).
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

// Elements of a row, N of them as bytes in N / 4 words.
template <int DT, int N>
__device__ __forceinline__ void quantise(const Words<N> &r, int byte, uint32_t (&w)[N / 4]) {
    const float inv = __uint_as_float(static_cast<uint32_t>(2 * KV_EXP_BIAS - byte) << 23);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(r.template at<DT>(4 * i) * inv, r.template at<DT>(4 * i + 1) * inv, 0,
                                                false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(r.template at<DT>(4 * i + 2) * inv, r.template at<DT>(4 * i + 3) * inv, v,
                                            true);
        w[i] = static_cast<uint32_t>(v);
    }
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
template <int DT, int D>
__global__ __launch_bounds__(256) void k_kv_write(KvCache c, const uint16_t *k, int64_t k_stride, const uint16_t *v,
                                                  int64_t v_stride, const int32_t *slots, int n_tokens, int per,
                                                  int groups) {
    constexpr int N = D / LANES;
    __shared__ Window w;
    __shared__ __align__(16) uint8_t turned[2][D * VT_LD];
    const int first = static_cast<int>(blockIdx.x) / groups * TOKENS, h0 = static_cast<int>(blockIdx.x) % groups * per;
    const int h1 = h0 + per < c.heads ? h0 + per : c.heads;
    const int me = threadIdx.x / LANES, l = threadIdx.x % LANES;
    const Tile tile = find_tile(slots, n_tokens, first, c.n_pages << c.page_shift, w);
    if (h0 == 0 && l == 0) {
        const int mine = w.s[15 + me];
        if (first + me < n_tokens && mine != -1 && tile.slot < 0) atomicAdd(c.err, 1ull);
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
    // Writes the key and both exponents, leaves the value's bytes in vw.
    auto put = [&](const Pair &x, long R, uint32_t (&vw)[N / 4]) {
        float ka = 0.0f, va = 0.0f;
        bool fin = true;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float kx = x.k.template at<DT>(i), vx = x.v.template at<DT>(i);
            // A value that is not finite has the exponent bits all set; fmax drops NaN.
            fin &= (__float_as_uint(kx) & 0x7F800000u) != 0x7F800000u;
            fin &= (__float_as_uint(vx) & 0x7F800000u) != 0x7F800000u;
            ka = fmaxf(ka, fabsf(kx));
            va = fmaxf(va, fabsf(vx));
        }
        ka = max16(ka);
        va = max16(va);
        const bool poison = max16(fin ? 0.0f : 1.0f) != 0.0f;
        const int kb = poison ? KV_EXP_BIAS : exp_byte(ka), vb = poison ? KV_EXP_BIAS : exp_byte(va);
        uint32_t kw[N / 4];
        quantise<DT, N>(x.k, kb, kw);
        quantise<DT, N>(x.v, vb, vw);
        if (poison) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) kw[i] = 0x7F7F7F7Fu, vw[i] = 0u;
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
            uint8_t *turn = turned[(head - h0) & 1];
            uint32_t vw[N / 4] = {};
            long R = 0;
            if (tile.single) {
                next = load(first + me, head + 1 < h1 ? head + 1 : head);
                R = row_of(c, tile.slot, head);
                put(x, R, vw);
            }
            if (word) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    turn[(l * N + i) * VT_LD + me] = static_cast<uint8_t>(vw[i / 4] >> (8 * (i % 4)));
            }
            if (tile.any_word) __syncthreads();
            uint8_t *vd = c.v + (R & ~15L) * D + (R & 15);
            if (word) {
#pragma unroll
                for (int i = 0; i < N / 4; ++i) {
                    const int d = l * N + q * (N / 4) + i;
                    uint32_t four;
                    __builtin_memcpy(&four, turn + d * VT_LD + w0, 4);
                    *reinterpret_cast<uint32_t *>(vd - q + d * KV_BLOCK) = four;
                }
            } else if (tile.single) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    vd[(l * N + i) * KV_BLOCK] = static_cast<uint8_t>(vw[i / 4] >> (8 * (i % 4)));
            }
            x = next;
        }
        if (tile.any_word) __syncthreads();  // `turned` is written again
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
            uint8_t *turn = turned[(head - h0) & 1];
            uint32_t vw[N / 4] = {};
            const long R = row_of(c, slot0, head);
            if (there) {
                next = load(token, head + 1 < h1 ? head + 1 : head);
                put(x, R + me, vw);
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
                turn[(l * N + i) * VT_LD + me] = static_cast<uint8_t>(vw[i / 4] >> (8 * (i % 4)));
            __syncthreads();
            // 256 threads x N bytes: the block's D x 16 bytes in order.
            const int at = threadIdx.x * N, d = at / KV_BLOCK, part = at % KV_BLOCK;
            uint8_t *vd = c.v + R * D + at;
            const uint8_t *from = turn + d * VT_LD + part;
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
        __syncthreads();  // `turned` is written again
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
// in flight.
struct Cut {
    int per, groups;
    unsigned grid;
    Cut(const KvCache &c, int T) {
        const int tiles = (T + TOKENS - 1) / TOKENS;
        per = tiles * static_cast<long>(c.heads) >= 4 * FULL_WGS ? 4 : 1;
        groups = (c.heads + per - 1) / per;
        grid = static_cast<unsigned>(tiles) * static_cast<unsigned>(groups);
    }
};

template <int DT, int D>
hipError_t write(const KvCache &c, const void *k, int64_t ks, const void *v, int64_t vs, const int32_t *slots, int T,
                 hipStream_t st) {
    const Cut cut(c, T);
    k_kv_write<DT, D><<<cut.grid, 256, 0, st>>>(c, static_cast<const uint16_t *>(k), ks,
                                                static_cast<const uint16_t *>(v), vs, slots, T, cut.per, cut.groups);
    return hipGetLastError();
}

template <int DT, int D>
hipError_t read(const KvCache &c, const int32_t *slots, int T, void *k, void *v, hipStream_t st) {
    const Cut cut(c, T);
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

hipError_t launch_kv_read(const KvCache &c, const int32_t *slots, int T, void *k, void *v, hipStream_t st) {
    if (c.dtype == DT_F16)
        return c.dim == 128 ? read<DT_F16, 128>(c, slots, T, k, v, st) : read<DT_F16, 64>(c, slots, T, k, v, st);
    return c.dim == 128 ? read<DT_BF16, 128>(c, slots, T, k, v, st) : read<DT_BF16, 64>(c, slots, T, k, v, st);
}

}  // namespace lora
