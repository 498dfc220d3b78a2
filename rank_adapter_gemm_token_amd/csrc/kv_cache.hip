// kv_cache.hip -- keys and values quantised into the paged cache as they are
// written, and rows of it read back.
//
// A row x of D values (one token, one head) is held as e4m3 elements e and
// one exponent s:  s the least whole number >= KV_MIN_EXP with
// max|x| <= 448 * 2^s,  e = x * 2^-s rounded to e4m3, ties to even.  Scaling
// by a power of two is exact, so the one rounding is the element's.
#include "dtype.hpp"
#include "kv_internal.hpp"

namespace lora {

namespace {

typedef float f32x2_t __attribute__((ext_vector_type(2)));

constexpr int TOKENS = 16;   // tokens of a workgroup: 16 lanes each
constexpr int LANES = 16;
constexpr int VT_LD = 20;    // bytes of one element's 16 tokens in LDS, padded

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

// A value as the write sees it: its magnitude for the row's maximum, and
// whether it is finite.
template <int N>
struct Row {
    float x[N];
};

template <int DT, int N>
__device__ __forceinline__ Row<N> load_row(const uint16_t *p) {
    Row<N> r;
    uint16_t w[N];
    if constexpr (N == 8)
        *reinterpret_cast<u32x4_t *>(w) = *reinterpret_cast<const u32x4_t *>(p);
    else
        *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) r.x[i] = Elem<DT>::to_f(w[i]);
    return r;
}

// Elements of a row, N of them as bytes in N / 4 words.
template <int N>
__device__ __forceinline__ void quantise(const Row<N> &r, int byte, uint32_t (&w)[N / 4]) {
    const float inv = __uint_as_float(static_cast<uint32_t>(2 * KV_EXP_BIAS - byte) << 23);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(r.x[4 * i] * inv, r.x[4 * i + 1] * inv, 0, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(r.x[4 * i + 2] * inv, r.x[4 * i + 3] * inv, v, true);
        w[i] = static_cast<uint32_t>(v);
    }
}

// The tokens a workgroup deals with.  It owns 16 neighbouring tokens of the
// call.  Where 16 neighbours of the call fill a block of 16 rows in order,
// the block's values are turned in LDS and move as whole words; the workgroup
// that owns the block's first token takes all of it.  The other tokens it
// owns move a byte at a time.
struct Tile {
    int slot;        // of the lane's own token, or -1
    bool single;     // not part of a full block
    int lead;        // first token of the block led from here, or -1 (uniform)
};

__device__ __forceinline__ Tile find_tile(const int32_t *slots, int n_tokens, int first, int n_rows, int *s) {
    // s: the slots of tokens first - 15 .. first + 30.
    const int t = threadIdx.x;
    if (t < 46) {
        const int at = first - 15 + t;
        s[t] = at >= 0 && at < n_tokens ? slots[at] : -1;
    }
    __syncthreads();
    const int me = t / LANES;  // the lane's token: s[15 + me]
    Tile r;
    const int mine = s[15 + me];
    r.slot = mine >= 0 && mine < n_rows ? mine : -1;
    // The block that token `me` would be part of starts `mine % 16` before it.
    auto full = [&](int lead_at, int slot0) {
        if (lead_at < 0 || lead_at + 15 >= 46) return false;
        bool ok = slot0 >= 0 && slot0 <= n_rows - KV_BLOCK;
#pragma unroll
        for (int i = 0; i < KV_BLOCK; ++i) ok &= s[lead_at + i] == slot0 + i;
        return ok;
    };
    r.single = r.slot >= 0 && !full(15 + me - (r.slot & 15), r.slot & ~15);
    // A token leads when its slot is a block's first; two leaders are at
    // least 16 tokens apart, so a workgroup has one at most.
    const bool leads = r.slot >= 0 && (r.slot & 15) == 0 && !r.single;
    int *lead = s + 46;
    if (t == 0) *lead = -1;
    __syncthreads();
    if (leads && (t & 15) == 0) *lead = me;
    __syncthreads();
    r.lead = uniform(*lead);
    return r;
}

__device__ __forceinline__ long row_of(const KvCache &c, int slot, int head) {
    const int page = slot >> c.page_shift, off = slot & ((1 << c.page_shift) - 1);
    return ((static_cast<long>(page) * c.heads + head) << c.page_shift) + off;
}

template <int DT, int D>
__global__ __launch_bounds__(256) void k_kv_write(KvCache c, const uint16_t *k, int64_t k_stride, const uint16_t *v,
                                                  int64_t v_stride, const int32_t *slots, int n_tokens) {
    constexpr int N = D / LANES;
    __shared__ int s[48];
    __shared__ __align__(16) uint8_t turned[D * VT_LD];
    const int first = blockIdx.x * TOKENS, head = blockIdx.y;
    const int me = threadIdx.x / LANES, l = threadIdx.x % LANES;
    const Tile tile = find_tile(slots, n_tokens, first, c.n_pages << c.page_shift, s);
    if (head == 0 && l == 0) {
        const int mine = s[15 + me];
        if (first + me < n_tokens && mine != -1 && tile.slot < 0) atomicAdd(c.err, 1ull);
    }

    auto rows = [&](int token, int slot, uint32_t (&vw)[N / 4], long &R) {
        const Row<N> kr = load_row<DT, N>(k + token * k_stride + static_cast<long>(head) * D + l * N);
        const Row<N> vr = load_row<DT, N>(v + token * v_stride + static_cast<long>(head) * D + l * N);
        float ka = 0.0f, va = 0.0f;
        bool fin = true;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // A value that is not finite has the exponent bits all set; fmax drops NaN.
            fin &= (__float_as_uint(kr.x[i]) & 0x7F800000u) != 0x7F800000u;
            fin &= (__float_as_uint(vr.x[i]) & 0x7F800000u) != 0x7F800000u;
            ka = fmaxf(ka, fabsf(kr.x[i]));
            va = fmaxf(va, fabsf(vr.x[i]));
        }
        ka = max16(ka);
        va = max16(va);
        const bool poison = max16(fin ? 0.0f : 1.0f) != 0.0f;
        const int kb = poison ? KV_EXP_BIAS : exp_byte(ka), vb = poison ? KV_EXP_BIAS : exp_byte(va);
        uint32_t kw[N / 4];
        quantise<N>(kr, kb, kw);
        quantise<N>(vr, vb, vw);
        if (poison) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) kw[i] = 0x7F7F7F7Fu, vw[i] = 0u;
        }
        R = row_of(c, slot, head);
        uint32_t *kd = reinterpret_cast<uint32_t *>(c.k + (R & ~15L) * D + key_byte<D>(R & 15, l * N));
#pragma unroll
        for (int i = 0; i < N / 4; ++i) kd[i] = kw[i];
        if (l == 0) {
            c.kexp[R] = static_cast<uint8_t>(kb);
            c.vinv[R] = static_cast<uint8_t>(poison ? KV_POISON : 2 * KV_EXP_BIAS - vb);
        }
    };

    // The cross-lane maxima stay within a token's 16 lanes, which go the same way.
    if (tile.single) {
        uint32_t vw[N / 4];
        long R;
        rows(first + me, tile.slot, vw, R);
        uint8_t *vd = c.v + (R & ~15L) * D + (R & 15) + l * N * KV_BLOCK;
#pragma unroll
        for (int i = 0; i < N; ++i) vd[i * KV_BLOCK] = static_cast<uint8_t>(vw[i / 4] >> (8 * (i % 4)));
    }
    if (tile.lead < 0) return;
    const int slot0 = s[15 + tile.lead];
    uint32_t vw[N / 4];
    long R;
    rows(first + tile.lead + me, slot0 + me, vw, R);
#pragma unroll
    for (int i = 0; i < N; ++i) turned[(l * N + i) * VT_LD + me] = static_cast<uint8_t>(vw[i / 4] >> (8 * (i % 4)));
    __syncthreads();
    // 256 threads x N bytes: the block's D x 16 bytes in order.
    const int at = threadIdx.x * N, d = at / KV_BLOCK, part = at % KV_BLOCK;
    uint32_t *vd = reinterpret_cast<uint32_t *>(c.v + (R & ~15L) * D + at);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) vd[i] = *reinterpret_cast<const uint32_t *>(turned + d * VT_LD + part + 4 * i);
}

template <int DT, int D>
__global__ __launch_bounds__(256) void k_kv_read(KvCache c, const int32_t *slots, int n_tokens, uint16_t *k,
                                                 uint16_t *v) {
    constexpr int N = D / LANES;
    __shared__ int s[48];
    __shared__ __align__(16) uint8_t turned[D * VT_LD];
    const int first = blockIdx.x * TOKENS, head = blockIdx.y;
    const int me = threadIdx.x / LANES, l = threadIdx.x % LANES;
    const Tile tile = find_tile(slots, n_tokens, first, c.n_pages << c.page_shift, s);

    // N values of a row: their elements in words w, all scaled by 2^(byte - 127).
    auto put = [&](uint16_t *to, int token, const uint32_t (&w)[N / 4], int byte, bool poison) {
        const float f = __uint_as_float(static_cast<uint32_t>(byte) << 23);
        uint16_t o[N];
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), false);
            const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), true);
            const float x[4] = {lo.x * f, lo.y * f, hi.x * f, hi.y * f};
#pragma unroll
            for (int j = 0; j < 4; ++j) o[4 * i + j] = poison ? Elem<DT>::qnan : Elem<DT>::from_f(x[j]);
        }
        uint16_t *at = to + (static_cast<long>(token) * c.heads + head) * D + l * N;
        if constexpr (N == 8)
            *reinterpret_cast<u32x4_t *>(at) = *reinterpret_cast<const u32x4_t *>(o);
        else
            *reinterpret_cast<uint2 *>(at) = *reinterpret_cast<const uint2 *>(o);
    };
    auto keys = [&](int token, long R, bool poison) {
        uint32_t w[N / 4];
#pragma unroll
        for (int i = 0; i < N / 4; ++i) w[i] = reinterpret_cast<const uint32_t *>(c.k + (R & ~15L) * D + key_byte<D>(R & 15, l * N))[i];
        put(k, token, w, c.kexp[R], poison);
    };

    if (first + me < n_tokens && (tile.single || tile.slot < 0)) {
        const int token = first + me;
        uint32_t w[N / 4] = {};
        if (tile.slot < 0) {
            // Nothing is held for this token: an explicit NaN row.
            if (head == 0 && l == 0) atomicAdd(c.err, 1ull);
            put(k, token, w, 0, true);
            put(v, token, w, 0, true);
        } else {
            const long R = row_of(c, tile.slot, head);
            const int vi = c.vinv[R];
            keys(token, R, vi == KV_POISON);
            const uint8_t *vs = c.v + (R & ~15L) * D + (R & 15) + l * N * KV_BLOCK;
#pragma unroll
            for (int i = 0; i < N; ++i) w[i / 4] |= static_cast<uint32_t>(vs[i * KV_BLOCK]) << (8 * (i % 4));
            put(v, token, w, 2 * KV_EXP_BIAS - vi, vi == KV_POISON);
        }
    }
    if (tile.lead < 0) return;
    const int token = first + tile.lead + me;
    const long R = row_of(c, s[15 + tile.lead] + me, head);
    const int vi = c.vinv[R];
    const int at = threadIdx.x * N, d = at / KV_BLOCK, part = at % KV_BLOCK;
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = reinterpret_cast<const uint32_t *>(c.v + (R & ~15L) * D + at)[i];
    keys(token, R, vi == KV_POISON);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) *reinterpret_cast<uint32_t *>(turned + d * VT_LD + part + 4 * i) = w[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) w[i / 4] |= static_cast<uint32_t>(turned[(l * N + i) * VT_LD + me]) << (8 * (i % 4));
    put(v, token, w, 2 * KV_EXP_BIAS - vi, vi == KV_POISON);
}

template <int DT, int D>
hipError_t write(const KvCache &c, const void *k, int64_t ks, const void *v, int64_t vs, const int32_t *slots, int T,
                 hipStream_t st) {
    k_kv_write<DT, D><<<dim3((T + TOKENS - 1) / TOKENS, c.heads), 256, 0, st>>>(
        c, static_cast<const uint16_t *>(k), ks, static_cast<const uint16_t *>(v), vs, slots, T);
    return hipGetLastError();
}

template <int DT, int D>
hipError_t read(const KvCache &c, const int32_t *slots, int T, void *k, void *v, hipStream_t st) {
    k_kv_read<DT, D><<<dim3((T + TOKENS - 1) / TOKENS, c.heads), 256, 0, st>>>(
        c, slots, T, static_cast<uint16_t *>(k), static_cast<uint16_t *>(v));
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
