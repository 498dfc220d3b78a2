// attend.hip -- attention of a batch's new tokens over the quantised cache,
// with the prefix that a group of sequences shares computed once for all of
// its query rows.
//
// In the log2 domain, for one query row over keys t with scores s_t, value
// exponents b_t (v_t = 2^b_t v8_t) and c = scale * log2(e), against an m near
// max(c s_t + b_t) - 15:
//     y_t = c s_t + (b_t - m),   p_t = 2^y_t
//     O = sum p_t v8_t,    l = sum p_t 2^-b_t,   out = O / l,
//     lse = ln 2 * (m + log2 l).
// The value's exponent goes into the weight, so that the values' elements
// feed the matrix instruction as they are and p_t is at most 2^15 for values
// of any size: exact enough in fp16.  m has at most 15 bits after the
// point, so b_t - m is exact and y_t is rounded once, where it is small.
//
// Both products are computed transposed, S^T = K Q^T and O^T = V^T P^T: the
// keys' rows of S^T come out in the lanes that P^T needs them in, so the
// weights never leave the registers.  A wave takes 64 keys at a time straight
// from the cache into registers, 16 bytes a lane; no key is read by two waves
// for the same rows.  Each wave keeps m, l and O of its own keys; the four
// waves of a workgroup either work on one item and join at the end, or each
// on an item of its own.
//
// What bounds it.  Few rows a key: memory; 64 sequences of 4096 own tokens, 32
// heads of 128, stream at 6.7 TB/s.  Many rows on one prefix: issue slots; a
// tile of 64 keys and 32 rows is 454 vector instructions, 64 of them MFMA
// (each costs 11 issue cycles beside others), about 2390 cycles.  256
// sequences of one own token on a prefix of 12288 take 82 us with the join,
// 0.63 PFLOP/s.  32 rows fill the 256 registers that leave two waves a SIMD;
// 16 would widen every element twice as often.
#include <atomic>
#include <type_traits>

#include "attend_plan.hpp"
#include "dtype.hpp"
#include "kv_internal.hpp"

namespace lora {

namespace {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr float LN2 = 0.69314718055994530942f;
// The largest weight stands as high as fp16 reaches, at most at 2^TOP: a
// weight keeps its 11 bits down to 2^-29 of the largest and counts down to
// 2^-40, so that the many light keys of a long sequence, which are all in l,
// are all in O too.  A row's m is moved when a y passes TOP, so that its
// largest y stands slack() below.  With 32 rows moving costs, and most tiles
// scale nothing (light keys then count down to 2^-32).  With 16, memory is the
// bound: the largest p is a power of two, which fp16 holds exactly, and a row
// with one key far above the others keeps all its bits.
constexpr float TOP = 15.0f;
constexpr float slack(int QB) { return QB == 1 ? 0.0f : 8.0f; }

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// l is scaled by 2^x in two halves: v_exp flushes below 2^-126, and between a
// row of zeros (b = -64) and the largest of bf16 (b = 120) m moves by 184,
// which l's 2^64 of that row makes up for.
__device__ __forceinline__ float half_of(float x) { return exp2_fast(0.5f * x); }

// Whether any of 16 value exponents is above 31 (a byte of vinv below 96: bit
// 7 clear, and bit 6 or 5).
__device__ __forceinline__ bool any_above_31(const u32x4_t &vinv) {
    uint32_t high = 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) high &= vinv[i] | ((vinv[i] << 1) & (vinv[i] << 2));
    return high != 0x80808080u;
}

// bf16 keys are this power of two smaller as operands, the scale of their
// scores larger.
constexpr uint32_t KEXP_LESS = 8;

// Eight e4m3 elements (two words) as an MFMA operand, scaled by a power of two.
template <int DT>
__device__ __forceinline__ typename Elem<DT>::vec8 widen(uint32_t lo, uint32_t hi, float scale) {
    if constexpr (DT == DT_F16) {
        const f16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, scale, false);
        const f16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, scale, true);
        const f16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, scale, false);
        const f16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, scale, true);
        return f16x8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
    } else {
        const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
        const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
        const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
        const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
        return bf16x8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
    }
}

__device__ __forceinline__ uint32_t byte_of(const u32x4_t &w, int i) { return (w[i / 4] >> (8 * (i % 4))) & 255u; }

// 2^(byte - 127) (byte 0: 0).
__device__ __forceinline__ float pow2(uint32_t byte) { return __uint_as_float(byte << 23); }

// The values of lanes r, r + 16, r + 32 and r + 48 joined by op, to all four:
// neighbouring rows of 16 lanes swap, then the halves of the wave.
template <typename Op>
__device__ __forceinline__ float over_g(float v, Op op) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return op(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

__device__ __forceinline__ float max_over_g(float v) {
    return over_g(v, [](float x, float y) { return fmaxf(x, y); });
}

__device__ __forceinline__ float sum_over_g(float v) {
    return over_g(v, [](float x, float y) { return x + y; });
}

// The token (of an item) of a query row: row / gq for row < 64, gq <= 32.
__device__ __forceinline__ int token_of_row(const AttendArgs &a, int row) { return (row * a.gq_inv) >> 16; }

// LDS: for each wave ATTEND_ROWS rows of D + 4 floats -- its item's queries and
// tokens, then its O for the join -- and for each of its rows m and l.  The
// wave's part is at the same place whatever its item's rows: the waves of a
// workgroup may have items of different sizes.
constexpr int wave_floats(int D) { return ATTEND_ROWS * (D + 4); }
constexpr int lds_floats(int D) { return ATTEND_WAVES * (wave_floats(D) + ATTEND_ROWS * 2); }

// Partial results are joined either in the launch (HERE), by the workgroup or
// wave that adds a token's last one, or by a second launch.  HERE they go to
// the agent's coherence point and come from there: the caches of another XCD
// may hold a copy that an earlier call left.
template <bool HERE>
__device__ __forceinline__ void put8(float *p, float x, float y) {
    if constexpr (!HERE) {
        *reinterpret_cast<float2 *>(p) = float2{x, y};
        return;
    }
    __hip_atomic_store(reinterpret_cast<uint64_t *>(p),
                       static_cast<uint64_t>(__float_as_uint(y)) << 32 | __float_as_uint(x), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}

template <bool HERE>
__device__ __forceinline__ float2 get8(const float *p) {
    if constexpr (!HERE) return *reinterpret_cast<const float2 *>(p);
    const uint64_t w =
        __hip_atomic_load(reinterpret_cast<const uint64_t *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return float2{__uint_as_float(static_cast<uint32_t>(w)), __uint_as_float(static_cast<uint32_t>(w >> 32))};
}

// Four of an output row's elements (d .. d + 3).
template <int DT, int D>
__device__ __forceinline__ void put_out(const AttendArgs &a, int token, int head, int d, f32x4_t sum, float M, float L) {
    const long at = static_cast<long>(token) * a.heads + head;
    // No key seen: zeros.  (L is NaN, not 0, where a seen key is poisoned.)
    const float f = L == 0.0f ? 0.0f : 1.0f / L;
    typename Elem<DT>::raw w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = Elem<DT>::from_f(sum[j] * f);
    *reinterpret_cast<uint2 *>(a.out + at * D + d) = *reinterpret_cast<const uint2 *>(w);
    if (d == 0 && a.lse != nullptr) a.lse[at] = LN2 * (M + log2f(L));
}

// Four of a row's elements, of token i of the item: a partial result, or the output.
template <int DT, int D, bool HERE>
__device__ __forceinline__ void emit(const AttendArgs &a, const AttendItem &it, int token, int i, int head, int d,
                                     f32x4_t sum, float M, float L) {
    if (it.part0 < 0) return put_out<DT, D>(a, token, head, d, sum, M, L);
    const long at = static_cast<long>(it.part0 + i) * a.heads + head;
    put8<HERE>(a.part_o + at * D + d, sum[0], sum[1]);
    put8<HERE>(a.part_o + at * D + d + 2, sum[2], sum[3]);
    if (d == 0) put8<HERE>(a.part_ml + at * 2, M, L);
}

// Counts this item's partial results of token i (its stores have completed);
// whether they were the last of the token's for this key/value head.
__device__ __forceinline__ bool count_parts(const AttendArgs &a, const AttendItem &it, const AttendToken *toks, int i,
                                            int kvh) {
    unsigned *cnt = a.count + static_cast<long>(it.tok0 + i) * a.kv_heads + kvh;
    const unsigned all = static_cast<unsigned>(toks[i].n[0] + toks[i].n[1]);
    if (__hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != all - 1) return false;
    __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

// Joins a token's partial results: four elements of one row.
template <int DT, int D, bool HERE>
__device__ __forceinline__ void join_parts(const AttendArgs &a, const AttendToken &tk, int head, int d) {
    const int n = tk.n[0] + tk.n[1];
    auto row = [&](int j) {
        const int p = j < tk.n[0] ? tk.part[0] + j * tk.stride[0] : tk.part[1] + (j - tk.n[0]) * tk.stride[1];
        return static_cast<long>(p) * a.heads + head;
    };
    constexpr int STEP = ATTEND_JOIN_STEP;  // results asked for together
    float M = -INFINITY, L = 0.0f;
    f32x4_t sum{0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < n; j += STEP) {
        float2 ml[STEP], lo[STEP], hi[STEP];
#pragma unroll
        for (int k = 0; k < STEP; ++k) {
            const long at = row(j + k < n ? j + k : n - 1);
            ml[k] = get8<HERE>(a.part_ml + at * 2);
            lo[k] = get8<HERE>(a.part_o + at * D + d);
            hi[k] = get8<HERE>(a.part_o + at * D + d + 2);
        }
#pragma unroll
        for (int k = 0; k < STEP; ++k) {
            if (j + k >= n) break;
            const float to = fmaxf(M, ml[k].x);
            const float ref = to == -INFINITY ? 0.0f : to;
            const float h0 = half_of(M - ref), h1 = half_of(ml[k].x - ref);
            M = to;
            L = L * h0 * h0 + ml[k].y * h1 * h1;
            sum = sum * (h0 * h0) + f32x4_t{lo[k].x, lo[k].y, hi[k].x, hi[k].y} * (h1 * h1);
        }
    }
    put_out<DT, D>(a, tk.token, head, d, sum, M, L);
}

// The lane's number, counted where it is asked for: a value that the compiler
// does not keep, and spill, in between.
__device__ __forceinline__ int lane_anew() {
    int lane;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(lane));
    return lane;
}

// One wave's item for one key/value head.  QB blocks of 16 query rows; row =
// token of the item x query head of the key head.
template <int DT, int D, int QB, bool HERE>
__device__ __forceinline__ void attend_item(const AttendArgs &a, const AttendItem &it, const AttendToken *toks,
                                            const int32_t *pages, const uint32_t *nodes, int kvh, int wave,
                                            float *lds) {
    using V8 = typename Elem<DT>::vec8;
    constexpr int NC = D / 64;   // 64-element parts of a key's row: 16 bytes a lane each
    constexpr int NH = D / 16;   // 16-element rows of V^T
    constexpr int ROWS = 16 * QB;
    // Made anew for each item, in the branch for masks and after the loop: the
    // compiler would keep, and spill, addresses made of it over all of them (3 to
    // 8 registers; one sequence of 2001 tokens 9.9 us instead of 9.4).
    int lane = lane_anew(), r = lane & 15, g = lane >> 4;
    const bool joined = (it.flags & ATTEND_JOINED) != 0;
    const int step = joined ? ATTEND_WAVES : 1;

    // bm = 127 - m: y = c s + (bm - vinv).  thr: what y must pass to move m.
    float bm[QB], thr[QB], l[QB];
    f32x4_t o[NH][QB];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
        bm[b] = static_cast<float>(KV_EXP_BIAS);
        thr[b] = -INFINITY;  // until the row has seen a key
        l[b] = 0.0f;
#pragma unroll
        for (int h = 0; h < NH; ++h) o[h][b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // p_t 2^-b_t is l's term as long as p_t is not flushed: while no m was made
    // of an exponent above 31, that takes a term below 2^-38 of the largest (b
    // = -64).  After one was (values of 10^12 and more, in bf16 alone), terms
    // are made of 2^(y_t - b_t) = 2^(c s_t - m) by themselves, 2^40 larger, so
    // that none that counts is flushed: one more exponential a weight.
    constexpr bool SPREAD = DT == DT_BF16;
    bool spread = false;

    // Of a tile of 64 keys, block j of 16 is keys 16 j .. 16 j + 15.  S^T is
    // computed in four products x = 0..3 whose row 4 j + i is key 16 j + 4 x
    // + i; lane (r, g) then holds the scores of keys 16 g .. 16 g + 15, in
    // order, of query row r.  Keys: lane (r, g) loads elements 64 c + 16 g ..
    // + 15 of key 16 (r / 4) + 4 x + r % 4.  Values: lane (r, g) loads element 16 h +
    // r of block g's 16 keys.
    const int t_end = (it.end + ATTEND_TILE - 1) / ATTEND_TILE;
    int t = it.begin / ATTEND_TILE + (joined ? wave : 0);
    const int last_block = it.end > 0 ? (it.end - 1) / KV_BLOCK : 0;
    const int page_mask = (1 << a.page_shift) - 1;

    // The 16 rows of block `blk` of keys (past the end: the last one): their
    // page's number, and with that their first row.
    auto block_page = [&](int blk) {
        blk = blk < last_block ? blk : last_block;
        return pages[(blk * KV_BLOCK) >> a.page_shift];
    };
    auto block_row = [&](int blk, int page) {
        blk = blk < last_block ? blk : last_block;
        return ((static_cast<long>(page) * a.kv_heads + kvh) << a.page_shift) + ((blk * KV_BLOCK) & page_mask);
    };
    // The key exponents of lane (r, g): of the keys whose elements it loads, or
    // (fp16) of those whose scores it holds, the values' rows.
    constexpr bool KEXP_LATE = DT == DT_F16;
    // Loads return in the order of their issue.  A tile's keys and exponents
    // are issued one tile ahead, after the scores of the tile before, its
    // values after that tile's second product; the pages of the tile after
    // that are looked up between the two, and first looked at when they are
    // needed, so that no wait for one of these covers a later one.  Blocks past
    // the end read the last one again.
    //
    // Keys of few rows have no other reader: they pass the L2 by, which
    // streams faster (64 sequences of 4096 tokens: 6.7 TB/s instead of 6.1)
    // and leaves it to the prefixes that several blocks of rows read.
    u32x4_t kw[4][NC], vw[NH], ke, ve;
    auto load16 = [&](const uint8_t *p) {
        const u32x4_t *w = reinterpret_cast<const u32x4_t *>(p);
        if constexpr (QB == 1)
            return __builtin_nontemporal_load(w);
        else
            return *w;
    };
    auto load_k = [&](long R, long vR) {
        const uint8_t *p = a.k + R * D + key_byte<D>(r & 3, g * 16);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int c = 0; c < NC; ++c) kw[x][c] = load16(p + key_byte<D>(4 * x, c * 64));
        ke = *reinterpret_cast<const u32x4_t *>(a.kexp + (KEXP_LATE ? vR : R));
    };
    auto load_v = [&](long R) {
        const uint8_t *p = a.v + R * D + r * KV_BLOCK;
#pragma unroll
        for (int h = 0; h < NH; ++h) vw[h] = load16(p + h * 16 * KV_BLOCK);
    };
    const int kb0 = 4 * t + (r >> 2), vb0 = 4 * t + g;
    int kp = 0, vp = 0;
    if (t < t_end) {
        kp = block_page(kb0);
        vp = block_page(vb0);
    }

    // Queries: lane (r, g) holds row r of each block, elements 64 c + 16 g + 8
    // h .. + 7, in LDS (16 bytes a lane): in registers they would push the
    // loop over 256 and its spills would wait for the prefetch.  The wave's
    // part of LDS is its own until the join.  They are asked for before the
    // first keys, which need as many reads before them (the page; the token).
    u32x4_t *qf = reinterpret_cast<u32x4_t *>(lds + wave * wave_floats(D)) + lane;
    static_assert(QB * 2 * NC * 256 + ROWS <= wave_floats(D), "the queries and tokens fit the wave's part");
    u32x4_t q0[QB][2 * NC];
    int tok[QB], head[QB];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
        const int row = b * 16 + r, i = token_of_row(a, row);
        const int at = i < it.n_tok ? i : 0;
        head[b] = kvh * a.gq + row - i * a.gq;
        tok[b] = toks[at].token;
    }
#pragma unroll
    for (int b = 0; b < QB; ++b) {
        const uint16_t *q = a.q + tok[b] * a.q_stride + static_cast<long>(head[b]) * D;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                q0[b][2 * c + h] = *reinterpret_cast<const u32x4_t *>(q + c * 64 + g * 16 + h * 8);
    }
    // Below this every row sees every key: of a tree's item the sequence's
    // tokens before the new ones.
    const bool in_tree = (it.flags & ATTEND_TREE) != 0;
    const int before = it.limit0 - 1 - (it.flags >> ATTEND_FIRST_SHIFT);
    const int sure = in_tree ? before : it.limit0, all = sure < it.end ? sure : it.end;
    __builtin_amdgcn_sched_barrier(0);
    if (t < t_end) {
        const long vR = block_row(vb0, vp);
        load_k(block_row(kb0, kp), vR);
        ve = *reinterpret_cast<const u32x4_t *>(a.vinv + vR);
        kp = block_page(kb0 + 4 * step);
        vp = block_page(vb0 + 4 * step);
        __builtin_amdgcn_sched_barrier(0);
        load_v(vR);
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int b = 0; b < QB; ++b)
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i) qf[(b * 2 * NC + i) * 64] = q0[b][i];
    // The rows' tokens, behind the queries.
    auto token_in_lds = [&] { return reinterpret_cast<int *>(lds + wave * wave_floats(D) + QB * 2 * NC * 256); };
    if (g == 0)
#pragma unroll
        for (int b = 0; b < QB; ++b) token_in_lds()[b * 16 + r] = tok[b];

    auto tile = [&](auto more) __attribute__((always_inline)) {
        asm volatile("" ::: "memory");  // the queries are read again, not kept
        const int key0 = t * ATTEND_TILE;
        // Scores.  bf16 holds any element times its scale (2^KEXP_LESS below it:
        // the largest row's elements reach 2^128), which the conversion takes
        // along.  fp16 does not -- small keys beside a large
        // one would lose bits, also to one that the row does not see -- so
        // there the elements are converted as they are, which is exact, and
        // the scale goes into the score.
        f32x4_t s[4][QB];
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int b = 0; b < QB; ++b) s[x][b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                V8 qv[QB];
#pragma unroll
                for (int b = 0; b < QB; ++b) qv[b] = __builtin_bit_cast(V8, qf[(b * 2 * NC + 2 * c + h) * 64]);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t byte = __builtin_amdgcn_ubfe(ke[x], 8 * (r & 3), 8);
                    const float scale = KEXP_LATE ? 1.0f : pow2(byte - KEXP_LESS);
                    const V8 kf = widen<DT>(kw[x][c][2 * h], kw[x][c][2 * h + 1], scale);
#pragma unroll
                    for (int b = 0; b < QB; ++b) s[x][b] = Elem<DT>::mfma(kf, qv[b], s[x][b]);
                }
            }
        __builtin_amdgcn_sched_barrier(0);
        const u32x4_t vi4 = ve, ki4 = ke;
        long vR = 0;
        if constexpr (more) {
            const int kb1 = 4 * (t + step) + (r >> 2), vb1 = 4 * (t + step) + g;
            vR = block_row(vb1, vp);
            load_k(block_row(kb1, kp), vR);
            ve = *reinterpret_cast<const u32x4_t *>(a.vinv + vR);
            kp = block_page(kb1 + 4 * step);
            vp = block_page(vb1 + 4 * step);
        }

        float top[QB];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float vi = static_cast<float>(byte_of(vi4, i));
            const float c = KEXP_LATE ? a.scale * pow2(byte_of(ki4, i)) : a.scale;
#pragma unroll
            for (int b = 0; b < QB; ++b) s[i / 4][b][i % 4] = fmaf(s[i / 4][b][i % 4], c, bm[b] - vi);
        }
        if constexpr (more) {
            // A load after every six of these: in one burst the wave would
            // stand still for most of them.
#pragma unroll
            for (int i = 0; i < 4 * NC + 4; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);  // a read from memory
                __builtin_amdgcn_sched_group_barrier(0x2, 6, 0);   // VALU
            }
        }
        if (uniform(key0 + ATTEND_TILE > all)) {
            asm volatile("");  // a branch: as selects it would cost every tile 100 instructions
            const int lane = lane_anew(), r = lane & 15, g = lane >> 4;
            uint32_t hidden[QB];  // bit i: key 16 g + i of the tile
            if (in_tree) {
                // Lane n looks at key key0 + n, whose node is at that place of
                // the shifted list (which reaches a tile past the nodes on both
                // sides), for one token of the item after the other.
                const int key = key0 + lane;
                const uint32_t other = nodes[key - it.limit0 + 1], mine = nodes[lane < it.n_tok ? lane : 0];
#pragma unroll
                for (int b = 0; b < QB; ++b) hidden[b] = 0;
                for (int n = 0; n < it.n_tok; ++n) {
                    const uint32_t node = __builtin_amdgcn_readlane(mine, n);
                    const unsigned long long all =
                        __ballot(key >= before && (key >= it.limit0 + n || !attend_above(other, node)));
                    const uint32_t half = g < 2 ? static_cast<uint32_t>(all) : static_cast<uint32_t>(all >> 32);
#pragma unroll
                    for (int b = 0; b < QB; ++b)
                        if (token_of_row(a, b * 16 + r) == n) hidden[b] = half >> (16 * (g & 1));
                }
            } else {
#pragma unroll
                for (int b = 0; b < QB; ++b) {
                    const int i = token_of_row(a, b * 16 + r);
                    const int seen = it.limit0 + ((it.flags & ATTEND_STEP) && i < it.n_tok ? i : 0);
                    const int n = (seen < it.end ? seen : it.end) - (key0 + 16 * g);  // of the lane's keys
                    hidden[b] = n >= 16 ? 0u : n <= 0 ? 0xFFFFu : 0xFFFFu << n;
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int b = 0; b < QB; ++b)
                    if ((hidden[b] >> i) & 1) s[i / 4][b][i % 4] = -INFINITY;
        }
        bool moves = false;
#pragma unroll
        for (int b = 0; b < QB; ++b) {
            float v = s[0][b][0];
#pragma unroll
            for (int i = 1; i < 16; ++i) v = fmaxf(v, s[i / 4][b][i % 4]);
            top[b] = v;
            moves |= v > thr[b];
        }
        // The lanes of a row agree on m, so they only have to look at each
        // other's scores when it moves.
        if (__any(moves)) {
            if constexpr (SPREAD) spread |= __any(any_above_31(vi4));
#pragma unroll
            for (int b = 0; b < QB; ++b) {
                // A row with no key yet, or with an infinite score, stays.
                const float most = max_over_g(top[b]);
                const float unit = fabsf(most) < 256.0f ? 32768.0f : 1.0f;
                const float to = bm[b] - (rintf(most * unit) * (1.0f / unit) - (TOP - slack(QB)));
                const bool move = most > thr[b] && fabsf(to) < INFINITY;
                const float d = move ? bm[b] - to : 0.0f;
                const float h = move && thr[b] > -INFINITY ? half_of(-d) : 1.0f, f = h * h;
                thr[b] = move ? TOP : thr[b];
                bm[b] -= d;
                l[b] = l[b] * h * h;
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i / 4][b][i % 4] -= d;
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[h][b][i] *= f;
            }
        }
        if (SPREAD && spread) {
            asm volatile("");  // a branch
#pragma unroll
            for (int b = 0; b < QB; ++b) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    sum += exp2_fast(s[i / 4][b][i % 4] + (static_cast<float>(byte_of(vi4, i)) - KV_EXP_BIAS + 40.0f));
                l[b] = fmaf(sum, 0x1p-40f, l[b]);
            }
        }
        // Weights, 8 keys an operand: half x holds keys 8 x .. 8 x + 7 of the lane's 16.
        // Their sum is added to l as one: many light keys beside a heavy one
        // are each below half a step of it.
        f16x8_t p[2][QB];
        float sum[QB];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float ib = pow2(byte_of(vi4, i));
#pragma unroll
            for (int b = 0; b < QB; ++b) {
                const float w = exp2_fast(s[i / 4][b][i % 4]);
                sum[b] = i == 0 ? w * ib : fmaf(w, ib, sum[b]);
                p[i / 8][b][i % 8] = static_cast<_Float16>(w);
            }
        }
#pragma unroll
        for (int b = 0; b < QB; ++b) l[b] = SPREAD ? fmaf(sum[b], spread ? 0.0f : 1.0f, l[b]) : l[b] + sum[b];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const f16x8_t vf = widen<DT_F16>(vw[h][2 * x], vw[h][2 * x + 1], 1.0f);
#pragma unroll
                for (int b = 0; b < QB; ++b) o[h][b] = Elem<DT_F16>::mfma(vf, p[x][b], o[h][b]);
            }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (more) load_v(vR);
        __builtin_amdgcn_sched_barrier(0);
    };
    for (; t + step < t_end; t += step) tile(std::true_type());
    if (t < t_end) tile(std::false_type());

    lane = lane_anew(), r = lane & 15, g = lane >> 4;
    const int thread = wave * 64 + lane;
    float m[QB];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
        l[b] = sum_over_g(l[b]);
        m[b] = thr[b] > -INFINITY ? static_cast<float>(KV_EXP_BIAS) - bm[b] : -INFINITY;
        // NaN stays in l even where no finite score has moved m.
        if (l[b] != l[b]) m[b] = l[b];
    }
    constexpr int PER = D / 4;  // lanes of a row, four elements each
    if (!joined) {
#pragma unroll
        for (int b = 0; b < QB; ++b) {
            const int row = b * 16 + r, i = token_of_row(a, row);
            if (i < it.n_tok)
#pragma unroll
                for (int h = 0; h < NH; ++h)
                    emit<DT, D, HERE>(a, it, token_in_lds()[b * 16 + r], i, kvh * a.gq + row - i * a.gq, h * 16 + g * 4, o[h][b], m[b], l[b]);
        }
        if (!HERE || it.part0 < 0) return;
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        unsigned long long last = __ballot(lane < it.n_tok && count_parts(a, it, toks, lane, kvh));
        for (; last != 0; last &= last - 1) {
            const AttendToken tk = toks[__builtin_ctzll(last)];
            for (int at = lane; at < a.gq * PER; at += 64) join_parts<DT, D, HERE>(a, tk, kvh * a.gq + at / PER, at % PER * 4);
        }
        return;
    }

    // Join the four waves: O scaled to the workgroup's maximum, added in LDS.
    float *lo = lds, *lm = lds + ATTEND_WAVES * wave_floats(D);
#pragma unroll
    for (int b = 0; b < QB; ++b) {
        if (g == 0) {
            lm[(wave * ATTEND_ROWS + b * 16 + r) * 2] = m[b];
            lm[(wave * ATTEND_ROWS + b * 16 + r) * 2 + 1] = l[b];
        }
#pragma unroll
        for (int h = 0; h < NH; ++h)
            *reinterpret_cast<f32x4_t *>(lo + (wave * ATTEND_ROWS + b * 16 + r) * (D + 4) + h * 16 + g * 4) = o[h][b];
    }
    __syncthreads();
    const int n_rows = it.n_tok * a.gq;
    for (int at = thread; at < n_rows * PER; at += 256) {
        const int row = at / PER, d = at % PER * 4;
        float mw[ATTEND_WAVES], M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int w = 0; w < ATTEND_WAVES; ++w) {
            mw[w] = lm[(w * ATTEND_ROWS + row) * 2];
            M = fmaxf(M, mw[w]);
        }
        const float ref = M == -INFINITY ? 0.0f : M;
        f32x4_t sum{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < ATTEND_WAVES; ++w) {
            const float h = half_of(mw[w] - ref);
            L = fmaf(h * lm[(w * ATTEND_ROWS + row) * 2 + 1], h, L);
            sum += h * h * *reinterpret_cast<const f32x4_t *>(lo + (w * ATTEND_ROWS + row) * (D + 4) + d);
        }
        const int i = token_of_row(a, row);
        emit<DT, D, HERE>(a, it, toks[i].token, i, kvh * a.gq + row - i * a.gq, d, sum, M, L);
    }
    if (HERE && it.part0 >= 0) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        unsigned long long *last = reinterpret_cast<unsigned long long *>(lm);
        if (wave == 0) {
            const unsigned long long mine = __ballot(lane < it.n_tok && count_parts(a, it, toks, lane, kvh));
            if (lane == 0) *last = mine;
        }
        __syncthreads();
        unsigned long long todo = *last;
        for (; todo != 0; todo &= todo - 1) {
            const AttendToken tk = toks[__builtin_ctzll(todo)];
            for (int at = thread; at < a.gq * PER; at += 256)
                join_parts<DT, D, HERE>(a, tk, kvh * a.gq + at / PER, at % PER * 4);
        }
    }
    __syncthreads();  // the next item writes LDS again
}

// Whether the plan is for caches like this one: a graph that was captured with
// one cache may be replayed after a plan for others, whose pages it must not
// follow.
__device__ __forceinline__ bool plan_fits(const AttendArgs &a, const AttendHeader *h) {
    return h->page_size == 1 << a.page_shift && h->n_pages == a.n_pages;
}

// NaN for the plan's tokens, whose outputs are not computed.
template <int DT>
__device__ __forceinline__ void put_nan(const AttendArgs &a, int n_tokens, int dim) {
    const long rows = static_cast<long>(n_tokens) * a.heads, threads = static_cast<long>(gridDim.x) * 256;
    const long at = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;
    constexpr uint32_t nan = Elem<DT>::qnan * 0x10001u;
    for (long i = at; i < rows * dim / 8; i += threads)
        *reinterpret_cast<u32x4_t *>(a.out + i * 8) = u32x4_t{nan, nan, nan, nan};
    if (a.lse != nullptr)
        for (long i = at; i < rows; i += threads) a.lse[i] = __uint_as_float(Elem<DT_F32>::qnan);
}

template <int DT, int D, bool HERE>
__global__ __launch_bounds__(256, 2) void k_attend(AttendArgs a) {
    extern __shared__ float lds[];
    const AttendHeader *h = reinterpret_cast<const AttendHeader *>(a.meta);
    const AttendItem *items = reinterpret_cast<const AttendItem *>(a.meta + sizeof(AttendHeader));
    const AttendToken *toks = reinterpret_cast<const AttendToken *>(a.meta + h->token_off);
    const int32_t *pages = reinterpret_cast<const int32_t *>(a.meta + h->page_off);
    const uint32_t *nodes = reinterpret_cast<const uint32_t *>(a.meta + h->node_off);
    if (!plan_fits(a, h)) return put_nan<DT>(a, h->n_tokens, D);
    const int n = h->n_groups * a.kv_heads;
    const int wave = uniform(threadIdx.x >> 6);
    for (int w = blockIdx.x; w < n; w += gridDim.x) {
        const int i = w / a.kv_heads, kvh = w - i * a.kv_heads;
        const AttendItem it = items[i * ATTEND_WAVES + wave];
        if (it.n_tok * a.gq > 16)
            attend_item<DT, D, 2, HERE>(a, it, toks + it.tok0, pages + it.page0, nodes + it.tok0, kvh, wave, lds);
        else if (it.n_tok > 0)
            attend_item<DT, D, 1, HERE>(a, it, toks + it.tok0, pages + it.page0, nodes + it.tok0, kvh, wave, lds);
    }
}

// The second launch: D / 4 lanes join a row.
template <int DT, int D>
__global__ __launch_bounds__(256) void k_attend_join(AttendArgs a) {
    const AttendHeader *h = reinterpret_cast<const AttendHeader *>(a.meta);
    const AttendToken *toks = reinterpret_cast<const AttendToken *>(a.meta + h->token_off);
    constexpr int PER = D / 4, ROWS = 256 / PER;
    const long n = h->n_split > 0 && plan_fits(a, h) ? static_cast<long>(h->n_tokens) * a.heads : 0;
    for (long row = static_cast<long>(blockIdx.x) * ROWS + threadIdx.x / PER; row < n;
         row += static_cast<long>(gridDim.x) * ROWS) {
        const int s = static_cast<int>(row / a.heads), head = static_cast<int>(row - static_cast<long>(s) * a.heads);
        const AttendToken tk = toks[s];
        if (tk.n[0] + tk.n[1] > 0) join_parts<DT, D, false>(a, tk, head, threadIdx.x % PER * 4);
    }
}

// Grids are as large as the plan at launch asks for; a graph replayed after a
// new plan may find more, or partial results where there were none.
template <int DT, int D, bool HERE>
hipError_t run(const AttendArgs &a, int n_groups, int n_tokens, hipStream_t st) {
    constexpr size_t lds = lds_floats(D) * sizeof(float);
    // Once a device: the kernel's LDS.
    static std::atomic<uint64_t> allowed{0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if ((allowed.load(std::memory_order_relaxed) & bit) == 0) {
        e = hipFuncSetAttribute(reinterpret_cast<const void *>(k_attend<DT, D, HERE>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
        if (e != hipSuccess) return e;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    auto grid = [](long n) { return static_cast<unsigned>(n < 1 ? 1 : n > 65536 ? 65536 : n); };
    k_attend<DT, D, HERE><<<grid(static_cast<long>(n_groups) * a.kv_heads), 256, lds, st>>>(a);
    if constexpr (!HERE) {
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        const long rows = static_cast<long>(n_tokens) * a.heads, per = 256 / (D / 4);
        k_attend_join<DT, D><<<grid((rows + per - 1) / per), 256, 0, st>>>(a);
    }
    return hipGetLastError();
}

// Joining in the launch saves the second one (5 us; 8 partial results of one
// sequence: 10.0 us instead of 12.5), but each wave then waits for its stores
// and its count before it ends, which is paid where workgroups share a CU or
// follow one another on it (64 sequences with drafts, 448 workgroups: 59 us
// instead of 55; 64 decoding ones, 1200: 49 instead of 43).  So: up to one a
// CU.  And the last of a block joins one token after the other, a step of
// results at a time: 16 steps (a tree of 32 on 2001 tokens) 24.8 us instead of
// 16.8, 4 steps (two tokens of eight results) 11.5 instead of 14.4.  At 8 steps
// it goes by the sequences: one with four tokens 13.5 instead of 14.1, two 14.1
// instead of 13.4, four 14.6 instead of 13.4.
constexpr int JOIN_HERE_WGS = 256, JOIN_HERE_STEPS = 6;

template <int DT, int D>
hipError_t run(const AttendArgs &a, int n_groups, int n_tokens, int join_steps, hipStream_t st) {
    const bool here = static_cast<long>(n_groups) * a.kv_heads <= JOIN_HERE_WGS && join_steps <= JOIN_HERE_STEPS;
    return here ? run<DT, D, true>(a, n_groups, n_tokens, st) : run<DT, D, false>(a, n_groups, n_tokens, st);
}

}  // namespace

hipError_t launch_attend(const AttendArgs &args, int dtype, int dim, int n_groups, int n_tokens, int join_steps,
                         hipStream_t st) {
    AttendArgs a = args;
    if (dtype == DT_F16)
        return dim == 128 ? run<DT_F16, 128>(a, n_groups, n_tokens, join_steps, st)
                          : run<DT_F16, 64>(a, n_groups, n_tokens, join_steps, st);
    a.scale *= static_cast<float>(1u << KEXP_LESS);
    return dim == 128 ? run<DT_BF16, 128>(a, n_groups, n_tokens, join_steps, st)
                      : run<DT_BF16, 64>(a, n_groups, n_tokens, join_steps, st);
}

}  // namespace lora
