// kv_internal.hpp -- records and launchers shared by kv_api.cpp and the .hip
// files of the cache, the attention over it and the draft verification.  Not
// part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace lora {

// The quantised cache.  A row is one token of one key/value head: D elements
// of e4m3, and an exponent byte b that scales them by 2^(b - 127).  Row
// (page, head, offset) has the number R = (page * heads + head) * page_size +
// offset.
// Blocks of 16 rows (R - R % 16 = B) are stored at byte B * D in the order in
// which the lanes of an MFMA operand load them, 16 bytes a lane, so that
// neighbouring lanes read neighbouring bytes:
//   keys    element d of row B + t at key_byte(t, d) of the block: for every
//           four rows and 64 elements, 16 elements of the four rows in turn
//   values  by element: element d of row B + t at d * 16 + t, so that 16 keys'
//           values of one element are one load
//   kexp, vinv  exponent bytes, one a row: a key's b, a value's 254 - b, of
//           which the attention makes 2^-s by a shift
// Elements are finite, except that a row whose key or value has a value that
// is not finite is POISONED: its key elements are NaN (its scores are then
// NaN, wherever they are looked at, and nothing else is), its value elements
// 0 and its vinv KV_POISON.
constexpr int KV_BLOCK = 16;        // rows of a block of values
constexpr int KV_POISON = 0;        // as a float's exponent bits: 0, which no weight of 0 makes NaN
constexpr int KV_EXP_BIAS = 127;
constexpr int KV_MIN_EXP = -64;     // least exponent kept: smaller values go to 0

template <int D>
__host__ __device__ constexpr int key_byte(int t, int d) {
    return (t / 4) * 4 * D + d / 64 * 256 + d % 64 / 16 * 64 + t % 4 * 16 + d % 16;
}

struct KvCache {
    uint8_t *k, *v, *kexp, *vinv;
    unsigned long long *err;
    int n_pages, page_shift, heads, dim;  // page_size = 1 << page_shift
    int dtype;
};

hipError_t launch_kv_write(const KvCache &c, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                           const int32_t *slots, int n_tokens, hipStream_t st);
hipError_t launch_kv_read(const KvCache &c, const int32_t *slots, int n_tokens, void *k, void *v, hipStream_t st);

struct AttendArgs {
    const char *meta;      // AttendHeader, items, tokens, pages
    const uint8_t *k, *v, *kexp, *vinv;
    const uint16_t *q;
    int64_t q_stride;      // elements from one token's heads to the next's
    uint16_t *out;         // [tokens][heads][dim]
    float *lse;            // [tokens][heads] or null
    float *part_o;         // [part rows][heads][dim]
    float *part_ml;        // [part rows][heads][2]
    unsigned *count;       // [tokens][kv_heads] partial results so far; 0 between calls
    int heads, kv_heads, gq, page_shift, n_pages;
    int gq_inv;            // 65536 / gq, rounded up
    float scale;           // softmax scale times log2(e)
};

hipError_t launch_attend(const AttendArgs &a, int dtype, int dim, int n_groups, int n_tokens, hipStream_t st);

struct VerifyArgs {
    const void *p, *q;
    const int32_t *draft, *row0;
    const float *u;
    int32_t *tokens, *accepted;
    double *sums;          // [seqs][VERIFY_PARTS]
    unsigned *count;       // [seqs], 0 between calls
    int n_seqs, n_rows, vocab;
    int parts, group;      // parts of a row, parts of a workgroup
};
constexpr int VERIFY_PART = 32768;    // elements of a part of a row
constexpr int VERIFY_PARTS = 64;      // parts of a row at most
constexpr int VERIFY_MAX_DRAFTS = 63; // drafted tokens of a sequence

hipError_t launch_verify(const VerifyArgs &a, int dtype, hipStream_t st);

}  // namespace lora
