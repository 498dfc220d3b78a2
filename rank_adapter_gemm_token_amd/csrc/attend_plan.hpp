// attend_plan.hpp -- how one batch's attention is cut into work items: pure
// host C++, no device call.
//
// A batch has sequences with a few new (query) tokens each.  A sequence's
// query tokens attend to the prefix of its group, if it has one, and to the
// sequence's own tokens.  The query tokens are sorted by group, so that all
// of a group's tokens lie together and the prefix is read once for a block of
// them, and a sequence's tokens stay neighbours.  Each (block of query
// tokens, run of keys) is a span; spans are split along the keys so that the
// items fill the device about evenly.
//
// A sequence's new tokens may form a tree (or several), parents first.  With
// its nodes numbered depth first, node i is j or above it where pre_i <= pre_j
// < pre_i + size_i (size: of the nodes below it, itself among them), so that
// two numbers a node say who sees whom, however many nodes there are.
#pragma once

#include <cstddef>
#include <cstdint>
#include <vector>

#ifdef __HIP__
#define ATTEND_DEVICE __host__ __device__
#else
#define ATTEND_DEVICE
#endif

namespace lora {

// One wave's work: the query tokens sorted at tok0 .. tok0 + n_tok - 1 (none:
// the wave idles) over the keys begin .. end - 1 of the span whose pages start
// at page0, or over every fourth tile of them where the workgroup's four waves
// are joined.  Query token tok0 + i sees keys below min(end, limit0 + i * step).
struct AttendItem {
    int32_t tok0, n_tok;
    int32_t page0;
    int32_t begin, end;
    int32_t limit0;
    int32_t flags;  // ATTEND_STEP, ATTEND_JOINED, ATTEND_TREE; the rest times 8: the block's first token in its sequence
    int32_t part0;  // partial results of token i go to row part0 + i; -1: no other item has this token
};
static_assert(sizeof(AttendItem) == 32, "read by the kernels as two 16-byte words");
enum : int32_t {
    ATTEND_STEP = 1,
    ATTEND_JOINED = 2,  // the four waves share this item
    ATTEND_TREE = 4,    // of the new tokens only those above the query token are seen
    ATTEND_FIRST_SHIFT = 3
};

// One sorted query token: its row in q and out, and where its partial results
// are: rows part[k] + j * stride[k], j < n[k] (k = 0 the prefix, 1 its own).
struct AttendToken {
    int32_t token;
    int32_t part[2], stride[2], n[2];
    int32_t pad;
};
static_assert(sizeof(AttendToken) == 32, "read by the kernels as two 16-byte words");

// What the kernels read first.  Offsets in bytes from the header; a workgroup
// (for one key/value head) has four items, one for each wave.
struct AttendHeader {
    int32_t n_groups, n_tokens, n_split;  // n_split: tokens with partial results
    int32_t token_off, page_off;
    int32_t page_size, n_pages;         // of the caches it is for
    int32_t node_off;                   // of sorted token 0's node; 0: no trees
    int32_t pad[8];
};
static_assert(sizeof(AttendHeader) == 64, "items follow at byte 64");

constexpr int ATTEND_TILE = 64;       // keys a wave takes at a time
constexpr int ATTEND_WAVES = 4;       // waves of a workgroup
constexpr int ATTEND_MAX_GQ = 32;     // query heads per key/value head
constexpr int ATTEND_MAX_KEYS = 1 << 30;  // keys of one sequence or prefix (tiles times 64 stay whole 32-bit numbers)
constexpr int ATTEND_ROWS = 32;       // query rows (tokens x heads of a key head) of an item
constexpr int ATTEND_SLOTS = 2048;    // waves that run at once: two workgroups on each of 256 CUs
constexpr int ATTEND_NODE_PAD = 64;   // words before and after the nodes: the tile that holds one may begin, and end, so far away
constexpr int ATTEND_JOIN_STEP = 4;   // results of a token that are read together
constexpr int ATTEND_EXTRA = 1024;    // workgroups that splitting may add, over all key/value heads

// A token of a tree as the kernels read it, and whether i is j or above it.
inline uint32_t attend_node(int pre, int size) {
    return static_cast<uint32_t>(pre) | static_cast<uint32_t>(size - 1) << 16;
}
ATTEND_DEVICE inline bool attend_above(uint32_t i, uint32_t j) { return (j & 0xFFFFu) - (i & 0xFFFFu) <= i >> 16; }

// Query tokens of one item, for gq query heads per key/value head.
inline int attend_block_tokens(int gq) { return gq >= ATTEND_ROWS ? 1 : ATTEND_ROWS / gq; }

// The batch as the caller gives it (host arrays).
struct AttendBatch {
    int n_seqs, n_groups;
    const int32_t *q_len, *kv_len, *group;
    const int32_t *pages, *page0;
    const int32_t *prefix_len, *prefix_pages, *prefix_page0;
    // Of each new token the new token of its sequence that it follows, or -1;
    // null: each follows the one before, unless the list has to be there.
    const int32_t *parent;
    bool tree = false;  // it has to be, where there are new tokens
};

struct AttendGeometry {
    int n_heads, n_kv_heads;
    int page_size, n_pages;
};

class AttendPlanner {
public:
    // Everything is allocated here: plan() does not.
    AttendPlanner(int max_seqs, int max_groups, int max_tokens, int max_pages, int n_heads, int n_kv_heads);

    // Rows of partial results that a batch may need at most.
    int max_part_rows() const { return max_part_rows_; }
    // Bytes of the header, items, tokens, pages and nodes at most.
    size_t max_bytes() const;

    // Cut the batch.  0, or the negative status of the first thing wrong with
    // it (LORA_EINVAL, LORA_ETOKENS); the plan is then empty.
    int plan(const AttendBatch &b, const AttendGeometry &geo);

    // The bytes the device reads, max_bytes() at most; returns how many.
    size_t write(void *to) const;

    // As write(): a plan of no work, for no cache (of 0 pages), of n_tokens
    // tokens, for which the device writes NaN.
    static size_t write_none(void *to, int n_tokens);

    const std::vector<AttendItem> &items() const { return items_; }  // four a workgroup
    int groups() const { return static_cast<int>(items_.size()) / ATTEND_WAVES; }
    const std::vector<AttendToken> &tokens() const { return tokens_; }
    const std::vector<int32_t> &pages() const { return pages_; }
    const std::vector<uint32_t> &nodes() const { return nodes_; }  // of the sorted tokens; empty: no trees
    int part_rows() const { return part_rows_; }
    // What the last item of a block has to join at most, in steps of up to four
    // results of one token.
    int join_steps() const { return join_steps_; }
    int n_split() const { return n_split_; }

private:
    struct Span {
        int tok0, n_tok, page0, end, limit0, flags;
        bool own;
        int splits;   // workgroups; 0: one wave
        int tiles;
        int64_t cost;
    };
    struct Piece {
        AttendItem it;
        int64_t cost;
    };
    int check(const AttendBatch &b, const AttendGeometry &geo) const;
    void clear();

    int max_seqs_, max_groups_, max_tokens_, max_pages_, n_heads_, n_kv_heads_;
    int max_spans_, max_extra_, max_groups_wg_, max_part_rows_;
    std::vector<AttendItem> items_;
    std::vector<Piece> whole_, single_;  // of a workgroup, of a wave
    std::vector<AttendToken> tokens_;
    std::vector<int32_t> pages_;
    std::vector<uint32_t> nodes_;
    std::vector<int32_t> size_, next_;  // of one sequence's nodes
    std::vector<char> tree_;            // of each sequence: not a mere chain
    std::vector<Span> spans_;
    std::vector<int32_t> seq_tok_, grp_tok_, seq_page_, grp_page_, q_first_;
    int part_rows_ = 0, join_steps_ = 0, n_split_ = 0, page_size_ = 0, n_pages_ = 0;
};

}  // namespace lora
