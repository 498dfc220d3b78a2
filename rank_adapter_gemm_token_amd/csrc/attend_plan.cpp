// attend_plan.cpp -- cutting one batch's attention into work items
// (attend_plan.hpp).
#include "attend_plan.hpp"

#include <algorithm>
#include <cstring>

#include "../../include/lora.h"

namespace lora {

namespace {

int ceil_div(int a, int b) { return (a + b - 1) / b; }

// All times in tenths of a microsecond, as measured on an MI355X.
//
// A tile of 64 keys on a SIMD that two waves share, in which case it is as
// fast as it gets: the arithmetic of one or two blocks of 16 query rows, or
// its 16 KB from memory where nobody else reads them (blocks of rows that read
// the same keys at the same time find them in the L2).
int tile_cost(int rows, int readers) { return std::max(rows <= 16 ? 9 : 13, 25 / readers); }

// The arithmetic alone, in units of its own.
int tile_weight(int rows) { return rows <= 16 ? 10 : 16; }

constexpr int CUS = 256, SIMDS = 4 * CUS;
// What a workgroup takes to begin and to end.
constexpr double ENDS = 80.0;
// What a tile takes a wave that waits for nothing but itself.
constexpr double TILE_ALONE = 15.0;

// How long workgroups of `x` work each (a tile's cost is what it takes two
// waves of a SIMD) run on a CU that two of them share, and on one of their own.
double beside(double x) { return x / 2 + ENDS; }
double alone(double x) { return x / 3 + ENDS; }

// Time of n equal workgroups of x work, two at once on a CU, and of `single`
// work in waves of their own, which run in what these leave free.
double launch_time(int64_t n, double x, double single) {
    const int64_t rest = n % (2 * CUS);
    double t = static_cast<double>(n / (2 * CUS)) * beside(x);
    if (rest > 0) {
        const double last = rest <= CUS ? alone(x) : beside(x);
        t += last;
        // Half the slots do 0.7 of what all of them do.
        single -= 1.4 * last * static_cast<double>(2 * CUS - rest) / (2 * CUS);
    }
    return t + std::max(0.0, single);
}

}  // namespace

AttendPlanner::AttendPlanner(int max_seqs, int max_groups, int max_tokens, int max_pages, int n_heads,
                             int n_kv_heads)
    : max_seqs_(max_seqs),
      max_groups_(max_groups),
      max_tokens_(max_tokens),
      max_pages_(max_pages),
      n_heads_(n_heads),
      n_kv_heads_(n_kv_heads) {
    const int gq = n_heads / n_kv_heads;
    // A block has at least one token, of one sequence or of one group.
    max_spans_ = 2 * max_tokens;
    // What splitting may add.
    const int extra = ceil_div(ATTEND_EXTRA, n_kv_heads) + 1;
    max_extra_ = extra;
    max_groups_wg_ = max_spans_ + extra;
    // Every span's tokens once, and a block's tokens for each further workgroup.
    max_part_rows_ = 2 * max_tokens + extra * attend_block_tokens(gq);
    items_.reserve(static_cast<size_t>(max_groups_wg_) * ATTEND_WAVES);
    whole_.reserve(static_cast<size_t>(max_groups_wg_));
    single_.reserve(static_cast<size_t>(max_spans_));
    tokens_.reserve(static_cast<size_t>(max_tokens));
    pages_.reserve(static_cast<size_t>(max_pages) + 1);
    spans_.reserve(static_cast<size_t>(max_spans_));
    seq_tok_.resize(static_cast<size_t>(max_seqs));
    seq_page_.resize(static_cast<size_t>(max_seqs));
    q_first_.resize(static_cast<size_t>(max_seqs));
    grp_tok_.resize(static_cast<size_t>(max_groups) + 2);
    grp_page_.resize(static_cast<size_t>(max_groups) + 1);
}

size_t AttendPlanner::max_bytes() const {
    return sizeof(AttendHeader) + static_cast<size_t>(max_groups_wg_) * ATTEND_WAVES * sizeof(AttendItem) +
           static_cast<size_t>(max_tokens_) * sizeof(AttendToken) + (static_cast<size_t>(max_pages_) + 4) * 4;
}

void AttendPlanner::clear() {
    items_.clear();
    whole_.clear();
    single_.clear();
    tokens_.clear();
    pages_.clear();
    spans_.clear();
    part_rows_ = n_split_ = 0;
}

int AttendPlanner::check(const AttendBatch &b, const AttendGeometry &geo) const {
    if (b.n_seqs < 0 || b.n_seqs > max_seqs_ || b.n_groups < 0 || b.n_groups > max_groups_) return LORA_EINVAL;
    if (geo.n_heads != n_heads_ || geo.n_kv_heads != n_kv_heads_ || geo.page_size < 1 || geo.n_pages < 1)
        return LORA_EINVAL;
    if (b.n_seqs > 0 && (b.q_len == nullptr || b.kv_len == nullptr || b.group == nullptr || b.page0 == nullptr))
        return LORA_EINVAL;
    if (b.n_groups > 0 && (b.prefix_len == nullptr || b.prefix_page0 == nullptr)) return LORA_EINVAL;
    // Bounds that ascend from 0 or above: no list is looked at past its last one.
    auto ascend = [](const int32_t *at, int n) {
        if (n > 0 && at[0] < 0) return false;
        for (int i = 0; i < n; ++i)
            if (at[i + 1] < at[i]) return false;
        return true;
    };
    if (!ascend(b.page0, b.n_seqs) || !ascend(b.prefix_page0, b.n_groups)) return LORA_EINVAL;
    int64_t tokens = 0, pages = 0;
    // A row of pages: `len` keys in pages[first .. last).
    auto row = [&](const int32_t *list, const int32_t *at, int i, int32_t len) {
        if (len < 0 || len > ATTEND_MAX_KEYS) return false;
        const int64_t need = (static_cast<int64_t>(len) + geo.page_size - 1) / geo.page_size;
        if (need > at[i + 1] - at[i]) return false;
        if (need > 0 && list == nullptr) return false;
        for (int64_t k = 0; k < need; ++k)
            if (list[at[i] + k] < 0 || list[at[i] + k] >= geo.n_pages) return false;
        pages += need;
        return true;
    };
    for (int s = 0; s < b.n_seqs; ++s) {
        if (b.q_len[s] < 0 || b.group[s] < -1 || b.group[s] >= b.n_groups) return LORA_EINVAL;
        if (!row(b.pages, b.page0, s, b.kv_len[s])) return LORA_EINVAL;
        tokens += b.q_len[s];
    }
    for (int i = 0; i < b.n_groups; ++i)
        if (!row(b.prefix_pages, b.prefix_page0, i, b.prefix_len[i])) return LORA_EINVAL;
    if (tokens > max_tokens_) return LORA_ETOKENS;
    if (pages > max_pages_) return LORA_EINVAL;
    return LORA_OK;
}

int AttendPlanner::plan(const AttendBatch &b, const AttendGeometry &geo) {
    clear();
    const int rc = check(b, geo);
    if (rc != LORA_OK) return rc;
    page_size_ = geo.page_size;
    n_pages_ = geo.n_pages;
    const int gq = n_heads_ / n_kv_heads_;
    const int block = attend_block_tokens(gq);

    // Pages: each span's own, none that its length does not reach.
    auto add_pages = [&](const int32_t *list, const int32_t *at, int i, int32_t len) {
        const int first = static_cast<int>(pages_.size());
        const int need = static_cast<int>((static_cast<int64_t>(len) + geo.page_size - 1) / geo.page_size);
        if (need > 0) pages_.insert(pages_.end(), list + at[i], list + at[i] + need);
        return first;
    };
    for (int i = 0; i < b.n_groups; ++i)
        grp_page_[i] = add_pages(b.prefix_pages, b.prefix_page0, i, b.prefix_len[i]);
    for (int s = 0; s < b.n_seqs; ++s) seq_page_[s] = add_pages(b.pages, b.page0, s, b.kv_len[s]);

    // Query tokens sorted by group (group -1 last), sequences in order.
    std::fill(grp_tok_.begin(), grp_tok_.end(), 0);
    int total = 0;
    for (int s = 0; s < b.n_seqs; ++s) {
        q_first_[s] = total;
        total += b.q_len[s];
        grp_tok_[(b.group[s] < 0 ? b.n_groups : b.group[s]) + 1] += b.q_len[s];
    }
    for (int i = 0; i <= b.n_groups; ++i) grp_tok_[i + 1] += grp_tok_[i];
    tokens_.resize(static_cast<size_t>(total));
    {
        // grp_tok_[i] walks through group i and ends at group i + 1's start.
        for (int s = 0; s < b.n_seqs; ++s) {
            int &at = grp_tok_[b.group[s] < 0 ? b.n_groups : b.group[s]];
            seq_tok_[s] = at;
            for (int j = 0; j < b.q_len[s]; ++j) {
                AttendToken t{};
                t.token = q_first_[s] + j;
                tokens_[static_cast<size_t>(at + j)] = t;
            }
            at += b.q_len[s];
        }
    }

    // Spans, and the tokens that none reaches (nothing to attend to).
    int64_t weight = 0;
    auto add_span = [&](int tok0, int n, int page0, int end, int limit0, int step, bool own, int readers) {
        const int tiles = ceil_div(end, ATTEND_TILE), c = tile_cost(n * gq, readers);
        spans_.push_back(Span{tok0, n, page0, end, limit0, step, own, 0, tiles, static_cast<int64_t>(tiles) * c});
        weight += static_cast<int64_t>(tiles) * tile_weight(n * gq);
    };
    for (int i = 0; i < b.n_groups; ++i) {
        const int first = i == 0 ? 0 : grp_tok_[i - 1], n = grp_tok_[i] - first;
        if (b.prefix_len[i] == 0) continue;
        for (int t = 0; t < n; t += block)
            add_span(first + t, std::min(block, n - t), grp_page_[i], b.prefix_len[i], b.prefix_len[i], 0, false,
                     ceil_div(n, block));
    }
    for (int s = 0; s < b.n_seqs; ++s) {
        const int before = b.kv_len[s] - b.q_len[s];  // query token j sees before + j + 1 of its own
        for (int t = 0; t < b.q_len[s]; t += block) {
            const int n = std::min(block, b.q_len[s] - t);
            const int end = before + t + n;
            const bool prefix = b.group[s] >= 0 && b.prefix_len[b.group[s]] > 0;
            // A block that sees nothing still has its rows to write.
            if (end > 0 || !prefix)
                add_span(seq_tok_[s] + t, n, seq_page_[s], std::max(0, end), before + t + 1, 1, true,
                         ceil_div(b.q_len[s], block));
        }
    }

    // A span of up to a wave's share of the whole goes to one wave: its loop is
    // as long as it can be for what it costs to begin and end.  Longer ones go
    // to whole workgroups, whose waves take alternating tiles and join in LDS.
    // The shares are of the arithmetic: beside a prefix that several blocks
    // read, waves that stream have the memory to themselves (by time, 64
    // sequences with drafts had most of theirs in workgroups: 60 us, not 52).
    const int64_t share = std::max<int64_t>(weight * n_kv_heads_ / ATTEND_SLOTS, tile_weight(1));
    int64_t longest = 0;
    double stream = 0.0, waits = 0.0;
    for (Span &s : spans_) {
        s.splits = static_cast<int64_t>(s.tiles) * tile_weight(s.n_tok * gq) > share ? 1 : 0;
        if (s.splits)
            longest = std::max(longest, s.cost);
        else
            stream += static_cast<double>(s.cost), waits += TILE_ALONE * s.tiles + ENDS;
    }
    const double single = n_kv_heads_ * std::max(stream / SIMDS, waits / ATTEND_SLOTS);
    // How much of these a workgroup gets: what makes the launch shortest.  (A
    // fixed share, two a wave, left 320 workgroups for 256 CUs where 480 fit:
    // 64 sequences with drafts took 52 us.)  The longest span is cut into 64
    // pieces at most, which is as far as the model has been compared with
    // times: a span of over 16384 keys alone on one or two key/value heads
    // could use more (131072 keys of one head: 24 us, 14 by the model).
    int64_t best = longest;
    double best_time = 0.0;
    for (int k = 1; longest > 0 && k <= 64; k += k < 8 ? 1 : k < 16 ? 2 : 8) {
        const int64_t x = (longest + k - 1) / k;
        int64_t n = 0, more = 0;
        double work = 0.0;
        bool whole_tiles = true;  // no span in pieces of less than a tile a wave
        for (const Span &s : spans_)
            if (s.splits) {
                const int64_t pieces = (s.cost + x - 1) / x;
                n += pieces;
                more += pieces - 1;
                work += static_cast<double>(s.cost);
                whole_tiles = whole_tiles && (pieces == 1 || pieces * ATTEND_WAVES <= s.tiles + ATTEND_WAVES - 1);
            }
        if (k > 1 && (more >= max_extra_ || !whole_tiles)) break;
        const double t = launch_time(n * n_kv_heads_, work / static_cast<double>(n), single);
        if (k == 1 || t < 0.97 * best_time) {  // more pieces have to be worth it
            best = x;
            best_time = t;
        }
    }
    for (Span &s : spans_) {
        if (s.splits) s.splits = static_cast<int>((s.cost + best - 1) / best);
        for (int i = 0; i < s.n_tok; ++i) tokens_[static_cast<size_t>(s.tok0 + i)].n[s.own] = std::max(1, s.splits);
    }
    for (Span &s : spans_) {
        // Alone: no token of the block has a result of another item.
        bool alone = s.splits <= 1;
        for (int i = 0; alone && i < s.n_tok; ++i) alone = tokens_[static_cast<size_t>(s.tok0 + i)].n[!s.own] == 0;
        const int tiles = s.tiles, splits = std::max(1, s.splits);
        const int base = part_rows_;
        for (int k = 0; k < splits; ++k) {
            const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * k / splits);
            const int t1 = static_cast<int>(static_cast<int64_t>(tiles) * (k + 1) / splits);
            (s.splits > 0 ? whole_ : single_)
                .push_back(Piece{{s.tok0, s.n_tok, s.page0, t0 * ATTEND_TILE, std::min(s.end, t1 * ATTEND_TILE), s.limit0,
                                  (s.step ? ATTEND_STEP : 0) | (s.splits > 0 ? ATTEND_JOINED : 0),
                                  alone ? -1 : base + k * s.n_tok},
                                 s.cost / splits});
        }
        for (int i = 0; i < s.n_tok; ++i) {
            AttendToken &t = tokens_[static_cast<size_t>(s.tok0 + i)];
            if (alone) {
                t.pad = 1;
            } else {
                t.part[s.own] = base + i;
                t.stride[s.own] = s.n_tok;
            }
        }
        if (!alone) part_rows_ += splits * s.n_tok;
    }
    for (AttendToken &t : tokens_) {
        if (t.pad) t.n[0] = t.n[1] = 0;
        t.pad = 0;
        n_split_ += t.n[0] + t.n[1] > 0;
    }
    // The dearest first, so that what is left at the end is short and the four
    // waves of a workgroup end together.
    auto dearer = [](const Piece &a, const Piece &b) {
        if (a.cost != b.cost) return a.cost > b.cost;
        // The blocks of rows that read the same keys side by side: they share
        // them in the L2.
        const AttendItem &x = a.it, &y = b.it;
        if (x.page0 != y.page0) return x.page0 < y.page0;
        return x.begin != y.begin ? x.begin < y.begin : x.tok0 < y.tok0;
    };
    std::sort(whole_.begin(), whole_.end(), dearer);
    std::sort(single_.begin(), single_.end(), dearer);
    // Both kinds side by side over the whole launch: the first is bound by
    // arithmetic where a prefix has many rows, the second by memory.  The
    // blocks of rows that read the same keys stay together.
    const size_t nw = whole_.size(), ns = (single_.size() + ATTEND_WAVES - 1) / ATTEND_WAVES;
    for (size_t w = 0, s = 0; w < nw || s < ns;) {
        if (s == ns || (w < nw && w * ns <= s * nw)) {
            do {
                items_.insert(items_.end(), ATTEND_WAVES, whole_[w++].it);
            } while (w < nw && whole_[w].it.page0 == whole_[w - 1].it.page0 &&
                     whole_[w].it.begin == whole_[w - 1].it.begin);
        } else {
            for (size_t i = s * ATTEND_WAVES; i < (s + 1) * ATTEND_WAVES; ++i)
                items_.push_back(i < single_.size() ? single_[i].it : AttendItem{});
            ++s;
        }
    }
    return LORA_OK;
}

size_t AttendPlanner::write(void *to) const {
    AttendHeader h{};
    h.n_groups = groups();
    h.n_tokens = static_cast<int32_t>(tokens_.size());
    h.n_split = n_split_;
    h.page_size = page_size_;
    h.n_pages = n_pages_;
    const size_t items = items_.size() * sizeof(AttendItem), toks = tokens_.size() * sizeof(AttendToken);
    h.token_off = static_cast<int32_t>(sizeof h + items);
    h.page_off = static_cast<int32_t>(sizeof h + items + toks);
    char *p = static_cast<char *>(to);
    std::memcpy(p, &h, sizeof h);
    if (items) std::memcpy(p + sizeof h, items_.data(), items);
    if (toks) std::memcpy(p + h.token_off, tokens_.data(), toks);
    if (!pages_.empty()) std::memcpy(p + h.page_off, pages_.data(), pages_.size() * 4);
    return static_cast<size_t>(h.page_off) + pages_.size() * 4;
}

size_t AttendPlanner::write_none(void *to, int n_tokens) {
    AttendHeader h{};
    h.n_tokens = n_tokens;
    h.token_off = h.page_off = static_cast<int32_t>(sizeof h);
    std::memcpy(to, &h, sizeof h);
    return sizeof h;
}

}  // namespace lora
