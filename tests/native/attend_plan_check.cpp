// Checks of the attention planner (attend_plan.cpp), pure host code: over
// random batches every (query token, key it sees) is in exactly one item,
// every partial row is written once and read once, and everything stays
// within the sizes the planner promised at creation; bad batches are refused.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <random>
#include <set>
#include <vector>

#include "../../include/lora.h"
#include "../../rank_adapter_gemm_token_amd/csrc/attend_plan.hpp"

using namespace lora;

#define CHECK(x)                                                      \
    do {                                                              \
        if (!(x)) {                                                   \
            std::printf("line %d: %s\n", __LINE__, #x);               \
            std::exit(1);                                             \
        }                                                             \
    } while (0)

struct Lists {
    std::vector<int32_t> q, kv, grp, pages, page0, plen, ppages, ppage0;
    AttendBatch batch() const {
        return {static_cast<int>(q.size()), static_cast<int>(plen.size()), q.data(), kv.data(), grp.data(),
                pages.data(), page0.data(), plen.data(), ppages.data(), ppage0.data()};
    }
};

static void check_plan(const AttendPlanner &p, const Lists &b, int heads, int kv_heads, int page) {
    const int gq = heads / kv_heads;
    std::vector<int> seq_of, pos;
    for (size_t s = 0; s < b.q.size(); ++s)
        for (int j = 0; j < b.q[s]; ++j) seq_of.push_back(static_cast<int>(s)), pos.push_back(j);
    CHECK(p.tokens().size() == seq_of.size());
    std::set<int> once;
    for (const AttendToken &t : p.tokens()) CHECK(once.insert(t.token).second && t.token < (int)seq_of.size());
    CHECK(p.part_rows() <= p.max_part_rows());
    // Per sorted token: what the items cover, and where their results go.
    std::vector<std::vector<char>> pre(seq_of.size()), own(seq_of.size());
    std::vector<int> direct(seq_of.size(), 0);
    std::map<int, int> part_owner;
    CHECK(p.items().size() % ATTEND_WAVES == 0);
    for (size_t n = 0; n < p.items().size(); ++n) {
        const AttendItem &it = p.items()[n];
        const AttendItem &first = p.items()[n - n % ATTEND_WAVES];
        CHECK((it.flags & ATTEND_JOINED) == (first.flags & ATTEND_JOINED) || it.n_tok == 0);
        if (it.flags & ATTEND_JOINED) {
            CHECK(std::memcmp(&it, &first, sizeof it) == 0);
            if (n % ATTEND_WAVES != 0) continue;  // the four waves share one item
        }
        if (it.n_tok == 0) continue;  // nothing for this wave
        CHECK(it.n_tok >= 1 && it.n_tok <= attend_block_tokens(gq) && it.n_tok * gq <= ATTEND_ROWS);
        CHECK(it.begin % ATTEND_TILE == 0 && it.begin <= it.end);
        for (int i = 0; i < it.n_tok; ++i) {
            const int sorted = it.tok0 + i;
            const AttendToken &t = p.tokens()[static_cast<size_t>(sorted)];
            const int s = seq_of[static_cast<size_t>(t.token)];
            const int g = b.grp[static_cast<size_t>(s)];
            if (it.part0 < 0)
                ++direct[static_cast<size_t>(sorted)];
            else
                CHECK(part_owner.insert({it.part0 + i, sorted}).second && it.part0 + i < p.part_rows());
            const bool is_prefix = (it.flags & ATTEND_STEP) == 0;
            const int len = is_prefix ? b.plen[static_cast<size_t>(g)] : b.kv[static_cast<size_t>(s)];
            const int32_t *list = is_prefix ? &b.ppages[static_cast<size_t>(b.ppage0[static_cast<size_t>(g)])]
                                            : b.pages.data() + b.page0[static_cast<size_t>(s)];
            const int seen = is_prefix ? len : len - b.q[static_cast<size_t>(s)] + pos[static_cast<size_t>(t.token)] + 1;
            auto &mine = (is_prefix ? pre : own)[static_cast<size_t>(sorted)];
            mine.resize(static_cast<size_t>(len), 0);
            const int lim = std::min(it.end, it.limit0 + (is_prefix ? 0 : i));
            CHECK(it.end <= len);
            for (int k = it.begin; k < it.end; ++k) {
                CHECK(p.pages()[static_cast<size_t>(it.page0 + k / page)] == list[k / page]);
                CHECK((k < lim) == (k < seen));
                if (k < lim) ++mine[static_cast<size_t>(k)];
            }
        }
    }
    size_t parts = 0;
    int split = 0;
    for (size_t i = 0; i < p.tokens().size(); ++i) {
        const AttendToken &t = p.tokens()[i];
        const int s = seq_of[static_cast<size_t>(t.token)], g = b.grp[static_cast<size_t>(s)];
        const int seen = std::max(0, b.kv[static_cast<size_t>(s)] - b.q[static_cast<size_t>(s)] + pos[static_cast<size_t>(t.token)] + 1);
        const int plen = g < 0 ? 0 : b.plen[static_cast<size_t>(g)];
        pre[i].resize(static_cast<size_t>(plen), 0);
        for (int k = 0; k < plen; ++k) CHECK(pre[i][static_cast<size_t>(k)] == 1);
        own[i].resize(std::max(own[i].size(), static_cast<size_t>(seen)), 0);
        for (size_t k = 0; k < own[i].size(); ++k) CHECK(own[i][k] == (static_cast<int>(k) < seen));
        split += t.n[0] + t.n[1] > 0;
        CHECK((t.n[0] + t.n[1] > 0) != (direct[i] == 1) && direct[i] <= 1);
        for (int k = 0; k < 2; ++k)
            for (int j = 0; j < t.n[k]; ++j, ++parts) {
                auto f = part_owner.find(t.part[k] + j * t.stride[k]);
                CHECK(f != part_owner.end() && f->second == static_cast<int>(i));
            }
    }
    CHECK(parts == part_owner.size() && split == p.n_split());
    std::vector<char> buf(p.max_bytes());
    const size_t n = p.write(buf.data());
    CHECK(n <= p.max_bytes());
    AttendHeader h;
    std::memcpy(&h, buf.data(), sizeof h);
    CHECK(h.n_groups == p.groups() && h.n_tokens == (int)p.tokens().size() && h.n_split == split);
    CHECK(h.page_size == page);
    CHECK(std::memcmp(buf.data() + sizeof h, p.items().data(), p.items().size() * sizeof(AttendItem)) == 0);
}

int main() {
    std::mt19937 rng(7);
    auto draw = [&](int lo, int hi) { return lo + static_cast<int>(rng() % static_cast<unsigned>(hi - lo + 1)); };
    for (int round = 0; round < 400; ++round) {
        const int kv_heads = 1 << draw(0, 5), gq = draw(1, 32), heads = kv_heads * gq;
        const int page = 16 << draw(0, 3);
        const int B = draw(0, 20), G = draw(0, 4), n_pages = draw(1, 500);
        Lists b;
        int tokens = 0, pages = 0;
        b.page0.push_back(draw(0, 1));
        b.pages.assign(static_cast<size_t>(b.page0[0]), -5);  // never looked at
        for (int s = 0; s < B; ++s) {
            b.q.push_back(draw(0, round % 3 ? 4 : 70));
            b.kv.push_back(draw(0, round % 2 ? 300 : 5000));
            b.grp.push_back(draw(-1, G - 1));
            const int need = (b.kv.back() + page - 1) / page, more = draw(0, 2);
            for (int k = 0; k < need; ++k) b.pages.push_back(draw(0, n_pages - 1));
            for (int k = 0; k < more; ++k) b.pages.push_back(-9);  // past the length: not looked at
            b.page0.push_back(static_cast<int32_t>(b.pages.size()));
            tokens += b.q.back();
            pages += need;
        }
        b.ppage0.push_back(0);
        for (int g = 0; g < G; ++g) {
            b.plen.push_back(draw(0, 4) ? draw(1, 9000) : 0);
            const int need = (b.plen.back() + page - 1) / page;
            for (int k = 0; k < need; ++k) b.ppages.push_back(draw(0, n_pages - 1));
            b.ppage0.push_back(static_cast<int32_t>(b.ppages.size()));
            pages += need;
        }
        AttendPlanner p(std::max(1, B), G, std::max(1, tokens), pages, heads, kv_heads);
        const size_t cap = p.items().capacity();
        CHECK(p.plan(b.batch(), {heads, kv_heads, page, n_pages}) == LORA_OK);
        CHECK(p.items().capacity() == cap);  // nothing allocated after creation
        check_plan(p, b, heads, kv_heads, page);
        if (round % 10 == 0) {  // again, after another batch
            Lists none;
            none.page0 = none.ppage0 = {0};
            CHECK(p.plan(none.batch(), {heads, kv_heads, page, n_pages}) == LORA_OK && p.items().empty());
            CHECK(p.plan(b.batch(), {heads, kv_heads, page, n_pages}) == LORA_OK);
            check_plan(p, b, heads, kv_heads, page);
        }
    }
    // Refusals: each leaves the plan empty.
    Lists ok;
    ok.q = {1, 2};
    ok.kv = {20, 40};
    ok.grp = {0, -1};
    ok.pages = {3, 1, 0, 2, 4};
    ok.page0 = {0, 2, 5};
    ok.plen = {33};
    ok.ppages = {5, 6, 7};
    ok.ppage0 = {0, 3};
    AttendPlanner p(2, 1, 3, 8, 4, 2);
    const AttendGeometry geo{4, 2, 16, 8};
    auto refused = [&](const Lists &b, int rc) {
        CHECK(p.plan(ok.batch(), geo) == LORA_OK && !p.items().empty());
        CHECK(p.plan(b.batch(), geo) == rc);
        CHECK(p.items().empty() && p.tokens().empty());
    };
    Lists b;
    b = ok, b.pages[1] = 8, refused(b, LORA_EINVAL);        // a page past the cache
    b = ok, b.pages[4] = -1, refused(b, LORA_EINVAL);
    b = ok, b.ppages[2] = 8, refused(b, LORA_EINVAL);
    b = ok, b.kv[0] = 33, refused(b, LORA_EINVAL);          // three pages needed, two given
    b = ok, b.kv[0] = -1, refused(b, LORA_EINVAL);
    b = ok, b.kv[0] = 0x7FFFFFFF, refused(b, LORA_EINVAL);
    b = ok, b.plen[0] = 49, refused(b, LORA_EINVAL);
    b = ok, b.q[0] = -1, refused(b, LORA_EINVAL);
    b = ok, b.q[0] = 2, refused(b, LORA_ETOKENS);           // four new tokens, room for three
    b = ok, b.q[0] = 0x7FFFFFFF, b.q[1] = 0x7FFFFFFF, refused(b, LORA_ETOKENS);
    b = ok, b.grp[1] = 1, refused(b, LORA_EINVAL);
    b = ok, b.grp[1] = -2, refused(b, LORA_EINVAL);
    b = ok, b.page0[1] = 6, refused(b, LORA_EINVAL);        // a row that ends before it begins
    b = ok, b.page0[0] = -1, refused(b, LORA_EINVAL);
    b = ok, b.q.push_back(0), b.kv.push_back(0), b.grp.push_back(-1), b.page0.push_back(5), refused(b, LORA_EINVAL);
    AttendBatch nul = ok.batch();
    nul.kv_len = nullptr;
    CHECK(p.plan(nul, geo) == LORA_EINVAL);
    nul = ok.batch(), nul.pages = nullptr;
    CHECK(p.plan(nul, geo) == LORA_EINVAL);
    nul = ok.batch(), nul.prefix_page0 = nullptr;
    CHECK(p.plan(nul, geo) == LORA_EINVAL);
    std::printf("ok\n");
    return 0;
}
