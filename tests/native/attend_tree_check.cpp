// Checks of the attention planner's trees (attend_plan.cpp), pure host code:
// over random batches the nodes say exactly who is above whom, items of trees
// and of chains are marked as such and name the tokens they begin with, the
// bytes for the device hold the nodes with room for a tile on both sides, and
// lists of parents that are no trees are refused.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "../../include/lora.h"
#include "../../rank_adapter_gemm_token_amd/csrc/attend_plan.hpp"

using namespace lora;

#define CHECK(x)                                        \
    do {                                                \
        if (!(x)) {                                     \
            std::printf("line %d: %s\n", __LINE__, #x); \
            std::exit(1);                               \
        }                                               \
    } while (0)

static bool above(const std::vector<int32_t> &parent, int i, int j) {
    for (; j >= 0; j = parent[static_cast<size_t>(j)])
        if (i == j) return true;
    return false;
}

int main() {
    std::mt19937 rng(11);
    auto draw = [&](int lo, int hi) { return lo + static_cast<int>(rng() % static_cast<unsigned>(hi - lo + 1)); };
    for (int round = 0; round < 300; ++round) {
        const int kv_heads = 1 << draw(0, 3), gq = draw(1, 9), heads = kv_heads * gq, page = 16;
        const int B = draw(1, 9), G = draw(0, 2);
        std::vector<int32_t> q, kv, grp, pages, page0{0}, plen, ppages, ppage0{0}, parent;
        std::vector<std::vector<int32_t>> trees;
        bool any = false;
        for (int s = 0; s < B; ++s) {
            const int n = draw(0, round % 5 ? 12 : 300), kind = draw(0, 4);
            std::vector<int32_t> t;
            for (int j = 0; j < n; ++j)
                t.push_back(kind == 0 ? j - 1 : kind == 1 ? (j > 0 ? 0 : -1) : kind == 2 ? draw(-1, j - 1) : j ? draw(j > 4 ? j - 4 : 0, j - 1) : -1);
            for (int j = 0; j < n; ++j) any = any || t[static_cast<size_t>(j)] != j - 1;
            parent.insert(parent.end(), t.begin(), t.end());
            trees.push_back(t);
            q.push_back(n);
            kv.push_back(draw(0, 1) ? n + draw(0, 200) : draw(0, n));
            grp.push_back(draw(-1, G - 1));
            for (int k = 0; k < (kv.back() + page - 1) / page; ++k) pages.push_back(k % 7);
            page0.push_back(static_cast<int32_t>(pages.size()));
        }
        for (int g = 0; g < G; ++g) {
            plen.push_back(draw(0, 90));
            for (int k = 0; k < (plen.back() + page - 1) / page; ++k) ppages.push_back(k % 7);
            ppage0.push_back(static_cast<int32_t>(ppages.size()));
        }
        AttendPlanner p(B, G, static_cast<int>(parent.size()) + 1, static_cast<int>(pages.size() + ppages.size()), heads, kv_heads);
        parent.push_back(-7);  // past the batch's tokens: not looked at
        AttendBatch b{B, G, q.data(), kv.data(), grp.data(), pages.data(), page0.data(), plen.data(), ppages.data(), ppage0.data(), parent.data()};
        const AttendGeometry geo{heads, kv_heads, page, 7};
        const size_t cap = p.nodes().capacity();
        CHECK(p.plan(b, geo) == LORA_OK && p.nodes().capacity() == cap);
        CHECK(p.nodes().size() == (any ? p.tokens().size() : 0u));
        std::vector<int> seq_of, pos;
        for (int s = 0; s < B; ++s)
            for (int j = 0; j < q[static_cast<size_t>(s)]; ++j) seq_of.push_back(s), pos.push_back(j);
        for (size_t x = 0; any && x < p.tokens().size(); ++x)
            for (size_t y = 0; y < p.tokens().size(); ++y) {
                const size_t i = static_cast<size_t>(p.tokens()[x].token), j = static_cast<size_t>(p.tokens()[y].token);
                if (seq_of[i] != seq_of[j]) continue;
                CHECK(attend_above(p.nodes()[x], p.nodes()[y]) == above(trees[static_cast<size_t>(seq_of[i])], pos[i], pos[j]));
            }
        for (const AttendItem &it : p.items()) {
            if (it.n_tok == 0 || !(it.flags & ATTEND_STEP)) {
                CHECK(!(it.flags & ATTEND_TREE));
                continue;
            }
            const size_t first = static_cast<size_t>(p.tokens()[static_cast<size_t>(it.tok0)].token);
            const size_t s = static_cast<size_t>(seq_of[first]);
            CHECK(it.flags >> ATTEND_FIRST_SHIFT == pos[first]);
            CHECK(it.limit0 - 1 - pos[first] == kv[s] - q[s]);
            bool chain = true;
            for (int j = 0; j < q[s]; ++j) chain = chain && trees[s][static_cast<size_t>(j)] == j - 1;
            CHECK(((it.flags & ATTEND_TREE) != 0) == !chain);
        }
        std::vector<char> buf(p.max_bytes());
        const size_t n = p.write(buf.data());
        AttendHeader h;
        std::memcpy(&h, buf.data(), sizeof h);
        CHECK(n <= p.max_bytes() && (h.node_off != 0) == any && h.node_off % 4 == 0);
        if (any) {
            CHECK(h.node_off >= h.page_off + static_cast<int>(p.pages().size()) * 4 + ATTEND_NODE_PAD * 4);
            CHECK(static_cast<size_t>(h.node_off) + (p.nodes().size() + ATTEND_NODE_PAD) * 4 == n);
            CHECK(std::memcmp(buf.data() + h.node_off, p.nodes().data(), p.nodes().size() * 4) == 0);
        }
        b.parent = nullptr;  // a chain after a tree
        CHECK(p.plan(b, geo) == LORA_OK && p.nodes().empty());
        for (const AttendItem &it : p.items()) CHECK(!(it.flags & ATTEND_TREE));
        if (!p.tokens().empty()) {
            b.parent = parent.data();
            const size_t at = static_cast<size_t>(draw(0, static_cast<int>(p.tokens().size()) - 1));
            for (int32_t bad : {pos[at], pos[at] + 1, -2, 0x7FFFFFFF, -0x7FFFFFFF - 1}) {
                const int32_t was = parent[at];
                parent[at] = bad;
                CHECK(p.plan(b, geo) == LORA_EINVAL && p.items().empty() && p.nodes().empty());
                parent[at] = was;
            }
        }
    }
    std::printf("ok\n");
    return 0;
}
