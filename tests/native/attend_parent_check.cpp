// Checks that the attention planner (attend_plan.cpp) asks for a tree's list of
// parents only after the batch's counts: a batch of more sequences than the plan
// has room for is refused before any of its lists is read (run with the address
// sanitizer, each list shorter than the count), and a missing list where there
// are new tokens.
#include <cstdio>
#include <cstdlib>
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

int main() {
    const AttendGeometry geo{4, 2, 16, 8};
    AttendPlanner p(2, 0, 8, 8, 4, 2);
    const std::vector<int32_t> two{2, 2}, none{0, 0}, len{20, 2}, group{-1, -1}, pages{0, 1, 2}, page0{0, 2, 3};
    AttendBatch b{2, 0, two.data(), len.data(), group.data(), pages.data(), page0.data(), nullptr, nullptr, nullptr, nullptr, true};
    CHECK(p.plan(b, geo) == LORA_EINVAL && p.items().empty() && p.tokens().empty());
    for (int n : {3, 1 << 20, -1}) {
        b.n_seqs = n;
        CHECK(p.plan(b, geo) == LORA_EINVAL);
    }
    b.n_seqs = 2;
    b.tree = false;  // a chain
    CHECK(p.plan(b, geo) == LORA_OK && p.tokens().size() == 4);
    b.tree = true;
    b.q_len = none.data();  // no new tokens, no list
    CHECK(p.plan(b, geo) == LORA_OK && p.tokens().empty());
    const std::vector<int32_t> parent{-1, -1, -1, 0};
    b.q_len = two.data();
    b.parent = parent.data();
    CHECK(p.plan(b, geo) == LORA_OK && p.tokens().size() == 4 && p.nodes().size() == 4);
    std::printf("ok\n");
    return 0;
}
