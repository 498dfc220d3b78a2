// Checks that the attention planner (attend_plan.cpp) looks at a page list
// only between its first and its last bound: the bounds are known to ascend
// before any entry is read, so lists that do not are refused unread.  Run with
// the address sanitizer, each list as long as its last bound says.
#include <cstdio>
#include <cstdlib>
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

int main() {
    const AttendGeometry geo{4, 2, 16, 8};
    AttendPlanner p(4, 4, 8, 64, 4, 2);
    const std::vector<int32_t> one{1, 1}, len{100, 20}, none{-1, -1}, zero{0, 0};
    const std::vector<int32_t> falls{0, 7, 2}, rises{0, 7, 9};
    // As many entries as the last bound says.
    const std::vector<int32_t> two{1, 2}, nine{0, 1, 2, 3, 4, 5, 6, 7, 0};
    // A sequence's list, then a prefix's.
    AttendBatch b{2, 0, one.data(), len.data(), none.data(), two.data(), falls.data(), nullptr, nullptr, nullptr};
    CHECK(p.plan(b, geo) == LORA_EINVAL && p.items().empty());
    b.pages = nine.data(), b.page0 = rises.data();
    CHECK(p.plan(b, geo) == LORA_OK && !p.items().empty());
    const std::vector<int32_t> flat{0, 0, 0};
    AttendBatch g{2, 2, one.data(), zero.data(), zero.data(), nullptr, flat.data(), len.data(), two.data(), falls.data()};
    CHECK(p.plan(g, geo) == LORA_EINVAL && p.items().empty());
    g.prefix_pages = nine.data(), g.prefix_page0 = rises.data();
    CHECK(p.plan(g, geo) == LORA_OK && !p.items().empty());
    std::printf("ok\n");
    return 0;
}
