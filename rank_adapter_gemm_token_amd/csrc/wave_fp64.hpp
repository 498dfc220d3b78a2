// wave_fp64.hpp -- sums of a wave's lanes in fp64, and the lane at which a
// running sum passes a number: what a token is drawn with.
#pragma once

#include "dtype.hpp"

namespace lora {

// v plus what lane data-parallel move CTRL brings to the lanes of the rows in
// MASK (nothing to the others).
template <int CTRL, int MASK>
__device__ __forceinline__ double add_moved(double v) {
    const uint64_t w = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(w), CTRL, MASK, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(w >> 32), CTRL, MASK, 0xf, false);
    return v + __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// Inclusive running sum over the wave's lanes, in registers: a sequence's
// answer waits for five of these one after the other, and by way of LDS each
// would take 0.3 us.
__device__ __forceinline__ double wave_scan(double v) {
    v = add_moved<0x111, 0xf>(v);  // row_shr:1
    v = add_moved<0x112, 0xf>(v);
    v = add_moved<0x114, 0xf>(v);
    v = add_moved<0x118, 0xf>(v);
    v = add_moved<0x142, 0xa>(v);     // lane 15 to the second and fourth row of 16
    return add_moved<0x143, 0xc>(v);  // lane 31 to the third and fourth
}

// Lane `l` of v, to all lanes.
__device__ __forceinline__ double lane_of(double v, int l) {
    const uint64_t w = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(w), l);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(w >> 32), l);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ double wave_sum(double v) { return lane_of(wave_scan(v), 63); }

// Of lanes that hold neighbouring runs' sums v, running r: the first with any
// weight whose running sum passes `aim`, or else the last with any weight.  (A
// lane of none may be the first to pass: the scan adds the same weights in
// another order for each lane, so its sum may stand a rounding above its left
// neighbour's.)
__device__ __forceinline__ int pick_lane(double v, double r, double aim) {
    const unsigned long long some = __ballot(v > 0.0), passes = __ballot(r > aim) & some;
    return uniform(passes ? __builtin_ctzll(passes) : some ? 63 - __builtin_clzll(some) : 0);
}

}  // namespace lora
