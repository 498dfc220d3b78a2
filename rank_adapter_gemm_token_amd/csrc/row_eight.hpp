// row_eight.hpp -- rows of a vocabulary, which begin at any element and end
// anywhere, read eight neighbouring elements a lane.
#pragma once

#include "dtype.hpp"

namespace lora {

template <int DT>
struct Eight {
    using raw = typename Elem<DT>::raw;
    uint32_t w[2 * sizeof(raw)];

    __device__ __forceinline__ float at(int j) const {
        if constexpr (DT == DT_F32) return __uint_as_float(w[j]);
        else return Elem<DT>::to_f(static_cast<raw>(w[j / 2] >> (16 * (j % 2))));
    }
    __device__ __forceinline__ void put(int j, raw x) {
        if constexpr (DT == DT_F32) w[j] = x;
        else w[j / 2] = (w[j / 2] & (0xFFFFu << (16 * (1 - j % 2)))) | static_cast<uint32_t>(x) << (16 * (j % 2));
    }

    // The index of the first of those that load() brings for elements i .. i + 7
    // of a row of V: near the end, its last eight.
    static __device__ __forceinline__ int first(int i, int V) { return i + 8 <= V ? i : V - 8; }

    // No branch: several of these are in flight together.  (A load under a
    // branch for the row's end was waited for in it.)
    __device__ __forceinline__ void load(const raw *row, int i, int V) {
        if (V < 8) {  // uniform
#pragma unroll
            for (int j = 0; j < 8; ++j) put(j, row[j < V ? j : V - 1]);
            asm volatile("" ::: "memory");  // or these loads and the wide one become one set, element by element
        } else {
            __builtin_memcpy(w, row + first(i, V), sizeof w);
        }
    }

    // `none` in the place of what is not among elements i .. i + 7 of the row.
    __device__ __forceinline__ void clear(int i, int V, raw none) {
        const int skip = V < 8 ? i : i - first(i, V);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < skip || (V < 8 && j >= V)) put(j, none);
    }
};

}  // namespace lora
