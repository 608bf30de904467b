// Sums and maxima over teams of 2^k lanes of a wave, without LDS.
#pragma once

#include "muon_internal.h"

namespace muon {

template <int CTRL>
__device__ __forceinline__ uint32_t lane_move(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}

// (T: 32 bits.)  The two halves of a team of 2 * HALF lanes, each already alike in all its
// lanes, brought to every lane: op(own, other).  Every lane of the wave has to
// be active.  Within 16 lanes by lane moves (neighbours, pairs, mirrored
// halves and rows), beyond by v_permlane16_swap and v_permlane32_swap.
template <int HALF, class T, class F>
__device__ __forceinline__ T team_step(T v, F&& op) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    if constexpr (HALF >= 16) {
        const auto s = HALF == 16 ? __builtin_amdgcn_permlane16_swap(b, b, false, false)
                                  : __builtin_amdgcn_permlane32_swap(b, b, false, false);
        return op(__builtin_bit_cast(T, (uint32_t)s[0]), __builtin_bit_cast(T, (uint32_t)s[1]));
    } else {
        constexpr int ctrl = HALF == 1 ? 0xb1 : HALF == 2 ? 0x4e : HALF == 4 ? 0x141 : 0x140;
        return op(v, __builtin_bit_cast(T, lane_move<ctrl>(b)));
    }
}

// op over the team's L lanes, the same bits in every lane of the team (op is
// commutative, and both halves of a step combine the same two values).
template <int L, class T, class F>
__device__ __forceinline__ T team_reduce(T v, F&& op) {
    if constexpr (L > 1) v = team_step<1>(v, op);
    if constexpr (L > 2) v = team_step<2>(v, op);
    if constexpr (L > 4) v = team_step<4>(v, op);
    if constexpr (L > 8) v = team_step<8>(v, op);
    if constexpr (L > 16) v = team_step<16>(v, op);
    if constexpr (L > 32) v = team_step<32>(v, op);
    return v;
}

template <int L>
__device__ __forceinline__ float team_sum(float v) {
    return team_reduce<L>(v, [](float a, float b) { return a + b; });
}

}  // namespace muon
