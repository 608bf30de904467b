// Sums and maxima over teams of 2^k lanes of a wave, without LDS.
#pragma once

#include <type_traits>

#include "muon_internal.h"

namespace muon {

template <int CTRL>
__device__ __forceinline__ uint32_t lane_move(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}

// The two halves of a team of 2 * HALF lanes, each already alike in all its lanes,
// brought to every lane: op(own, other), T of 32 bits.  Every lane of the wave has
// to be active.  Within 16 lanes by lane moves (neighbours, pairs, mirrored
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

// v summed over the lanes that have the same place in their teams of L lanes,
// in every lane.
template <int L>
__device__ __forceinline__ float across_teams(float v) {
    auto turn = [&](auto ctrl) {
        v += __builtin_bit_cast(float, lane_move<ctrl.value>(__builtin_bit_cast(uint32_t, v)));
    };
    using std::integral_constant;
    if constexpr (L <= 8) turn(integral_constant<int, 0x128>{});  // rows of 16 lanes turned by 8, 4, 2, 1
    if constexpr (L <= 4) turn(integral_constant<int, 0x124>{});
    if constexpr (L <= 2) turn(integral_constant<int, 0x122>{});
    if constexpr (L <= 1) turn(integral_constant<int, 0x121>{});
    auto add = [](float a, float b) { return a + b; };
    if constexpr (L <= 16) v = team_step<16>(v, add);
    if constexpr (L <= 32) v = team_step<32>(v, add);
    return v;
}

// The wave's sum in every lane, in 64 bits.
__device__ __forceinline__ double wave_sum64(double v) {
    auto step = [&](auto ctrl) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint64_t o = (uint64_t)lane_move<ctrl.value>((uint32_t)(b >> 32)) << 32 | lane_move<ctrl.value>((uint32_t)b);
        v += __builtin_bit_cast(double, o);
    };
    using std::integral_constant;
    step(integral_constant<int, 0xb1>{});
    step(integral_constant<int, 0x4e>{});
    step(integral_constant<int, 0x141>{});
    step(integral_constant<int, 0x140>{});
    auto swap = [&](auto half) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32);
        const auto l = half.value == 16 ? __builtin_amdgcn_permlane16_swap(lo, lo, false, false)
                                        : __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
        const auto h = half.value == 16 ? __builtin_amdgcn_permlane16_swap(hi, hi, false, false)
                                        : __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
        v = __builtin_bit_cast(double, (uint64_t)h[0] << 32 | l[0]) + __builtin_bit_cast(double, (uint64_t)h[1] << 32 | l[1]);
    };
    swap(integral_constant<int, 16>{});
    swap(integral_constant<int, 32>{});
    return v;
}

// The sum of the lanes up to this one, within its row of 16 lanes.
__device__ __forceinline__ int row_prefix(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    return v;
}

// The sum of the lanes up to this one.
__device__ __forceinline__ int wave_prefix(int v) {
    // the rows before it: their last lanes go to rows 1 and 3, then to 2 and 3
    v = row_prefix(v);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
    return v;
}

}  // namespace muon
