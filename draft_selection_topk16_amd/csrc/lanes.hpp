// Reductions and prefix sums over a wave without LDS: every step is a register
// move between lanes (DPP within 16 lanes, the row and half swaps of gfx950 beyond),
// a few cycles where a permutation through LDS takes over a hundred.
#pragma once

#include "common.hpp"

namespace df2 {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xf, 0xf, false);
}

// Both values of a pair of lanes (or rows, or halves) that a reduction's step
// joins, the same two in either; the step of distance O assumes that the
// distances below are done.
template <int O>
__device__ __forceinline__ void pair_of(uint32_t x, uint32_t& a, uint32_t& b) {
    static_assert(O == 1 || O == 2 || O == 4 || O == 8 || O == 16 || O == 32, "a power of two");
    a = x;
    if constexpr (O == 1) b = dpp_move<0xB1>(x);            // neighbours
    else if constexpr (O == 2) b = dpp_move<0x4E>(x);       // pairs of a quad
    else if constexpr (O == 4) b = dpp_move<0x141>(x);      // mirrored within 8
    else if constexpr (O == 8) b = dpp_move<0x140>(x);      // mirrored within 16
    else {
        const auto r = O == 16 ? __builtin_amdgcn_permlane16_swap(x, x, false, false)
                               : __builtin_amdgcn_permlane32_swap(x, x, false, false);
        a = r[0];
        b = r[1];
    }
}
template <int O>
__device__ __forceinline__ void pair_of(float x, float& a, float& b) {
    uint32_t u, v;
    pair_of<O>(__float_as_uint(x), u, v);
    a = __uint_as_float(u);
    b = __uint_as_float(v);
}
template <int O>
__device__ __forceinline__ void pair_of(double x, double& a, double& b) {
    const uint64_t w = (uint64_t)__double_as_longlong(x);
    uint32_t u0, v0, u1, v1;
    pair_of<O>((uint32_t)w, u0, v0);
    pair_of<O>((uint32_t)(w >> 32), u1, v1);
    a = __longlong_as_double((long long)(((uint64_t)u1 << 32) | u0));
    b = __longlong_as_double((long long)(((uint64_t)v1 << 32) | v0));
}

// op over groups of N lanes (a power of two), the result in each lane.
template <int N = 64, typename T, typename Op>
__device__ __forceinline__ T lanes_reduce(T x, Op op) {
    T a, b;
    if constexpr (N > 1) { pair_of<1>(x, a, b); x = op(a, b); }
    if constexpr (N > 2) { pair_of<2>(x, a, b); x = op(a, b); }
    if constexpr (N > 4) { pair_of<4>(x, a, b); x = op(a, b); }
    if constexpr (N > 8) { pair_of<8>(x, a, b); x = op(a, b); }
    if constexpr (N > 16) { pair_of<16>(x, a, b); x = op(a, b); }
    if constexpr (N > 32) { pair_of<32>(x, a, b); x = op(a, b); }
    return x;
}
template <int N = 64, typename T>
__device__ __forceinline__ T lanes_sum(T x) {
    return lanes_reduce<N>(x, [](T a, T b) { return a + b; });
}
template <int N = 64>
__device__ __forceinline__ float lanes_max(float x) {
    return lanes_reduce<N>(x, [](float a, float b) { return fmaxf(a, b); });
}

// One step of a prefix sum: x plus what the lane (or row, or half) before holds,
// for the lanes that have one.
template <int CTRL, int ROWS>
__device__ __forceinline__ int scan_step(int x) {
    return x + __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double scan_step(double x) {
    const uint64_t w = (uint64_t)__double_as_longlong(x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)w, CTRL, ROWS, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(w >> 32), CTRL, ROWS, 0xf, false);
    return x + __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
// Sum over the lanes up to this one.
template <typename T>
__device__ __forceinline__ T lanes_scan(T x) {
    x = scan_step<0x111, 0xf>(x);       // within 16 lanes: shifts by 1, 2, 4, 8
    x = scan_step<0x112, 0xf>(x);
    x = scan_step<0x114, 0xf>(x);
    x = scan_step<0x118, 0xf>(x);
    x = scan_step<0x142, 0xa>(x);       // lane 15 to the next 16, 47 likewise
    x = scan_step<0x143, 0xc>(x);       // lane 31 to the upper half
    return x;
}

__device__ __forceinline__ double lane_value(double x, int lane) {
    const uint64_t w = (uint64_t)__double_as_longlong(x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)w, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(w >> 32), lane);
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

}  // namespace df2
