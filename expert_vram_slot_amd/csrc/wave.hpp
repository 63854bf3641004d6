// Reductions over the 64 lanes of a wave without LDS: data-parallel-primitive
// moves inside each row of 16 lanes, then the row swaps.  Every lane ends with
// the result, and with the same bits: each step adds the same two numbers in
// both lanes of a pair.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// v of lane ^ 1, of lane ^ 2, of the lane mirrored in its half row, in its row
constexpr int DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E, DPP_HALF_MIRROR = 0x141, DPP_MIRROR = 0x140;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

template <int CTRL, typename T>
__device__ __forceinline__ T dpp_of(T v) {
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(T, dpp<CTRL>(__builtin_bit_cast(uint32_t, v)));
    } else {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        return __builtin_bit_cast(T, (uint64_t)dpp<CTRL>((uint32_t)b) | ((uint64_t)dpp<CTRL>((uint32_t)(b >> 32)) << 32));
    }
}

// The two values that rows 2i and 2i + 1 (FAR: lanes below and above 32) hold.
template <bool FAR, typename T>
__device__ __forceinline__ void row_pair(T v, T& a, T& b) {
    const auto swap = [](uint32_t x, uint32_t& lo, uint32_t& hi) {
        if constexpr (FAR) {
            const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
            lo = r[0], hi = r[1];
        } else {
            const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
            lo = r[0], hi = r[1];
        }
    };
    if constexpr (sizeof(T) == 4) {
        uint32_t x, y;
        swap(__builtin_bit_cast(uint32_t, v), x, y);
        a = __builtin_bit_cast(T, x), b = __builtin_bit_cast(T, y);
    } else {
        const uint64_t w = __builtin_bit_cast(uint64_t, v);
        uint32_t x0, y0, x1, y1;
        swap((uint32_t)w, x0, y0);
        swap((uint32_t)(w >> 32), x1, y1);
        a = __builtin_bit_cast(T, x0 | ((uint64_t)x1 << 32)), b = __builtin_bit_cast(T, y0 | ((uint64_t)y1 << 32));
    }
}

template <typename T, typename Op>
__device__ __forceinline__ T wave_all(T v, Op op) {
    v = op(v, dpp_of<DPP_XOR1>(v));
    v = op(v, dpp_of<DPP_XOR2>(v));
    v = op(v, dpp_of<DPP_HALF_MIRROR>(v));
    v = op(v, dpp_of<DPP_MIRROR>(v));
    T a, b;
    row_pair<false>(v, a, b);
    v = op(a, b);
    row_pair<true>(v, a, b);
    return op(a, b);
}

template <typename T>
__device__ __forceinline__ T wave_all_sum(T v) {
    return wave_all(v, [](T a, T b) { return a + b; });
}

// v of the lane that CTRL names, in the rows of the mask ROWS; 0 where there is none.
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T dpp_or_0(T v) {
    const auto move = [](uint32_t w) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, CTRL, ROWS, 0xF, false); };
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(T, move(__builtin_bit_cast(uint32_t, v)));
    } else {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        return __builtin_bit_cast(T, (uint64_t)move((uint32_t)b) | ((uint64_t)move((uint32_t)(b >> 32)) << 32));
    }
}

// Inclusive sum over the lanes up to this one.
template <typename T>
__device__ __forceinline__ T wave_upto(T v) {
    v += dpp_or_0<0x111, 0xF>(v);  // from 1, 2, 4, 8 lanes below in the row of 16
    v += dpp_or_0<0x112, 0xF>(v);
    v += dpp_or_0<0x114, 0xF>(v);
    v += dpp_or_0<0x118, 0xF>(v);
    v += dpp_or_0<0x142, 0xA>(v);  // lane 15 of rows 0 and 2 to rows 1 and 3
    v += dpp_or_0<0x143, 0xC>(v);  // lane 31 to rows 2 and 3
    return v;
}

__device__ __forceinline__ float wave_all_max(float v) {
    return wave_all(v, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace moe
