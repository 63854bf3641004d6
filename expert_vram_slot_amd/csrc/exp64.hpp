// exp of a double in plain multiply-adds, for kernels whose sums are checked
// to 64 bits (router shares, sampling masses).
//
// x = n ln 2 + r with |r| <= ln 2 / 2; exp(r) by the polynomial of degree 10
// through its values at the 11 Chebyshev nodes of that interval (relative
// error below 2^-51.6), times 2^n by an addition to the exponent.  n is taken
// from the low word of x / ln 2 + 1.5 * 2^52, with no conversion.  Contraction
// is off and every fused step is written as one, so the same x gives the same
// bits wherever the function is inlined.  0 below -708 (the smallest normal
// numbers), NaN stays NaN; x at most 700.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// a * b + c with c in scalar registers.  Left to itself the compiler copies
// each of the polynomial's constants into vector registers first, which is as
// dear as the step.
__device__ __forceinline__ double fma_s(double a, double b, double c) {
    double d;
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "s"(c));
    return d;
}

__device__ __forceinline__ double exp64(double x) {
#pragma clang fp contract(off)
    constexpr double SHIFT = 0x1.8p52;
    const double t = fma(x, 1.4426950408889634, SHIFT);  // 1 / ln 2
    const double n = t - SHIFT;
    double r = fma(n, -0x1.62e42feep-1, x);  // ln 2 cut to 32 binary places: n times it is exact
    r = fma(n, -0x1.a39ef35793c76p-33, r);   // and the rest of ln 2
    double p = fma_s(0x1.28a2c0a99e1f7p-22, r, 0x1.72faf02873319p-19);
    p = fma_s(p, r, 0x1.a019a66a7378bp-16);
    p = fma_s(p, r, 0x1.a01978c6b760ep-13);
    p = fma_s(p, r, 0x1.6c16c17f43a64p-10);
    p = fma_s(p, r, 0x1.1111112dd67d7p-7);
    p = fma_s(p, r, 0x1.55555555520afp-5);
    p = fma_s(p, r, 0x1.555555554b757p-3);
    p = fma_s(p, r, 0x1.0000000000005p-1);
    p = fma_s(p, r, 0x1.000000000001ep+0);
    p = fma(p, r, 1.0);
    const uint64_t b = __builtin_bit_cast(uint64_t, p);
    const uint32_t hi = (uint32_t)(b >> 32) + ((uint32_t)__builtin_bit_cast(uint64_t, t) << 20);
    const double v = __builtin_bit_cast(double, (uint64_t)(uint32_t)b | ((uint64_t)hi << 32));
    return x < -708.0 ? 0.0 : v;
}

}  // namespace moe
