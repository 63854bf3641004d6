// exp of a double in plain multiply-adds, for kernels whose sums are checked
// to 64 bits (router shares, sampling masses).
//
// x = n ln 2 + r with |r| <= ln 2 / 2; exp(r) by its Taylor series to r^13
// (the next term is below 2^-57 of the value), scaled by 2^n.  Contraction is
// off and every fused step is written as one, so the same x gives the same
// bits wherever the function is inlined.  exp(-inf) = 0, NaN stays NaN; x at
// most 700.
#pragma once

#include <hip/hip_runtime.h>

namespace moe {

__device__ __forceinline__ double exp64(double x) {
#pragma clang fp contract(off)
    x = x < -800.0 ? -800.0 : x;
    const double n = rint(x * 1.4426950408889634);  // 1 / ln 2
    double r = fma(n, -0x1.62e42feep-1, x);  // ln 2 cut to 32 binary places: n times it is exact
    r = fma(n, -0x1.a39ef35793c76p-33, r);   // and the rest of ln 2
    double p = 1.0 / 6227020800.0;
    p = fma(p, r, 1.0 / 479001600.0);
    p = fma(p, r, 1.0 / 39916800.0);
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return ldexp(p, (int)n);
}

}  // namespace moe
