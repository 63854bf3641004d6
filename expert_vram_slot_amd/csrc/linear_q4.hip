// Dense 4-bit product: y = x W^T (+ bias), W in 4-bit blocks with one fp16
// scale for each group of inputs of a row.
//
// y[t][n] = bias[n] + sum over groups b of d[n][b] * sum over k in b of
// x[t][k] * (q[n][k] - 8).  The codes lie as in a slab's Q4B32 plane (blocks
// of 32 inputs, byte j of a block: input j low, input j + 16 high), whatever
// the group.
//
// One wave takes one row and four tokens; a lane takes every 64th block of
// the row (16 bytes of codes), so a wave reads 1 KiB of a row at a time.
#include "common.hpp"

namespace {

using v4u = uint32_t __attribute__((ext_vector_type(4)));

constexpr int LIN_TOK = 4;

template <int XD>
__device__ __forceinline__ float load_x(const void* p, int64_t i) {
    if constexpr (XD == MOE_X_F32) return reinterpret_cast<const float*>(p)[i];
    else return moe::bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}

__device__ __forceinline__ void store_y(void* y, int y_dtype, int64_t i, float v) {
    if (y_dtype == MOE_X_F32) reinterpret_cast<float*>(y)[i] = v;
    else reinterpret_cast<__bf16*>(y)[i] = (__bf16)v;
}

template <int XD>
__global__ void __launch_bounds__(256) k_linear_q4(const void* __restrict__ x, int64_t ldx,
                                                   const v4u* __restrict__ wq, const _Float16* __restrict__ scales,
                                                   int gshift, const float* __restrict__ bias, int T, int N, int K,
                                                   void* __restrict__ y, int y_dtype, int64_t ldy) {
    const int lane = threadIdx.x & 63;
    const int n = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (n >= N) return;
    const int nb = K >> 5;
    for (int t0 = blockIdx.y * LIN_TOK; t0 < T; t0 += gridDim.y * LIN_TOK) {
        float acc[LIN_TOK] = {};
        for (int b = lane; b < nb; b += 64) {
            const v4u c = wq[(int64_t)n * nb + b];
            const float d = (float)scales[(int64_t)n * (K >> gshift) + ((b << 5) >> gshift)];
#pragma unroll
            for (int t = 0; t < LIN_TOK; ++t) {
                const int tt = t0 + t < T ? t0 + t : T - 1;
                float s = 0.0f;
                for (int j = 0; j < 16; ++j) {
                    const uint32_t byte = (c[j >> 2] >> (8 * (j & 3))) & 255u;
                    s = fmaf(load_x<XD>(x, tt * ldx + 32 * b + j), (float)((int)(byte & 15u) - 8), s);
                    s = fmaf(load_x<XD>(x, tt * ldx + 32 * b + 16 + j), (float)((int)(byte >> 4) - 8), s);
                }
                acc[t] = fmaf(d, s, acc[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < LIN_TOK; ++t) {
            const float v = moe::wave_sum(acc[t]);
            if (lane == 0 && t0 + t < T) store_y(y, y_dtype, (t0 + t) * ldy + n, bias ? v + bias[n] : v);
        }
    }
}

}  // namespace

extern "C" int moe_linear_q4(const void* x, int x_dtype, int64_t ldx, const void* wq, const void* scales, int group,
                             const float* bias, int T, int N, int K, void* y, int y_dtype, int64_t ldy,
                             hipStream_t stream) {
    MOE_REQUIRE((T == 0 || (x && y)) && wq && scales, MOE_E_ARG, "moe_linear_q4: x, wq, scales and y must be non-NULL");
    MOE_REQUIRE(T >= 0 && N >= 1 && K >= 1, MOE_E_ARG, "moe_linear_q4: T=%d N=%d K=%d", T, N, K);
    MOE_REQUIRE(x_dtype == MOE_X_F32 || x_dtype == MOE_X_BF16, MOE_E_DTYPE, "moe_linear_q4: activation format %d",
                x_dtype);
    MOE_REQUIRE(y_dtype == MOE_X_F32 || y_dtype == MOE_X_BF16, MOE_E_DTYPE, "moe_linear_q4: output format %d",
                y_dtype);
    MOE_REQUIRE(group == 32 || group == 64 || group == 128, MOE_E_SHAPE,
                "moe_linear_q4: groups of %d inputs (32, 64 or 128)", group);
    MOE_REQUIRE(K % group == 0, MOE_E_SHAPE, "moe_linear_q4: K=%d must be a multiple of the group of %d", K, group);
    MOE_REQUIRE(T <= MOE_LINEAR_MAX_T && N <= MOE_LINEAR_MAX_NK && K <= MOE_LINEAR_MAX_NK, MOE_E_SHAPE,
                "moe_linear_q4: T=%d N=%d K=%d beyond the limits", T, N, K);
    MOE_REQUIRE(ldx >= K && ldy >= N, MOE_E_ARG, "moe_linear_q4: row strides %lld and %lld below K=%d and N=%d",
                (long long)ldx, (long long)ldy, K, N);
    MOE_REQUIRE(ldx <= MOE_LINEAR_MAX_LD && ldy <= MOE_LINEAR_MAX_LD, MOE_E_SHAPE,
                "moe_linear_q4: row strides %lld and %lld beyond the limit", (long long)ldx, (long long)ldy);
    const int64_t xrow = ldx * (x_dtype == MOE_X_F32 ? 4 : 2);
    MOE_REQUIRE(moe_aligned16(x) && moe_aligned16(wq) && (T <= 1 || xrow % 16 == 0), MOE_E_ALIGN,
                "moe_linear_q4: x, its rows and wq must start on 16 bytes");
    const uintptr_t ym = y_dtype == MOE_X_F32 ? 3 : 1;
    MOE_REQUIRE(!(reinterpret_cast<uintptr_t>(scales) & 1u) && !(reinterpret_cast<uintptr_t>(bias) & 3u) &&
                    !(reinterpret_cast<uintptr_t>(y) & ym),
                MOE_E_ALIGN, "moe_linear_q4: scales, bias and y must be aligned to their elements");
    if (T == 0) return moe_ok();
    const int gshift = group == 32 ? 5 : group == 64 ? 6 : 7;
    const int gy = (T + LIN_TOK - 1) / LIN_TOK;
    const dim3 grid((unsigned)((N + 3) / 4), (unsigned)(gy < 65535 ? gy : 65535));
    auto k = x_dtype == MOE_X_F32 ? k_linear_q4<MOE_X_F32> : k_linear_q4<MOE_X_BF16>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, stream, x, ldx, reinterpret_cast<const v4u*>(wq),
                       reinterpret_cast<const _Float16*>(scales), gshift, bias, T, N, K, y, y_dtype, ldy);
    return moe_check_launch("moe_linear_q4");
}
