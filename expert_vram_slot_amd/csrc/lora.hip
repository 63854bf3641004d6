// Low-rank adapters of many requests beside a shared product:
//   y_t = base_t + scale_i B_i (A_i x_t), i = ids_t
// in two passes: h = scale A x (each token with its own adapter's rows), then
// y = base + B h.
#include "common.hpp"

namespace {

struct LoraArgs {
    const void* x;
    int64_t ldx;
    const uint16_t* a;
    const uint16_t* b;
    const int32_t* ranks;
    const float* scale;
    const int32_t* ids;
    int n, r, T, N, K;
    const void* base;
    int64_t ldb;
    void* y;
    int64_t ldy;
    float* h;  // [T][r]
};

// The adapter of token t and its rank; 0: none.
__device__ __forceinline__ int adapter(const LoraArgs& a, int64_t t, int& rank) {
    const int i = a.ids[t];
    rank = i < 0 || i >= a.n ? 0 : a.ranks ? min(max(a.ranks[i], 0), a.r) : a.r;
    return i;
}

template <int D>
__device__ __forceinline__ float load(const void* p, int64_t i) {
    if constexpr (D == MOE_X_F32) return reinterpret_cast<const float*>(p)[i];
    else return moe::bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}

// One workgroup a token, one wave a row of A at a time.
template <int XD>
__global__ void __launch_bounds__(256) k_lora_down(LoraArgs a) {
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    int rank;
    const int i = adapter(a, t, rank);
    for (int j = wid; j < rank; j += 4) {
        const uint16_t* row = a.a + ((int64_t)i * a.r + j) * a.K;
        float s = 0.0f;
        for (int k = lane; k < a.K; k += 64) s = fmaf(load<XD>(a.x, t * a.ldx + k), moe::bf16_to_f32(row[k]), s);
        s = moe::wave_sum(s);
        if (lane == 0) a.h[t * a.r + j] = a.scale ? a.scale[i] * s : s;
    }
}

// One thread an output.
template <int YD>
__global__ void __launch_bounds__(256) k_lora_up(LoraArgs a) {
    const int64_t t = blockIdx.y;
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= a.N) return;
    int rank;
    const int i = adapter(a, t, rank);
    float s = 0.0f;
    for (int j = 0; j < rank; ++j)
        s = fmaf(a.h[t * a.r + j], moe::bf16_to_f32(a.b[((int64_t)i * a.N + n) * a.r + j]), s);
    const float v = (a.base ? load<YD>(a.base, t * a.ldb + n) : 0.0f) + s;
    if constexpr (YD == MOE_X_F32) reinterpret_cast<float*>(a.y)[t * a.ldy + n] = v;
    else reinterpret_cast<__bf16*>(a.y)[t * a.ldy + n] = (__bf16)v;
}

bool on_elements(const void* p, int dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == MOE_X_F32 ? 3u : 1u)) == 0;
}

}  // namespace

extern "C" {

size_t moe_lora_workspace_bytes(int T, int K, int r) {
    if (T < 0 || T > MOE_LINEAR_MAX_T || K < 8 || K > MOE_LINEAR_MAX_NK || r < 8 || r > MOE_LORA_MAX_R) return 0;
    return (size_t)(T > 0 ? T : 1) * r * 4;
}

int moe_lora_add(const void* x, int x_dtype, int64_t ldx, const void* a, const void* b, const int32_t* ranks,
                 const float* scale, const int32_t* ids, int n, int r, int T, int N, int K, const void* base,
                 int64_t ldb, void* y, int y_dtype, int64_t ldy, void* ws, size_t ws_bytes, hipStream_t stream) {
    MOE_REQUIRE(T >= 0 && N >= 1 && K >= 1 && n >= 1 && r >= 1, MOE_E_ARG, "moe_lora_add: T=%d N=%d K=%d n=%d r=%d", T,
                N, K, n, r);
    MOE_REQUIRE(a && b && ws && (T == 0 || (x && ids && y)), MOE_E_ARG,
                "moe_lora_add: x, a, b, ids, y and ws must be non-NULL");
    MOE_REQUIRE(ldx >= K && ldy >= N && (!base || ldb >= N), MOE_E_ARG, "moe_lora_add: ldx, ldb or ldy shorter than a row");
    MOE_REQUIRE(base != y || !base || ldb == ldy, MOE_E_ARG, "moe_lora_add: y is base, with other strides");
    MOE_REQUIRE((x_dtype == MOE_X_F32 || x_dtype == MOE_X_BF16) && (y_dtype == MOE_X_F32 || y_dtype == MOE_X_BF16),
                MOE_E_DTYPE, "moe_lora_add: formats %d, %d", x_dtype, y_dtype);
    MOE_REQUIRE(K % 8 == 0 && r % 8 == 0 && r <= MOE_LORA_MAX_R && n <= MOE_LORA_MAX_N && T <= MOE_LINEAR_MAX_T &&
                    N <= MOE_LINEAR_MAX_NK && K <= MOE_LINEAR_MAX_NK && ldx <= MOE_LINEAR_MAX_LD &&
                    ldy <= MOE_LINEAR_MAX_LD && (!base || ldb <= MOE_LINEAR_MAX_LD),
                MOE_E_SHAPE, "moe_lora_add: T=%d N=%d K=%d n=%d r=%d beyond the limits or not in eights", T, N, K, n, r);
    MOE_REQUIRE(moe_aligned16(x) && moe_aligned16(a) && moe_aligned16(b) && moe_aligned16(ws) &&
                    ldx % (x_dtype == MOE_X_F32 ? 4 : 8) == 0 && on_elements(base, y_dtype) && on_elements(y, y_dtype) &&
                    on_elements(ids, MOE_X_F32) && on_elements(ranks, MOE_X_F32) && on_elements(scale, MOE_X_F32),
                MOE_E_ALIGN, "moe_lora_add: x, its rows, a, b and ws must start on 16 bytes, the others on their elements");
    MOE_REQUIRE(ws_bytes >= moe_lora_workspace_bytes(T, K, r), MOE_E_ARG, "moe_lora_add: workspace of %zu bytes, %zu needed",
                ws_bytes, moe_lora_workspace_bytes(T, K, r));
    if (T == 0) return moe_ok();
    const LoraArgs g{x, ldx, reinterpret_cast<const uint16_t*>(a), reinterpret_cast<const uint16_t*>(b), ranks, scale,
                     ids, n, r, T, N, K, base, ldb, y, ldy, reinterpret_cast<float*>(ws)};
    if (x_dtype == MOE_X_F32) hipLaunchKernelGGL(k_lora_down<MOE_X_F32>, dim3(T), dim3(256), 0, stream, g);
    else hipLaunchKernelGGL(k_lora_down<MOE_X_BF16>, dim3(T), dim3(256), 0, stream, g);
    if (int rc = moe_check_launch("moe_lora_add/down")) return rc;
    for (int t0 = 0; t0 < T; t0 += 65535) {
        LoraArgs c = g;
        const int rows = T - t0 < 65535 ? T - t0 : 65535;
        const size_t yb = y_dtype == MOE_X_F32 ? 4 : 2;
        c.ids += t0, c.h += (size_t)t0 * r;
        c.y = reinterpret_cast<char*>(y) + (size_t)t0 * ldy * yb;
        if (base) c.base = reinterpret_cast<const char*>(base) + (size_t)t0 * ldb * yb;
        const dim3 grid((N + 255) / 256, rows);
        if (y_dtype == MOE_X_F32) hipLaunchKernelGGL(k_lora_up<MOE_X_F32>, grid, dim3(256), 0, stream, c);
        else hipLaunchKernelGGL(k_lora_up<MOE_X_BF16>, grid, dim3(256), 0, stream, c);
        if (int rc = moe_check_launch("moe_lora_add/up")) return rc;
    }
    return moe_ok();
}

}  // extern "C"
