// Router statistics of a batch: picks and share of router mass per expert,
// the balance loss and the z loss, and the gradient of both to the logits.
//
// With p_t = softmax(z_t) over the n counted tokens, c_e the picks of expert
// e, f_e = c_e / sum c and P_e = mean of p_te:
//   balance  L_b = E * sum_e f_e P_e        z loss  L_z = mean lse_t^2
//   dz_te = p_te * (g_b E (f_e - sum_e' f_e' p_te') + 2 g_z lse_t) / n
// (the picks are whole numbers and carry no gradient).
//
// P_e is the brightness that "Nudge, don't cut" (oois.ee/pgo-sgb), "The method
// in five lines", grades its bias by, so it is made in double: the softmax and
// its sums run in double, in a fixed order.  One wave takes one token at a
// time and keeps its experts' running sums in registers (lane l holds experts
// l, l + 64, ...).
#include <math.h>

#include "common.hpp"

namespace {

constexpr int BAL_THREADS = 256;
constexpr int BAL_WAVES = BAL_THREADS / 64;
constexpr int BAL_MAX_BLOCKS = 512;

template <int ZD>
__device__ __forceinline__ float load_z(const void* p, int64_t i) {
    if constexpr (ZD == MOE_X_F32) return reinterpret_cast<const float*>(p)[i];
    else return moe::bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) v = fmaxf(v, __shfl_xor(v, s, moe::WAVE));
    return v;
}

// Workspace: per block, the sums of p per expert, the sum of lse^2, the picks
// per expert and the counted tokens.
struct BalWs {
    double* share;   // [blocks][E]
    double* lse2;    // [blocks]
    int32_t* picks;  // [blocks][E]
    int32_t* toks;   // [blocks]
};

__host__ __device__ inline size_t bal_bytes(int blocks, int E) { return (size_t)blocks * (12 * (size_t)E + 12); }

inline int bal_blocks(int T) {
    const int b = (T + BAL_WAVES - 1) / BAL_WAVES;
    return b < 1 ? 1 : b < BAL_MAX_BLOCKS ? b : BAL_MAX_BLOCKS;
}

inline BalWs bal_ws(void* ws, int blocks, int E) {
    BalWs w;
    w.share = reinterpret_cast<double*>(ws);
    w.lse2 = w.share + (size_t)blocks * E;
    w.picks = reinterpret_cast<int32_t*>(w.lse2 + blocks);
    w.toks = w.picks + (size_t)blocks * E;
    return w;
}

template <int ZD, int NE>
__global__ void __launch_bounds__(BAL_THREADS) k_balance(const void* __restrict__ z, const int32_t* __restrict__ ids,
                                                         const uint8_t* __restrict__ mask, int T, int E, int k,
                                                         float* __restrict__ lse, BalWs ws) {
    extern __shared__ __align__(16) unsigned char smem[];
    double* s_share = reinterpret_cast<double*>(smem);                 // [E]
    double* s_lse2 = s_share + E;                                      // [BAL_WAVES]
    int32_t* s_picks = reinterpret_cast<int32_t*>(s_lse2 + BAL_WAVES);  // [E]
    int32_t* s_toks = s_picks + E;                                     // [BAL_WAVES]
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    for (int e = threadIdx.x; e < E; e += BAL_THREADS) s_picks[e] = 0;
    __syncthreads();
    double acc[NE] = {}, lse2 = 0.0;
    int toks = 0;
    for (int64_t t = (int64_t)blockIdx.x * BAL_WAVES + wid; t < T; t += (int64_t)gridDim.x * BAL_WAVES) {
        bool live = !mask || mask[t];
        float v[NE], m = -INFINITY;
        if (live) {
#pragma unroll
            for (int j = 0; j < NE; ++j) {
                const int e = lane + 64 * j;
                v[j] = e < E ? load_z<ZD>(z, t * E + e) : -INFINITY;
                m = fmaxf(m, v[j]);
            }
            m = wave_max(m);  // NaN loses every comparison: looked for where nothing else is left
            bool nan = false;
            if (m == -INFINITY) {
#pragma unroll
                for (int j = 0; j < NE; ++j) nan |= v[j] != v[j];
            }
            live = m > -INFINITY || __any(nan);
        }
        float out = 0.0f;
        if (live) {
            double p[NE], sum = 0.0;
#pragma unroll
            for (int j = 0; j < NE; ++j) sum += p[j] = exp((double)v[j] - (double)m);
            sum = moe::wave_sum(sum);
            const double r = 1.0 / sum, l = (double)m + log(sum);
#pragma unroll
            for (int j = 0; j < NE; ++j) acc[j] += p[j] * r;
            lse2 += l * l;
            out = (float)l;
            ++toks;
            for (int j = lane; j < k; j += 64) {
                const int e = ids[t * k + j];
                if (e >= 0 && e < E) atomicAdd(&s_picks[e], 1);
            }
        }
        if (lane == 0) lse[t] = out;
    }
    for (int w = 0; w < BAL_WAVES; ++w) {
        if (wid == w) {
#pragma unroll
            for (int j = 0; j < NE; ++j) {
                const int e = lane + 64 * j;
                if (e < E) s_share[e] = w ? s_share[e] + acc[j] : acc[j];
            }
            if (lane == 0) s_lse2[w] = lse2, s_toks[w] = toks;
        }
        __syncthreads();
    }
    for (int e = threadIdx.x; e < E; e += BAL_THREADS) {
        ws.share[(int64_t)blockIdx.x * E + e] = s_share[e];
        ws.picks[(int64_t)blockIdx.x * E + e] = s_picks[e];
    }
    if (threadIdx.x == 0) {
        double l = 0.0;
        int n = 0;
        for (int w = 0; w < BAL_WAVES; ++w) l += s_lse2[w], n += s_toks[w];
        ws.lse2[blockIdx.x] = l;
        ws.toks[blockIdx.x] = n;
    }
}

__global__ void __launch_bounds__(1024) k_balance_final(BalWs ws, int blocks, int E, int32_t* __restrict__ counts,
                                                        int32_t* __restrict__ totals, double* __restrict__ share,
                                                        float* __restrict__ loss) {
    __shared__ double s_dot[16];
    __shared__ int64_t s_picks[16];
    int n = 0;
    double l2 = 0.0;
    for (int b = 0; b < blocks; ++b) n += ws.toks[b], l2 += ws.lse2[b];
    const double inv = n > 0 ? 1.0 / n : 0.0;
    double dot = 0.0;
    int64_t picks = 0;
    for (int e = threadIdx.x; e < E; e += 1024) {
        double s = 0.0;
        int c = 0;
        for (int b = 0; b < blocks; ++b) s += ws.share[(int64_t)b * E + e], c += ws.picks[(int64_t)b * E + e];
        s *= inv;
        counts[e] = c;
        share[e] = s;
        dot += s * c;
        picks += c;
    }
    dot = moe::wave_sum(dot);
    picks = moe::wave_sum((long long)picks);
    if ((threadIdx.x & 63) == 0) s_dot[threadIdx.x >> 6] = dot, s_picks[threadIdx.x >> 6] = picks;
    __syncthreads();
    if (threadIdx.x == 0) {
        dot = 0.0;
        picks = 0;
        for (int w = 0; w < 16; ++w) dot += s_dot[w], picks += s_picks[w];
        totals[0] = n;
        totals[1] = (int32_t)picks;
        loss[0] = picks > 0 ? (float)(E * dot / (double)picks) : 0.0f;
        loss[1] = (float)(l2 * inv);
    }
}

// f is taken less its mean 1/E, as whole numbers over whole numbers: the
// subtraction f_e - sum f p of nearly equal numbers (a balanced router) then
// costs no digits, since sum p = 1.
template <int ZD, int NE>
__global__ void __launch_bounds__(BAL_THREADS) k_balance_bwd(const void* __restrict__ z, const float* __restrict__ lse,
                                                             const uint8_t* __restrict__ mask,
                                                             const int32_t* __restrict__ counts,
                                                             const int32_t* __restrict__ totals,
                                                             const float* __restrict__ dloss, int T, int E,
                                                             void* __restrict__ dz) {
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const int n = totals[0], picks = totals[1];
    const double rn = n > 0 ? 1.0 / n : 0.0;
    const double gb = picks > 0 ? (double)dloss[0] * rn / picks : 0.0;
    const float gz = (float)(2.0 * (double)dloss[1] * rn);
    float f[NE];  // g_b E (f_e - 1/E) / n
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const int e = lane + 64 * j;
        f[j] = e < E ? (float)((double)((int64_t)counts[e] * E - picks) * gb) : 0.0f;
    }
    for (int64_t t = (int64_t)blockIdx.x * BAL_WAVES + wid; t < T; t += (int64_t)gridDim.x * BAL_WAVES) {
        const bool live = !mask || mask[t];
        float p[NE], dot = 0.0f;
        const float l = lse[t];
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const int e = lane + 64 * j;
            p[j] = live && e < E ? expf(load_z<ZD>(z, t * E + e) - l) : 0.0f;
            dot = fmaf(p[j], f[j], dot);
        }
        dot = moe::wave_sum(dot);
        const float c = gz * l - dot;
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const int e = lane + 64 * j;
            if (e >= E) continue;
            const float d = live ? p[j] * (f[j] + c) : 0.0f;
            if constexpr (ZD == MOE_X_F32) reinterpret_cast<float*>(dz)[t * E + e] = d;
            else reinterpret_cast<__bf16*>(dz)[t * E + e] = (__bf16)d;
        }
    }
}

template <int ZD>
void launch_rows(int blocks, size_t lds, hipStream_t st, const void* z, const int32_t* ids, const uint8_t* mask, int T,
                 int E, int k, float* lse, BalWs ws) {
    const auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3(blocks), dim3(BAL_THREADS), lds, st, z, ids, mask, T, E, k, lse, ws);
    };
    if (E <= 64) go(k_balance<ZD, 1>);
    else if (E <= 128) go(k_balance<ZD, 2>);
    else if (E <= 256) go(k_balance<ZD, 4>);
    else if (E <= 512) go(k_balance<ZD, 8>);
    else if (E <= 1024) go(k_balance<ZD, 16>);
    else if (E <= 2048) go(k_balance<ZD, 32>);
    else go(k_balance<ZD, 64>);
}

template <int ZD>
void launch_bwd(int blocks, hipStream_t st, const void* z, const float* lse, const uint8_t* mask,
                const int32_t* counts, const int32_t* totals, const float* dloss, int T, int E, void* dz) {
    const auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3(blocks), dim3(BAL_THREADS), 0, st, z, lse, mask, counts, totals, dloss, T, E, dz);
    };
    if (E <= 64) go(k_balance_bwd<ZD, 1>);
    else if (E <= 128) go(k_balance_bwd<ZD, 2>);
    else if (E <= 256) go(k_balance_bwd<ZD, 4>);
    else if (E <= 512) go(k_balance_bwd<ZD, 8>);
    else if (E <= 1024) go(k_balance_bwd<ZD, 16>);
    else if (E <= 2048) go(k_balance_bwd<ZD, 32>);
    else go(k_balance_bwd<ZD, 64>);
}

}  // namespace

extern "C" {

size_t moe_balance_workspace_bytes(int T, int E) {
    if (T < 0 || T > MOE_BALANCE_MAX_T || E < 1 || E > MOE_MAX_E) return 0;
    return (bal_bytes(bal_blocks(T), E) + 15) & ~(size_t)15;
}

int moe_balance_loss(const void* z, int z_dtype, const int32_t* ids, const uint8_t* mask, int T, int E, int k,
                     int32_t* counts, int32_t* totals, double* share, float* lse, float* loss, void* ws,
                     size_t ws_bytes, hipStream_t stream) {
    MOE_REQUIRE((T == 0 || (z && ids && lse)) && counts && totals && share && loss && ws, MOE_E_ARG,
                "moe_balance_loss: z, ids, the outputs and ws must be non-NULL");
    MOE_REQUIRE(T >= 0 && E >= 1 && k >= 1, MOE_E_ARG, "moe_balance_loss: T=%d E=%d k=%d", T, E, k);
    MOE_REQUIRE(z_dtype == MOE_X_F32 || z_dtype == MOE_X_BF16, MOE_E_DTYPE, "moe_balance_loss: logit format %d",
                z_dtype);
    MOE_REQUIRE(E <= MOE_MAX_E && k <= E && k <= MOE_MAX_K && T <= MOE_BALANCE_MAX_T, MOE_E_SHAPE,
                "moe_balance_loss: T=%d E=%d k=%d beyond the limits", T, E, k);
    MOE_REQUIRE(moe_aligned16(z) && moe_aligned16(ws) && moe_aligned16(share), MOE_E_ALIGN,
                "moe_balance_loss: z, share and ws must start on 16 bytes");
    MOE_REQUIRE(ws_bytes >= moe_balance_workspace_bytes(T, E), MOE_E_ARG,
                "moe_balance_loss: workspace of %zu bytes, %zu needed", ws_bytes, moe_balance_workspace_bytes(T, E));
    const int blocks = bal_blocks(T);
    const BalWs w = bal_ws(ws, blocks, E);
    const size_t lds = 12 * (size_t)E + 12 * BAL_WAVES;
    if (z_dtype == MOE_X_F32) launch_rows<MOE_X_F32>(blocks, lds, stream, z, ids, mask, T, E, k, lse, w);
    else launch_rows<MOE_X_BF16>(blocks, lds, stream, z, ids, mask, T, E, k, lse, w);
    if (int rc = moe_check_launch("moe_balance_loss")) return rc;
    hipLaunchKernelGGL(k_balance_final, dim3(1), dim3(1024), 0, stream, w, blocks, E, counts, totals, share, loss);
    return moe_check_launch("moe_balance_loss/final");
}

int moe_balance_loss_bwd(const void* z, int z_dtype, const float* lse, const uint8_t* mask, const int32_t* counts,
                         const int32_t* totals, const float* dloss, int T, int E, void* dz, hipStream_t stream) {
    MOE_REQUIRE((T == 0 || (z && lse && dz)) && counts && totals && dloss, MOE_E_ARG,
                "moe_balance_loss_bwd: z, lse, counts, totals, dloss and dz must be non-NULL");
    MOE_REQUIRE(T >= 0 && E >= 1, MOE_E_ARG, "moe_balance_loss_bwd: T=%d E=%d", T, E);
    MOE_REQUIRE(z_dtype == MOE_X_F32 || z_dtype == MOE_X_BF16, MOE_E_DTYPE, "moe_balance_loss_bwd: logit format %d",
                z_dtype);
    MOE_REQUIRE(E <= MOE_MAX_E && T <= MOE_BALANCE_MAX_T, MOE_E_SHAPE,
                "moe_balance_loss_bwd: T=%d E=%d beyond the limits", T, E);
    MOE_REQUIRE(moe_aligned16(z) && moe_aligned16(dz), MOE_E_ALIGN,
                "moe_balance_loss_bwd: z and dz must start on 16 bytes");
    if (T == 0) return moe_ok();
    const int blocks = (T + BAL_WAVES - 1) / BAL_WAVES < 2048 ? (T + BAL_WAVES - 1) / BAL_WAVES : 2048;
    if (z_dtype == MOE_X_F32) launch_bwd<MOE_X_F32>(blocks, stream, z, lse, mask, counts, totals, dloss, T, E, dz);
    else launch_bwd<MOE_X_BF16>(blocks, stream, z, lse, mask, counts, totals, dloss, T, E, dz);
    return moe_check_launch("moe_balance_loss_bwd");
}

}  // extern "C"
