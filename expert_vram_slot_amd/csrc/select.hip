// Selection rules of a router beyond moe_route's: sigmoid or softmax scores, a
// bias on the scores for the choice alone, groups, top-k, weights renormalised or
// not; the gradient of the weights to the logits; and a step of the bias that
// balances the picks.
//
//   c_e = s_e + b_e      picks: the k first by (c falling, z falling, id rising)
//   w_i = scale s_i [/ sum_j s_j]
// With h = scale dw, and q the weights over scale:
//   sigmoid  dz_i += s_i (1 - s_i) h_i          renormalised  q_i (1 - s_i) (h_i - sum h q)
//   softmax  dz_e = p_e (h_e - sum h p)         renormalised  q_i (h_i - sum h q)
// Choices decide which expert a token goes to, so they are compared as 64-bit
// numbers: fp32 would let experts nearly as good change places.
#include <math.h>

#include <type_traits>

#include "common.hpp"
#include "exp64.hpp"
#include "wave.hpp"

namespace {

constexpr int SEL_WAVES = 4;

struct SelArgs {
    const void* z;
    const float* bias;
    const uint8_t* mask;
    const int32_t* ids_in;
    int T, E, k;
    moe_select_rule rule;
    int32_t* ids;
    float* w;
};

template <int ZD>
__device__ __forceinline__ float load_z(const void* z, int64_t i) {
    if constexpr (ZD == MOE_X_F32) return reinterpret_cast<const float*>(z)[i];
    else return moe::bf16_to_f32(reinterpret_cast<const uint16_t*>(z)[i]);
}

// s of a sigmoid and 1 - s
__device__ __forceinline__ double sigmoid64(double z, double& rest) {
    const double e = moe::exp64(-fabs(z)), r = 1.0 / (1.0 + e);
    rest = z >= 0.0 ? e * r : r;
    return z >= 0.0 ? r : e * r;
}

// Softmax terms: exp(z - m), with every +inf counting 1 where m is +inf.
__device__ __forceinline__ double soft64(float z, float m) { return z == m ? 1.0 : moe::exp64((double)z - (double)m); }

// s_i over the sum of s over a token's picks (lane i, live: a pick with a score),
// from ratios to the largest pick's score, which neither vanish nor overflow.
__device__ __forceinline__ double share64(int score, float z, bool live) {
    const float m = moe::wave_all_max(live ? z : -INFINITY);
    double r = 0.0;
    if (live) {
        r = soft64(score == MOE_SCORE_SIGMOID ? fminf(z, 0.0f) : z, score == MOE_SCORE_SIGMOID ? fminf(m, 0.0f) : m);
        if (score == MOE_SCORE_SIGMOID) r *= (1.0 + moe::exp64(-fabs((double)m))) / (1.0 + moe::exp64(-fabs((double)z)));
    }
    const double sum = moe::wave_all_sum(r);
    return sum > 0.0 ? r / sum : 0.0;
}

// One wave a token; lane l holds experts l, l + 64, ...
template <int ZD, int NE>
__global__ void __launch_bounds__(64 * SEL_WAVES) k_select(SelArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 6) + wid;
    if (t >= a.T) return;
    const int E = a.E, k = a.k, G = a.rule.groups, gs = E / G;
    double* row = reinterpret_cast<double*>(smem) + (size_t)wid * E;
    if (a.mask && !a.mask[t]) {
        if (lane < k) {
            if (!a.ids_in) a.ids[t * k + lane] = -1;
            a.w[t * k + lane] = 0.0f;
        }
        return;
    }
    float z[NE], m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const int e = lane + 64 * j;
        z[j] = e < E ? load_z<ZD>(a.z, t * E + e) : -INFINITY;
        if (!(z[j] > -INFINITY)) z[j] = -INFINITY;
        m = fmaxf(m, z[j]);
    }
    const bool sigmoid = a.rule.score == MOE_SCORE_SIGMOID;
    double sum = 1.0;
    if (!sigmoid) {
        m = moe::wave_all_max(m);
        sum = 0.0;
#pragma unroll
        for (int j = 0; j < NE; ++j) sum += z[j] > -INFINITY ? soft64(z[j], m) : 0.0;
        sum = moe::wave_all_sum(sum);
    }
    const auto score = [&](float v) {
        double rest;
        return sigmoid ? sigmoid64(v, rest) : soft64(v, m) / sum;
    };
    int pick = -1;
    float zp = -INFINITY;
    if (a.ids_in) {
        if (lane < k) {
            const int e = a.ids_in[t * k + lane];
            if (e >= 0 && e < E) {
                const float v = load_z<ZD>(a.z, t * E + e);
                if (v > -INFINITY) pick = e, zp = v;
            }
        }
    } else {
        double c[NE];  // -inf: not open, or taken
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const int e = lane + 64 * j;
            const float b = e < E && a.bias ? a.bias[e] : 0.0f;
            c[j] = z[j] > -INFINITY && b > -INFINITY ? score(z[j]) + (double)b : -INFINITY;
            if (G > 1 && e < E) row[e] = c[j];
        }
        if (G > 1) {
            __builtin_amdgcn_wave_barrier();
            double best = -INFINITY, second = -INFINITY;
            for (int i = 0; lane < G && i < gs; ++i) {
                const double v = row[lane * gs + i];
                if (v > best) second = best, best = v;
                else if (v > second) second = v;
            }
            if (a.rule.group_top > 1 && second > -INFINITY) best += second;
            int rank = 0;
            for (int g = 0; g < G; ++g) {
                const double o = __shfl(best, g, moe::WAVE);
                rank += o > best || (o == best && g < lane);
            }
            const unsigned long long kept = __ballot(lane < G && rank < a.rule.groups_kept);
#pragma unroll
            for (int j = 0; j < NE; ++j) {
                const int e = lane + 64 * j;
                if (e < E && !((kept >> (e / gs)) & 1)) c[j] = -INFINITY;
            }
        }
        for (int r = 0; r < k; ++r) {
            double bc = -INFINITY;
            float bz = -INFINITY;
            int be = E;
#pragma unroll
            for (int j = 0; j < NE; ++j)
                if (c[j] > bc || (c[j] == bc && c[j] > -INFINITY && z[j] > bz)) bc = c[j], bz = z[j], be = lane + 64 * j;
#pragma unroll
            for (int s = 32; s >= 1; s >>= 1) {
                const double oc = __shfl_xor(bc, s, moe::WAVE);
                const float oz = __shfl_xor(bz, s, moe::WAVE);
                const int oe = __shfl_xor(be, s, moe::WAVE);
                if (oc > bc || (oc == bc && (oz > bz || (oz == bz && oe < be)))) bc = oc, bz = oz, be = oe;
            }
            if (!(bc > -INFINITY)) break;
            if (lane == r) pick = be, zp = bz;
#pragma unroll
            for (int j = 0; j < NE; ++j)
                if (lane + 64 * j == be) c[j] = -INFINITY;
        }
        if (lane < k) a.ids[t * k + lane] = pick;
    }
    const double s = a.rule.renorm ? share64(a.rule.score, zp, pick >= 0) : pick >= 0 ? score(zp) : 0.0;
    if (lane < k) a.w[t * k + lane] = (float)((double)a.rule.scale * s);
}

struct SelBwdArgs {
    const void* z;
    const int32_t* ids;
    const float* dw;
    int T, E, k;
    moe_select_rule rule;
    const void* add;
    void* dz;
};

// One wave a token; the picks' parts are gathered in a row of LDS.
template <int ZD>
__global__ void __launch_bounds__(64 * SEL_WAVES) k_select_bwd(SelBwdArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 6) + wid;
    if (t >= a.T) return;
    const int E = a.E, k = a.k;
    float* row = reinterpret_cast<float*>(smem) + (size_t)wid * E;
    const bool sigmoid = a.rule.score == MOE_SCORE_SIGMOID, dense = !sigmoid && !a.rule.renorm;
    int e = -1;
    float zp = -INFINITY;
    double h = 0.0;
    if (lane < k) {
        e = a.ids[t * k + lane];
        if (e >= 0 && e < E) zp = load_z<ZD>(a.z, t * E + e);
        if (zp > -INFINITY) h = (double)a.rule.scale * (double)a.dw[t * k + lane];
    }
    const bool live = zp > -INFINITY;
    float m = -INFINITY;
    double sum = 1.0;
    if (dense) {
        sum = 0.0;
        for (int i = lane; i < E; i += 64) m = fmaxf(m, load_z<ZD>(a.z, t * E + i));
        m = moe::wave_all_max(m);
        for (int i = lane; i < E; i += 64) {
            const float v = load_z<ZD>(a.z, t * E + i);
            sum += v > -INFINITY ? soft64(v, m) : 0.0;
        }
        sum = moe::wave_all_sum(sum);
    }
    double q, rest = 1.0;
    if (a.rule.renorm) q = share64(a.rule.score, zp, live);
    else q = !live ? 0.0 : sigmoid ? 1.0 : soft64(zp, m) / sum;
    if (sigmoid && live) {
        const double s = sigmoid64(zp, rest);
        if (!a.rule.renorm) q = s;
    }
    const double dot = sigmoid && !a.rule.renorm ? 0.0 : moe::wave_all_sum(live ? h * q : 0.0);
    // what this pick adds at its expert, the parts of an expert picked more than once together
    const double part = !live ? 0.0 : dense ? h * q : q * rest * (h - dot);
    double mine = 0.0;
    for (int i = 0; i < k; ++i) {
        const int o = __shfl(e, i, moe::WAVE);
        const double p = __shfl(part, i, moe::WAVE);
        if (o == e) mine += p;
    }
    for (int i = lane; i < E; i += 64) {
        double d = 0.0;
        if (dense) {
            const float v = load_z<ZD>(a.z, t * E + i);
            d = v > -INFINITY ? -dot * soft64(v, m) / sum : 0.0;
        }
        row[i] = (float)d;
    }
    __builtin_amdgcn_wave_barrier();
    if (live) row[e] = (float)(dense ? mine - dot * q : mine);
    __builtin_amdgcn_wave_barrier();
    for (int i = lane; i < E; i += 64) {
        const float d = row[i] + (a.add ? load_z<ZD>(a.add, t * E + i) : 0.0f);
        if constexpr (ZD == MOE_X_F32) reinterpret_cast<float*>(a.dz)[t * E + i] = d;
        else reinterpret_cast<__bf16*>(a.dz)[t * E + i] = (__bf16)d;
    }
}

// One workgroup a layer.  Whole numbers: C - n c is exact.
__global__ void __launch_bounds__(256) k_bias_balance(const int32_t* __restrict__ counts, const float* bias, int E,
                                                      float rate, float* out) {
    __shared__ long long s_sum[4], s_n[4];
    const int64_t at = (int64_t)blockIdx.x * E;
    long long sum = 0, n = 0;
    for (int e = threadIdx.x; e < E; e += 256)
        if (bias[at + e] > -INFINITY) sum += counts[at + e], ++n;
    sum = moe::wave_all_sum(sum);
    n = moe::wave_all_sum(n);
    if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum, s_n[threadIdx.x >> 6] = n;
    __syncthreads();
    sum = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
    n = s_n[0] + s_n[1] + s_n[2] + s_n[3];
    for (int e = threadIdx.x; e < E; e += 256) {
        const float b = bias[at + e];
        const long long d = sum - n * counts[at + e];
        out[at + e] = !(b > -INFINITY) || d == 0 ? b : d > 0 ? b + rate : b - rate;
    }
}

int check_rule(const char* who, int z_dtype, int T, int E, int k, const moe_select_rule* rule) {
    MOE_REQUIRE(rule, MOE_E_ARG, "%s: rule must be non-NULL", who);
    MOE_REQUIRE(T >= 0 && E >= 1 && k >= 1, MOE_E_ARG, "%s: T=%d E=%d k=%d", who, T, E, k);
    MOE_REQUIRE(rule->score == MOE_SCORE_SOFTMAX || rule->score == MOE_SCORE_SIGMOID, MOE_E_ARG, "%s: score %d", who,
                rule->score);
    MOE_REQUIRE(rule->groups >= 1 && rule->groups_kept >= 1 && rule->groups_kept <= rule->groups, MOE_E_ARG,
                "%s: %d of %d groups", who, rule->groups_kept, rule->groups);
    MOE_REQUIRE(rule->group_top == 1 || rule->group_top == 2, MOE_E_ARG, "%s: group_top=%d must be 1 or 2", who,
                rule->group_top);
    MOE_REQUIRE(rule->scale - rule->scale == 0.0f, MOE_E_ARG, "%s: scale=%g must be finite", who, (double)rule->scale);
    MOE_REQUIRE(z_dtype == MOE_X_F32 || z_dtype == MOE_X_BF16, MOE_E_DTYPE, "%s: logit format %d", who, z_dtype);
    MOE_REQUIRE(E <= MOE_MAX_E && k <= MOE_MAX_K && T <= MOE_SELECT_MAX_T, MOE_E_SHAPE,
                "%s: T=%d E=%d k=%d beyond the limits", who, T, E, k);
    MOE_REQUIRE(rule->groups <= MOE_SELECT_MAX_GROUPS && E % rule->groups == 0, MOE_E_SHAPE,
                "%s: E=%d experts in %d groups", who, E, rule->groups);
    MOE_REQUIRE(k <= E / rule->groups * rule->groups_kept, MOE_E_SHAPE,
                "%s: k=%d picks from %d groups of %d experts", who, k, rule->groups_kept, E / rule->groups);
    return MOE_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Waves of a workgroup whose tokens each take `bytes` of LDS.
int sel_waves(size_t bytes) { return bytes <= 8192 ? SEL_WAVES : 1; }

}  // namespace

extern "C" {

int moe_route_select(const void* z, int z_dtype, const float* bias, const uint8_t* mask, const int32_t* ids_in, int T,
                     int E, int k, const moe_select_rule* rule, int32_t* ids, float* w, hipStream_t stream) {
    if (int rc = check_rule("moe_route_select", z_dtype, T, E, k, rule)) return rc;
    MOE_REQUIRE(T == 0 || (z && w && (ids || ids_in)), MOE_E_ARG,
                "moe_route_select: z, w and ids (or ids_in) must be non-NULL");
    MOE_REQUIRE(moe_aligned16(z) && aligned4(ids) && aligned4(ids_in) && aligned4(w) && aligned4(bias), MOE_E_ALIGN,
                "moe_route_select: z must start on 16 bytes; ids, ids_in, w and bias on 4");
    if (T == 0) return moe_ok();
    const SelArgs a{z, bias, mask, ids_in, T, E, k, *rule, ids, w};
    const size_t bytes = rule->groups > 1 ? (size_t)8 * E : 0;
    const int waves = sel_waves(bytes);
    const auto go = [&](auto zd, auto ne) {
        hipLaunchKernelGGL((k_select<decltype(zd)::value, decltype(ne)::value>), dim3((T + waves - 1) / waves),
                           dim3(64 * waves), waves * bytes, stream, a);
    };
    const auto by_experts = [&](auto zd) {
        if (E <= 128) go(zd, std::integral_constant<int, 2>{});
        else if (E <= 512) go(zd, std::integral_constant<int, 8>{});
        else if (E <= 1024) go(zd, std::integral_constant<int, 16>{});
        else go(zd, std::integral_constant<int, 64>{});
    };
    if (z_dtype == MOE_X_F32) by_experts(std::integral_constant<int, MOE_X_F32>{});
    else by_experts(std::integral_constant<int, MOE_X_BF16>{});
    return moe_check_launch("moe_route_select");
}

int moe_route_select_bwd(const void* z, int z_dtype, const int32_t* ids, const float* dw, int T, int E, int k,
                         const moe_select_rule* rule, const void* dz_add, void* dz, hipStream_t stream) {
    if (int rc = check_rule("moe_route_select_bwd", z_dtype, T, E, k, rule)) return rc;
    MOE_REQUIRE(T == 0 || (z && ids && dw && dz), MOE_E_ARG, "moe_route_select_bwd: z, ids, dw and dz must be non-NULL");
    MOE_REQUIRE(moe_aligned16(z) && moe_aligned16(dz_add) && moe_aligned16(dz) && aligned4(ids) && aligned4(dw),
                MOE_E_ALIGN, "moe_route_select_bwd: z, dz_add and dz must start on 16 bytes; ids and dw on 4");
    if (T == 0) return moe_ok();
    const SelBwdArgs a{z, ids, dw, T, E, k, *rule, dz_add, dz};
    const size_t bytes = (size_t)4 * E;
    const int waves = sel_waves(bytes);
    const dim3 grid((T + waves - 1) / waves), block(64 * waves);
    if (z_dtype == MOE_X_F32) hipLaunchKernelGGL(k_select_bwd<MOE_X_F32>, grid, block, waves * bytes, stream, a);
    else hipLaunchKernelGGL(k_select_bwd<MOE_X_BF16>, grid, block, waves * bytes, stream, a);
    return moe_check_launch("moe_route_select_bwd");
}

int moe_bias_balance(const int32_t* counts, const float* bias, int L, int E, float rate, float* bias_out,
                     hipStream_t stream) {
    MOE_REQUIRE(counts && bias && bias_out, MOE_E_ARG, "moe_bias_balance: counts, bias and bias_out must be non-NULL");
    MOE_REQUIRE(L >= 1 && E >= 1, MOE_E_ARG, "moe_bias_balance: L=%d and E=%d must be >= 1", L, E);
    MOE_REQUIRE(rate - rate == 0.0f && rate >= 0.0f, MOE_E_ARG, "moe_bias_balance: rate=%g must be finite and >= 0",
                (double)rate);
    MOE_REQUIRE(E <= MOE_MAX_E && L <= 65535, MOE_E_SHAPE, "moe_bias_balance: L=%d E=%d beyond the limits", L, E);
    hipLaunchKernelGGL(k_bias_balance, dim3(L), dim3(256), 0, stream, counts, bias, E, rate, bias_out);
    return moe_check_launch("moe_bias_balance");
}

}  // extern "C"
