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
// in five lines", grades its bias by.  The bias table ranks the experts by it, and
// experts nearly as bright would change places with fp32's rounding, so the softmax
// and its sums run in double, in a fixed order.  One wave takes one token at a
// time and keeps its experts' running sums in registers (lane l holds experts
// l, l + 64, ...).
#include <math.h>

#include <type_traits>

#include "common.hpp"
#include "exp64.hpp"
#include "wave.hpp"

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int BAL_MAX_BLOCKS = 512;  // of the row kernel: two a CU
// Batches of up to this many tokens: one workgroup does it all, in one launch.  One
// and many workgroups, us, 4 picks, fp32: 64 experts 16 tokens 6.0 and 8.9, 64 tokens
// 8.0 and 9.0, 128 tokens 10.7 and 9.7; 256 experts 16 tokens 7.4 and 10.8, 128 tokens
// 16.2 and 10.9; 1024 experts 16 tokens 12.6 and 14.5, 128 tokens 49 and 15; 4096
// experts 4 tokens 25 and 34, 128 tokens 202 and 35.  The two cross near 100 tokens of
// 64 experts, 55 of 256, 35 of 512, 22 of 1024 and 10 of 4096: this rule, of tokens
// alone, does not follow that.
constexpr int BAL_ONE = 128;
constexpr int SUM_E = 16;            // experts of a workgroup of the second pass
constexpr int SUM_THREADS = 1024;

// Waves of a row-kernel workgroup: sixteen where it is the only one, eight, or
// four where a lane's experts fill its registers.
constexpr int bal_waves(int NE, bool one) { return NE > 8 ? 4 : one ? 16 : 8; }

// Lane l holds experts (l + 64 j) * VEC + v of a row in v[j * VEC + v]: single
// fp32 logits (no lane idles on a row of, say, 288 but in its last group), or
// bf16 pairs.  Past the row: -inf.
template <int ZD, int VEC, int NE>
__device__ __forceinline__ void load_row(const void* z, int64_t t, int E, int lane, float (&v)[NE]) {
#pragma unroll
    for (int j = 0; j < NE / VEC; ++j) {
        const int e = (lane + 64 * j) * VEC;
        const int64_t at = t * E + e;
        if constexpr (ZD == MOE_X_F32) {
            v[j] = e < E ? reinterpret_cast<const float*>(z)[at] : -INFINITY;
        } else if constexpr (VEC == 1) {
            v[j] = e < E ? moe::bf16_to_f32(reinterpret_cast<const uint16_t*>(z)[at]) : -INFINITY;
        } else {
            const uint32_t p = e < E ? *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint16_t*>(z) + at)
                                     : 0xFF80FF80u;
            v[2 * j] = moe::bf16_lo(p);
            v[2 * j + 1] = moe::bf16_hi(p);
        }
    }
}

// Workspace: per block of the row kernel the sums of p per expert, the sum of
// lse^2, the picks per expert and the counted tokens; per block of the second
// pass its part of sum_e c_e P_e and of sum_e c_e, and how many are done.
struct BalWs {
    double* share;   // [blocks][E]
    double* lse2;    // [blocks]
    double* dot;     // [parts]
    int32_t* picks;  // [blocks][E]
    int32_t* toks;   // [blocks]
    int32_t* sum;    // [parts]
    int32_t* done;
};

inline int bal_blocks(int T, int waves) {
    const int64_t b = ((int64_t)T + waves - 1) / waves;
    return T <= BAL_ONE ? 1 : b < BAL_MAX_BLOCKS ? (int)b : BAL_MAX_BLOCKS;
}

inline int bal_parts(int E) { return (E + SUM_E - 1) / SUM_E; }

inline size_t bal_bytes(int blocks, int E) {
    return (size_t)blocks * (12 * (size_t)E + 12) + (size_t)bal_parts(E) * 12 + 4;
}

inline BalWs bal_ws(void* ws, int blocks, int E) {
    BalWs w;
    w.share = reinterpret_cast<double*>(ws);
    w.lse2 = w.share + (size_t)blocks * E;
    w.dot = w.lse2 + blocks;
    w.picks = reinterpret_cast<int32_t*>(w.dot + bal_parts(E));
    w.toks = w.picks + (size_t)blocks * E;
    w.sum = w.toks + blocks;
    w.done = w.sum + bal_parts(E);
    return w;
}

// Rows of per-expert sums in LDS: one a wave of half the workgroup, or one.
constexpr int share_rows(int NE, bool one) { return NE <= 8 ? bal_waves(NE, one) / 2 : 1; }

struct BalOut {
    int32_t* counts;
    int32_t* totals;
    double* share;
    float* loss;
};

__device__ __forceinline__ void write_totals(const BalOut& o, int E, int n, int picks, double dot, double lse2) {
    o.totals[0] = n;
    o.totals[1] = picks;
    o.loss[0] = picks > 0 && n > 0 ? (float)(E * dot / (double)picks) : 0.0f;
    o.loss[1] = n > 0 ? (float)(lse2 / n) : 0.0f;
}

// A wave takes `per` tokens in a row (the first `more` waves one besides), 64 at
// a time: one after the other for the softmax (all lanes on one token), then
// side by side (a lane a token) for the logarithm, lse and the picks.  ONE: a
// single workgroup, which also writes the outputs (64 x 128: 8.8 us).
// Bound by the vector unit: about 40 instructions an exponential in double with
// its share of the token's reductions (65537 x 512 bf16: 52 us, the unit busy
// for four fifths of it; 16384 x 288 fp32: 15 us).
template <int ZD, int VEC, int NE, bool ONE>
__global__ void __launch_bounds__(64 * bal_waves(NE, ONE)) k_balance(const void* __restrict__ z,
                                                                     const int32_t* __restrict__ ids,
                                                                     const uint8_t* __restrict__ mask, int T, int E,
                                                                     int k, int per, int more,
                                                                     float* __restrict__ lse, BalWs ws, BalOut o) {
    constexpr int NW = bal_waves(NE, ONE);
    extern __shared__ __align__(16) unsigned char smem[];
    double* s_share = reinterpret_cast<double*>(smem);            // [share_rows(NE, ONE)][E]
    double* s_lse2 = s_share + (size_t)share_rows(NE, ONE) * E;   // [NW]
    int32_t* s_picks = reinterpret_cast<int32_t*>(s_lse2 + NW);    // [E]
    int32_t* s_toks = s_picks + E;                                // [NW]
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    for (int e = threadIdx.x; e < E; e += 64 * NW) s_picks[e] = 0;
    __syncthreads();
    double acc[NE] = {}, lse2 = 0.0;
    int toks = 0;
    const int w0 = (int)blockIdx.x * NW + wid;
    const int64_t first = (int64_t)w0 * per + (w0 < more ? w0 : more);
    const int64_t end = first + per + (w0 < more);
    for (int64_t t0 = first; t0 < end; t0 += 64) {
        const int n = end - t0 < 64 ? (int)(end - t0) : 64;
        const unsigned long long todo = __ballot(lane < n && (!mask || mask[t0 + lane]));
        float v[NE], my_m = 0.0f;
        double my_sum = 0.0;  // of token t0 + lane; 0: left out
        if (todo & 1) load_row<ZD, VEC, NE>(z, t0, E, lane, v);
        for (int i = 0; i < n; ++i) {
            float cur[NE], m = -INFINITY;
#pragma unroll
            for (int j = 0; j < NE; ++j) cur[j] = v[j];
            // the next token's logits, while this one's are summed
            if (i + 1 < n && (todo >> (i + 1)) & 1) load_row<ZD, VEC, NE>(z, t0 + i + 1, E, lane, v);
            if (!((todo >> i) & 1)) continue;
#pragma unroll
            for (int j = 0; j < NE; ++j) m = fmaxf(m, cur[j]);
            m = moe::wave_all_max(m);  // NaN loses every comparison: looked for where nothing else is left
            if (m == -INFINITY) {
                bool nan = false;
#pragma unroll
                for (int j = 0; j < NE; ++j) nan |= cur[j] != cur[j];
                if (!__any(nan)) continue;
            }
            double p[NE], sum = 0.0;
#pragma unroll
            for (int j = 0; j < NE; ++j) sum += p[j] = moe::exp64((double)cur[j] - (double)m);
            sum = moe::wave_all_sum(sum);
            // 1 / sum: the hardware's estimate and two Newton steps (sum lies in [1, E])
            double r = __builtin_amdgcn_rcp(sum);
            r = fma(fma(-sum, r, 1.0), r, r);
            r = fma(fma(-sum, r, 1.0), r, r);
#pragma unroll
            for (int j = 0; j < NE; ++j) acc[j] = fma(p[j], r, acc[j]);
            if (lane == i) my_m = m, my_sum = sum;
        }
        const bool live = my_sum != 0.0;
        const double l = live ? (double)my_m + log(my_sum) : 0.0;
        if (lane < n) lse[t0 + lane] = (float)l;
        lse2 += l * l;
        toks += live;
        const unsigned long long counted = __ballot(live);
        for (int i = lane; i < n * k; i += 64) {
            const int e = ids[t0 * k + i];
            if (((counted >> (i / k)) & 1) && e >= 0 && e < E) atomicAdd(&s_picks[e], 1);
        }
    }
    lse2 = moe::wave_all_sum(lse2);
    toks = moe::wave_all_sum(toks);
    if (lane == 0) s_lse2[wid] = lse2, s_toks[wid] = toks;
    // the waves' sums, in an order of their own: halves, quarters, ... (or one
    // after the other where LDS has room for one row)
    const auto at = [&](int j) { return (lane + 64 * (j / VEC)) * VEC + j % VEC; };
    if constexpr (share_rows(NE, ONE) > 1) {
#pragma unroll
        for (int h = NW / 2; h >= 1; h >>= 1) {
            if (wid >= h && wid < 2 * h) {
#pragma unroll
                for (int j = 0; j < NE; ++j)
                    if (at(j) < E) s_share[(size_t)(wid - h) * E + at(j)] = acc[j];
            }
            __syncthreads();
            if (wid < h) {
#pragma unroll
                for (int j = 0; j < NE; ++j)
                    if (at(j) < E) acc[j] += s_share[(size_t)wid * E + at(j)];
            }
            __syncthreads();
        }
        if (wid == 0) {
#pragma unroll
            for (int j = 0; j < NE; ++j)
                if (at(j) < E) s_share[at(j)] = acc[j];
        }
        __syncthreads();
    } else {
        for (int w = 0; w < NW; ++w) {
            if (wid == w) {
#pragma unroll
                for (int j = 0; j < NE; ++j)
                    if (at(j) < E) s_share[at(j)] = w ? s_share[at(j)] + acc[j] : acc[j];
            }
            __syncthreads();
        }
    }
    double l2 = 0.0;
    int n = 0;
    for (int w = 0; w < NW; ++w) l2 += s_lse2[w], n += s_toks[w];
    if constexpr (!ONE) {
        for (int e = threadIdx.x; e < E; e += 64 * NW) {
            ws.share[(int64_t)blockIdx.x * E + e] = s_share[e];
            ws.picks[(int64_t)blockIdx.x * E + e] = s_picks[e];
        }
        if (threadIdx.x == 0) ws.lse2[blockIdx.x] = l2, ws.toks[blockIdx.x] = n;
        if (blockIdx.x == 0 && threadIdx.x == 0) *ws.done = 0;
    } else {
        double dot = 0.0;
        int picks = 0;
        for (int e = threadIdx.x; e < E; e += 64 * NW) {
            const double s = n > 0 ? s_share[e] / n : 0.0;
            o.share[e] = s;
            o.counts[e] = s_picks[e];
            dot += s * s_picks[e];
            picks += s_picks[e];
        }
        dot = moe::wave_all_sum(dot);
        picks = moe::wave_all_sum(picks);
        __syncthreads();  // every thread has read s_lse2 and s_toks
        if (lane == 0) s_lse2[wid] = dot, s_toks[wid] = picks;
        __syncthreads();
        if (threadIdx.x == 0) {
            dot = 0.0;
            picks = 0;
            for (int w = 0; w < NW; ++w) dot += s_lse2[w], picks += s_toks[w];
            write_totals(o, E, n, picks, dot, l2);
        }
    }
}

// Second pass: SUM_E experts a workgroup, 64 groups of threads each adding up
// every 64th block, then the groups in order.  The last workgroup to end (its
// count says so) writes the losses, from every part in the parts' order.
// 512 blocks' rows of 288 and 512 experts: 6.6 and 7.1 us (8 experts a workgroup
// 6.7 and 7.8 us), most of it the launch, one load's and one atomic's way.
__global__ void __launch_bounds__(SUM_THREADS) k_balance_sum(BalWs ws, int blocks, int E, BalOut o) {
    __shared__ double s_share[SUM_THREADS];
    __shared__ int s_picks[SUM_THREADS], s_n[SUM_THREADS / 64];
    const int tid = threadIdx.x, e = blockIdx.x * SUM_E + tid % SUM_E;
    int n = 0;
    for (int b = tid; b < blocks; b += SUM_THREADS) n += ws.toks[b];
    n = moe::wave_all_sum(n);
    if ((tid & 63) == 0) s_n[tid >> 6] = n;
    double s = 0.0;
    int c = 0;
    if (e < E)
#pragma unroll 8
        for (int b = tid / SUM_E; b < blocks; b += SUM_THREADS / SUM_E)
            s += ws.share[(int64_t)b * E + e], c += ws.picks[(int64_t)b * E + e];
    s_share[tid] = s;
    s_picks[tid] = c;
    __syncthreads();
    if (tid >= 64) return;
    n = 0;
    for (int w = 0; w < SUM_THREADS / 64; ++w) n += s_n[w];
    // a wave holds four of the 64 groups: each lane adds every fourth, then the four
    s = 0.0;
    c = 0;
    for (int g = tid; g < SUM_THREADS; g += 64) s += s_share[g], c += s_picks[g];
    s += __shfl_xor(s, 16, moe::WAVE);
    s += __shfl_xor(s, 32, moe::WAVE);
    c += __shfl_xor(c, 16, moe::WAVE);
    c += __shfl_xor(c, 32, moe::WAVE);
    s = n > 0 ? s / n : 0.0;
    const bool mine = tid < SUM_E && e < E;
    if (mine) o.share[e] = s, o.counts[e] = c;
    const double dot = moe::wave_sum(mine ? s * c : 0.0);
    const int picks = moe::wave_sum(mine ? c : 0);
    int last = 0;
    if (tid == 0) {
        ws.dot[blockIdx.x] = dot, ws.sum[blockIdx.x] = picks;
        last = __hip_atomic_fetch_add(ws.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
    }
    if (!__shfl(last, 0, moe::WAVE)) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    double all = 0.0, l2 = 0.0;
    int of = 0;
    for (int p = tid; p < (int)gridDim.x; p += 64) all += ws.dot[p], of += ws.sum[p];
#pragma unroll 8
    for (int b = tid; b < blocks; b += 64) l2 += ws.lse2[b];
    all = moe::wave_sum(all);
    l2 = moe::wave_sum(l2);
    of = moe::wave_sum(of);
    if (tid == 0) write_totals(o, E, n, of, all, l2);
}

// p is exp(z - lse) over its own sum: lse is rounded to fp32, and without the
// division that rounding, 2^-24 |lse|, would be in every p (at logits around 10^4
// the fourth digit), and p would not add up to 1.  Where the sum shows that lse is
// further off than a factor of 2, the row's largest logit takes its place.  f is
// taken less its mean 1/E, as whole numbers over whole numbers: the subtraction
// f_e - sum f p of nearly equal numbers (a balanced router) then costs no digits,
// since sum p = 1.  The differences are rounded once, the exponentials, sums of
// positive terms and products are good to fp32's last bits, and dz is an fp32
// number or shorter: fp32 is enough.
// Bound by the vector unit: 65537 x 512 bf16 in 33 us, 4.1 TB/s of z and dz, 235
// instructions a token, the unit busy throughout (31.5 us without the sum).
template <int ZD, int VEC, int NE>
__global__ void __launch_bounds__(256) k_balance_bwd(const void* z, const float* __restrict__ lse,
                                                     const uint8_t* __restrict__ mask,
                                                     const int32_t* __restrict__ counts,
                                                     const int32_t* __restrict__ totals,
                                                     const float* __restrict__ dloss, int T, int E, void* dz) {
    constexpr int NW = 4;
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const int n = totals[0], picks = totals[1];
    const double rn = n > 0 ? 1.0 / n : 0.0;
    const double gb = picks > 0 ? (double)dloss[0] * rn / picks : 0.0;
    const float gz = (float)(2.0 * (double)dloss[1] * rn);
    float f[NE];  // g_b E (f_e - 1/E) / n
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const int e = (lane + 64 * (j / VEC)) * VEC + j % VEC;
        f[j] = e < E ? (float)((double)((int64_t)counts[e] * E - picks) * gb) : 0.0f;
    }
    for (int64_t t = (int64_t)blockIdx.x * NW + wid; t < T; t += (int64_t)gridDim.x * NW) {
        const auto put = [&](const auto& d) {
#pragma unroll
            for (int j = 0; j < NE / VEC; ++j) {
                const int e = (lane + 64 * j) * VEC;
                if (e >= E) continue;
                if constexpr (ZD == MOE_X_F32) {
                    reinterpret_cast<float*>(dz)[t * E + e] = d(j);
                } else if constexpr (VEC == 1) {
                    reinterpret_cast<__bf16*>(dz)[t * E + e] = (__bf16)d(j);
                } else {
                    reinterpret_cast<bf16x2*>(dz)[(t * E + e) / 2] = bf16x2{(__bf16)d(2 * j), (__bf16)d(2 * j + 1)};
                }
            }
        };
        if (mask && !mask[t]) {
            put([](int) { return 0.0f; });
            continue;
        }
        float p[NE], sum, dot;  // p: before the division
        const auto softmax = [&](float at) {
            sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int j = 0; j < NE; ++j) {
                p[j] = expf(p[j] - at);
                sum += p[j];
                dot = fmaf(p[j], f[j], dot);
            }
            sum = moe::wave_all_sum(sum);
            dot = moe::wave_all_sum(dot);
        };
        const float l = lse[t];
        load_row<ZD, VEC, NE>(z, t, E, lane, p);
        softmax(l);
        if (!(sum > 0.5f && sum < 2.0f)) {
            load_row<ZD, VEC, NE>(z, t, E, lane, p);
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < NE; ++j) m = fmaxf(m, p[j]);
            m = moe::wave_all_max(m);
            softmax(m == -INFINITY ? 0.0f : m);  // nothing above -inf: all 0 (a NaN stays one)
            if (sum == 0.0f) {
                put([](int) { return 0.0f; });
                continue;
            }
        }
        const float r = __builtin_amdgcn_rcpf(sum);  // to the last bit
        const float c = (gz * l - dot * r) * r;
        put([&](int i) { return p[i] * fmaf(f[i], r, c); });
    }
}

// Calls go with the number of experts a lane holds: one number for each group
// of 64 (64 pairs) up to eight, then 16, 32, 64.
template <int VEC, typename Go>
void by_experts(int E, const Go& go) {
    const int j = (E + 64 * VEC - 1) / (64 * VEC);
    if (j <= 1) go(std::integral_constant<int, VEC>{});
    else if (j <= 2) go(std::integral_constant<int, 2 * VEC>{});
    else if (j <= 3) go(std::integral_constant<int, 3 * VEC>{});
    else if (j <= 4) go(std::integral_constant<int, 4 * VEC>{});
    else if (j * VEC <= 6 && VEC == 1) go(std::integral_constant<int, 6>{});
    else if (j * VEC <= 8) go(std::integral_constant<int, 8>{});
    else if (j * VEC <= 16) go(std::integral_constant<int, 16>{});
    else if (j * VEC <= 32) go(std::integral_constant<int, 32>{});
    else go(std::integral_constant<int, 64>{});
}

// Format and pairs: bf16 rows of an even length are read in pairs.
template <typename Go>
void by_format(int z_dtype, int E, const Go& go) {
    using std::integral_constant;
    if (z_dtype == MOE_X_F32)
        by_experts<1>(E, [&](auto ne) { go(integral_constant<int, MOE_X_F32>{}, integral_constant<int, 1>{}, ne); });
    else if (E % 2)
        by_experts<1>(E, [&](auto ne) { go(integral_constant<int, MOE_X_BF16>{}, integral_constant<int, 1>{}, ne); });
    else
        by_experts<2>(E, [&](auto ne) { go(integral_constant<int, MOE_X_BF16>{}, integral_constant<int, 2>{}, ne); });
}

}  // namespace

extern "C" {

size_t moe_balance_workspace_bytes(int T, int E) {
    if (T < 0 || T > MOE_BALANCE_MAX_T || E < 1 || E > MOE_MAX_E) return 0;
    return (bal_bytes(bal_blocks(T, 4), E) + 15) & ~(size_t)15;
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
    const BalOut o{counts, totals, share, loss};
    int blocks = 0;
    BalWs w{};
    by_format(z_dtype, E, [&](auto zd, auto vec, auto ne) {
        constexpr int ZD = decltype(zd)::value, VEC = decltype(vec)::value, NE = decltype(ne)::value;
        const auto launch = [&](auto one) {
            constexpr bool ONE = decltype(one)::value;
            constexpr int NW = bal_waves(NE, ONE);
            blocks = ONE ? 1 : bal_blocks(T, NW);
            w = bal_ws(ws, blocks, E);
            const int waves = blocks * NW;
            const size_t lds = (size_t)E * (8 * share_rows(NE, ONE) + 4) + 12 * NW;
            hipLaunchKernelGGL((k_balance<ZD, VEC, NE, ONE>), dim3(blocks), dim3(64 * NW), lds, stream, z, ids, mask, T,
                               E, k, T / waves, T % waves, lse, w, o);
        };
        if (T <= BAL_ONE) launch(std::true_type{});
        else launch(std::false_type{});
    });
    if (int rc = moe_check_launch("moe_balance_loss")) return rc;
    if (T <= BAL_ONE) return moe_ok();
    hipLaunchKernelGGL(k_balance_sum, dim3(bal_parts(E)), dim3(SUM_THREADS), 0, stream, w, blocks, E, o);
    return moe_check_launch("moe_balance_loss/sum");
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
    const int blocks = (T + 3) / 4 < 2048 ? (T + 3) / 4 : 2048;
    by_format(z_dtype, E, [&](auto zd, auto vec, auto ne) {
        hipLaunchKernelGGL((k_balance_bwd<decltype(zd)::value, decltype(vec)::value, decltype(ne)::value>),
                           dim3(blocks), dim3(256), 0, stream, z, lse, mask, counts, totals, dloss, T, E, dz);
    });
    return moe_check_launch("moe_balance_loss_bwd");
}

}  // extern "C"
