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

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int SEL_WAVES = 4;
constexpr int CAND = 64;  // candidates of a token: one a lane

struct SelArgs {
    const void* z;
    const float* bias;
    const uint8_t* mask;
    const int32_t* ids_in;
    int T, E, k;
    moe_select_rule rule;
    int32_t* ids;
    float* w;
    int batch;  // tokens that a wave takes, one after the other
    int seg;    // lanes of a token's weights: 8, 16 or 32
};

template <int ZD>
__device__ __forceinline__ float load_z(const void* z, int64_t i) {
    if constexpr (ZD == MOE_X_F32) return reinterpret_cast<const float*>(z)[i];
    else return moe::bf16_to_f32(reinterpret_cast<const uint16_t*>(z)[i]);
}

// 1 / v to a double's last bits, v in [1, 2^30]: the hardware's estimate and two Newton steps
__device__ __forceinline__ double rcp64(double v) {
    double r = __builtin_amdgcn_rcp(v);
    r = fma(fma(-v, r, 1.0), r, r);
    return fma(fma(-v, r, 1.0), r, r);
}

// s of a sigmoid and 1 - s
__device__ __forceinline__ double sigmoid64(double z, double& rest) {
    const double e = moe::exp64(-fabs(z)), r = rcp64(1.0 + e);
    rest = z >= 0.0 ? e * r : r;
    return z >= 0.0 ? r : e * r;
}

// Softmax terms: exp(z - m), with every +inf counting 1 where m is +inf.
__device__ __forceinline__ double soft64(float z, float m) { return z == m ? 1.0 : moe::exp64((double)z - (double)m); }
__device__ __forceinline__ float soft32(float z, float m) { return z == m ? 1.0f : __builtin_amdgcn_exp2f((z - m) * 1.44269504f); }

// Order-preserving code of a number (no NaN), and back; -0 and +0 share one.
__device__ __forceinline__ uint32_t code_of(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_code(uint32_t c) { return __uint_as_float(c & 0x80000000u ? c ^ 0x80000000u : ~c); }

// What one lane of a wave wrote to LDS is there for its others.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Reduction over segments of 8, 16 or 32 lanes.
template <typename T, typename Op>
__device__ __forceinline__ T seg_all(T v, int seg, Op op) {
    v = op(v, moe::dpp_of<moe::DPP_XOR1>(v));
    v = op(v, moe::dpp_of<moe::DPP_XOR2>(v));
    v = op(v, moe::dpp_of<moe::DPP_HALF_MIRROR>(v));
    if (seg > 8) v = op(v, moe::dpp_of<moe::DPP_MIRROR>(v));
    if (seg > 16) {
        T x, y;
        moe::row_pair<false>(v, x, y);
        v = op(x, y);
    }
    return v;
}

// s_i over the sum of s over a token's picks (a segment of lanes; live: a pick with
// a score), from ratios to the largest pick's score, which neither vanish nor overflow.
__device__ __forceinline__ double share64(int score, float z, bool live, int seg) {
    const float m = seg_all(live ? z : -INFINITY, seg, [](float x, float y) { return fmaxf(x, y); });
    double r = 0.0;
    if (live) {
        r = soft64(score == MOE_SCORE_SIGMOID ? fminf(z, 0.0f) : z, score == MOE_SCORE_SIGMOID ? fminf(m, 0.0f) : m);
        if (score == MOE_SCORE_SIGMOID) r *= (1.0 + moe::exp64(-fabs((double)m))) * rcp64(1.0 + moe::exp64(-fabs((double)z)));
    }
    const double sum = seg_all(r, seg, [](double x, double y) { return x + y; });
    return sum > 0.0 ? r * rcp64(sum) : 0.0;
}

// v of a lane (the same for all)
__device__ __forceinline__ float lane_of(float v, int lane) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ double lane_of(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane) |
                                          ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane) << 32));
}

// LDS of a wave.
struct SelLds {
    double* row;   // [E], 64-bit choices (or, fp32, those of the group stage)
    float2* cand;  // [CAND] logit, id
    double* ord;   // [CAND + 1] choices in order
    float* ordz;   // [CAND + 1] and their logits
    float2* pick;  // [64] logit, id: `batch` tokens by `seg`
};

constexpr size_t SEL_FIXED = CAND * 8 + (CAND + 2) * 8 + (CAND + 2) * 4 + 64 * 8;
__host__ __device__ constexpr size_t sel_lds(int E) { return (((size_t)8 * E + SEL_FIXED) + 15) & ~(size_t)15; }

__device__ __forceinline__ SelLds sel_parts(unsigned char* p, int E) {
    SelLds l;
    l.row = reinterpret_cast<double*>(p);
    l.cand = reinterpret_cast<float2*>(l.row + E);
    l.ord = reinterpret_cast<double*>(l.cand + CAND);
    l.pick = reinterpret_cast<float2*>(l.ord + CAND + 2);
    l.ordz = reinterpret_cast<float*>(l.pick + 64);
    return l;
}

__device__ __forceinline__ float2 packed(float z, int id) { return float2{z, __int_as_float(id)}; }

// Which groups are kept, as bits: every one of the `per` lanes of a group holds
// that group's value.  unsure: values are off by up to err, and that may matter.
template <typename T>
__device__ __forceinline__ unsigned long long keep_groups(T value, T err, int G, int kept, int per, T* sorted, bool& unsure) {
    const int lane = threadIdx.x & 63, g = lane / per;
    int rank = 0;
    for (int o = 0; o < G; ++o) {
        const T v = lane_of(value, o * per);
        rank += v > value || (v == value && o < g);
    }
    const bool leads = lane % per == 0 && g < G && value > (T)-INFINITY;
    unsigned long long b = __ballot(leads && rank < kept);
    unsure = false;
    if (err > 0 && kept < G) {
        if (lane % per == 0 && g < G) sorted[rank] = value;
        wave_sync();
        const T last = sorted[kept - 1], next = sorted[kept];
        const T mid = next > (T)-INFINITY ? next + (T)0.5 * (last - next) : (T)-INFINITY;
        unsure = __any(leads && !(rank < kept ? value - err > mid : value + err < mid));
    }
    if (per == 1) return b;
    unsigned long long out = 0;  // a bit a group
    for (; b; b &= b - 1) out |= 1ull << (__builtin_ctzll(b) / per);
    return out;
}

// The two largest of a group's choices that a lane sees, joined with another's.
template <typename T>
__device__ __forceinline__ void top2(T v, T& best, T& second) {
    second = v > best ? best : v > second ? v : second;
    best = v > best ? v : best;
}

// A group's value: its lanes (per: a power of two, neighbours) go through its row.
// size: the magnitudes of what was added.
template <typename T>
__device__ __forceinline__ T group_value(const T* row, int G, int gs, int per, int top, T& size) {
    const int lane = threadIdx.x & 63, g = lane / per;
    T best = -INFINITY, second = -INFINITY;
    if (g < G)
        for (int i = lane % per; i < gs; i += per) top2(row[g * gs + i], best, second);
    for (int s = 1; s < per; s <<= 1) {
        const T b = __shfl_xor(best, s, moe::WAVE), c = __shfl_xor(second, s, moe::WAVE);
        top2(b, best, second);
        top2(c, best, second);
    }
    const bool two = top > 1 && second > (T)-INFINITY;
    size = two ? fabs(best) + fabs(second) : fabs(best);
    return two ? best + second : best;
}

__device__ __forceinline__ int lanes_per_group(int G) {
    int per = 64;
    while (per * G > 64) per >>= 1;
    return per;
}

// A token's picks with every choice in double, by k rounds: where fp32 does not
// tell the groups apart, or leaves more candidates than lanes (many logits equal,
// or nearly so).  plain: choices are the logits themselves.
template <int ZD>
__device__ __forceinline__ void choose64(const SelArgs& a, int64_t t, bool plain, SelLds l, float2* out) {
    const int lane = threadIdx.x & 63, E = a.E, G = a.rule.groups, gs = E / G;
    const bool sigmoid = a.rule.score == MOE_SCORE_SIGMOID;
    float m = -INFINITY;
    double r = 1.0;
    if (!sigmoid && !plain) {
        for (int e = lane; e < E; e += 64) m = fmaxf(m, load_z<ZD>(a.z, t * E + e));
        m = moe::wave_all_max(m);
        double sum = 0.0;
        for (int e = lane; e < E; e += 64) {
            const float z = load_z<ZD>(a.z, t * E + e);
            sum += z > -INFINITY ? soft64(z, m) : 0.0;
        }
        r = rcp64(moe::wave_all_sum(sum));
    }
    for (int e = lane; e < E; e += 64) {
        const float z = load_z<ZD>(a.z, t * E + e), b = a.bias ? a.bias[e] : 0.0f;
        double c = -INFINITY, rest;
        if (z > -INFINITY && b > -INFINITY) c = plain ? (double)z : (sigmoid ? sigmoid64(z, rest) : soft64(z, m) * r) + (double)b;
        l.row[e] = c;
    }
    wave_sync();
    if (G > 1) {
        const int per = lanes_per_group(G);
        double size;
        bool unsure;
        const double value = group_value<double>(l.row, G, gs, per, a.rule.group_top, size);
        const unsigned long long kept = keep_groups<double>(value, 0.0, G, a.rule.groups_kept, per, l.ord, unsure);
        for (int e = lane; e < E; e += 64)
            if (!((kept >> (e / gs)) & 1)) l.row[e] = -INFINITY;
        wave_sync();
    }
    for (int i = 0; i < a.k; ++i) {
        double bc = -INFINITY;
        float bz = -INFINITY;
        int be = E;
        for (int e = lane; e < E; e += 64) {
            const double c = l.row[e];
            if (c < bc || !(c > -INFINITY)) continue;
            const float z = load_z<ZD>(a.z, t * E + e);
            if (c > bc || z > bz) bc = c, bz = z, be = e;
        }
#pragma unroll
        for (int s = 32; s >= 1; s >>= 1) {
            const double oc = __shfl_xor(bc, s, moe::WAVE);
            const float oz = __shfl_xor(bz, s, moe::WAVE);
            const int oe = __shfl_xor(be, s, moe::WAVE);
            if (oc > bc || (oc == bc && (oz > bz || (oz == bz && oe < be)))) bc = oc, bz = oz, be = oe;
        }
        if (!(bc > -INFINITY)) break;
        if (lane == 0) out[i] = packed(bz, be), l.row[be] = -INFINITY;
        wave_sync();
    }
}

// One wave a token at a time.  Lane l holds experts (l + 64 j) VEC + v.
//
// The k best of E without k rounds: the lanes' largest keys bound the k-th best
// from below (there are k at least as good), by bisection between the smallest
// maximum of 8, 16 or 32 sets of lanes and the largest of all; whatever reaches
// that bound, some k + 4 experts, moves to a lane of its own and is ranked against
// the others.  The keys are the logits, or, where a bias or groups
// makes the scores themselves count (SCORED), fp32 choices with a bound on how far
// they are from the 64-bit ones: candidates are taken twice that below the bound,
// and ranked by 64-bit choices of which there is one a lane.
// The weights of up to eight tokens are then taken side by side.
template <int ZD, int VEC, int NE, bool SCORED>
__global__ void __launch_bounds__(64 * SEL_WAVES) k_select(SelArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const int64_t t0 = ((int64_t)blockIdx.x * (blockDim.x >> 6) + wid) * a.batch;
    if (t0 >= a.T) return;
    const int E = a.E, k = a.k, G = a.rule.groups, gs = E / G, seg = a.seg;
    const int n = a.T - t0 < a.batch ? (int)(a.T - t0) : a.batch;
    const SelLds l = sel_parts(smem + (size_t)wid * sel_lds(E), E);
    const bool sigmoid = a.rule.score == MOE_SCORE_SIGMOID;
    const bool sums = !sigmoid && (SCORED || !a.rule.renorm);  // the softmax over all experts is needed
    const auto at = [&](int j) { return (lane + 64 * (j / VEC)) * VEC + j % VEC; };
    const int mine = lane / seg;  // the token whose weights this lane takes
    float my_m = 0.0f, my_sum = 1.0f;
    l.pick[lane] = packed(-INFINITY, -1);
    wave_sync();
    unsigned long long todo = __ballot(lane < n && (!a.mask || a.mask[t0 + lane]));

    float bias[SCORED ? NE : 1];
    if constexpr (SCORED) {
#pragma unroll
        for (int j = 0; j < NE; ++j) bias[j] = a.bias ? (at(j) < E ? a.bias[at(j)] : -INFINITY) : 0.0f;
    }
    constexpr bool AHEAD = NE <= 16;  // the next token's logits while this one's are looked at
    float zn[NE];
    const auto load = [&](int64_t t) {
#pragma unroll
        for (int j = 0; j < NE / VEC; ++j) {
            const int e = (lane + 64 * j) * VEC;
            const int64_t i = t * E + e;
            if constexpr (VEC == 1) {
                zn[j] = e < E ? load_z<ZD>(a.z, i) : -INFINITY;
            } else {
                const uint32_t p = e < E ? *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint16_t*>(a.z) + i) : 0xFF80FF80u;
                zn[2 * j] = moe::bf16_lo(p);
                zn[2 * j + 1] = moe::bf16_hi(p);
            }
        }
    };
    const bool rows = !a.ids_in || sums;
    if (AHEAD && rows && (todo & 1)) load(t0);
    for (int i = 0; i < n && rows; ++i) {
        const int64_t t = t0 + i;
        float z[NE];
        if (!AHEAD && (todo & 1)) load(t);
#pragma unroll
        for (int j = 0; j < NE; ++j) z[j] = zn[j] > -INFINITY ? zn[j] : -INFINITY;
        if (AHEAD && (todo >> 1) & 1) load(t + 1);
        const bool on = todo & 1;
        todo >>= 1;
        if (!on) continue;

        float m = 0.0f, sum = 1.0f;
        if (sums) {
            m = z[0];
#pragma unroll
            for (int j = 1; j < NE; ++j) m = fmaxf(m, z[j]);
            m = moe::wave_all_max(m);
            if (m == -INFINITY) continue;  // nothing open
        }
        float key[NE];
        if (sums) {
            sum = 0.0f;
#pragma unroll
            for (int j = 0; j < NE; ++j) {
                key[j] = z[j] > -INFINITY ? soft32(z[j], m) : 0.0f;
                sum += key[j];
            }
            sum = moe::wave_all_sum(sum);
            if (mine == i) my_m = m, my_sum = sum;
        }
        if (a.ids_in) continue;
        float slack = 0.0f;  // how far a key may be from its 64-bit choice, but for the rounding of a sum with the bias
        if constexpr (SCORED) {
            if (sigmoid) {
                // |z| s (1 - s) 2^-23 < 2^-25 for the argument, 2^-25 for the exponential, 2^-24 + 2^-23 for sum and quotient
                slack = 0x1p-22f;
#pragma unroll
                for (int j = 0; j < NE; ++j) key[j] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z[j] * -1.44269504f));
            } else {
                // (1.5 ln E + 2 + E / 64 + 6) 2^-23 of a share for the sum, 3 of them for the term; shares are 1 / sum at most
                const float r = __builtin_amdgcn_rcpf(sum);
                slack = (2.0f * __logf((float)E) + (float)E * 0x1p-6f + 16.0f) * 0x1p-23f * r;
#pragma unroll
                for (int j = 0; j < NE; ++j) key[j] *= r;
            }
#pragma unroll
            for (int j = 0; j < NE; ++j) key[j] = z[j] > -INFINITY && bias[j] > -INFINITY ? key[j] + bias[j] : -INFINITY;
        } else {
#pragma unroll
            for (int j = 0; j < NE; ++j) key[j] = z[j];
        }
        float2* out = l.pick + i * seg;
        bool again = false;  // in double from the start
        if (SCORED && G > 1) {
            float* row = reinterpret_cast<float*>(l.row);
#pragma unroll
            for (int j = 0; j < NE; ++j)
                if (at(j) < E) row[at(j)] = key[j];
            wave_sync();
            const int per = lanes_per_group(G);
            float size;
            const float value = group_value<float>(row, G, gs, per, a.rule.group_top, size);
            // a choice is off by the slack and a rounding, a sum of two by a rounding more
            const float err = 2.0f * slack + size * 0x1p-22f;
            const unsigned long long kept = keep_groups<float>(value, err, G, a.rule.groups_kept, per, reinterpret_cast<float*>(l.ord), again);
#pragma unroll
            for (int j = 0; j < NE; ++j)
                if (at(j) < E && !((kept >> (at(j) / gs)) & 1)) key[j] = -INFINITY;
            wave_sync();
        }
        // a bound that k keys reach
        float v = key[0];
#pragma unroll
        for (int j = 1; j < NE; ++j) v = fmaxf(v, key[j]);
        const uint32_t code = code_of(v);
        uint32_t lo, hi;
        {
            const auto up = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
            const auto down = [](uint32_t x, uint32_t y) { return x < y ? x : y; };
            uint32_t c = up(code, moe::dpp_of<moe::DPP_XOR1>(code));
            uint32_t d = c, x, y;
            c = up(c, moe::dpp_of<moe::DPP_XOR2>(c));
            d = k > 16 ? down(d, moe::dpp_of<moe::DPP_XOR2>(d)) : c;
            const uint32_t c8 = up(c, moe::dpp_of<moe::DPP_HALF_MIRROR>(c));
            d = k > 8 ? down(d, moe::dpp_of<moe::DPP_HALF_MIRROR>(d)) : c8;
            c = up(c8, moe::dpp_of<moe::DPP_MIRROR>(c8));
            d = down(d, moe::dpp_of<moe::DPP_MIRROR>(d));
            moe::row_pair<false>(c, x, y);
            c = up(x, y);
            moe::row_pair<false>(d, x, y);
            d = down(x, y);
            moe::row_pair<true>(c, x, y);
            hi = __builtin_amdgcn_readfirstlane((int)up(x, y));
            moe::row_pair<true>(d, x, y);
            lo = __builtin_amdgcn_readfirstlane((int)down(x, y));
        }
        int have = __builtin_popcountll(__ballot(code >= lo));
        for (int it = 0; it < 24 && have > k + 2 && hi - lo > 1; ++it) {
            const uint32_t mid = lo + (hi - lo) / 2;
            const int c = __builtin_popcountll(__ballot(code >= mid));
            if (c >= k) lo = mid, have = c;
            else hi = mid;
        }
        float bound = of_code(lo);
        if constexpr (SCORED) bound = bound < INFINITY ? bound - (2.0f * slack + fabsf(bound) * 0x1p-22f) : bound;
        bound = fmaxf(bound, -3.402823466e38f);  // whatever is open
        int C = 0;
#pragma unroll
        for (int j = 0; j < NE / VEC; ++j) {
            if constexpr (VEC == 1) {
                const bool in = key[j] >= bound;
                const unsigned long long b = __ballot(in);
                if (!b) continue;
                const int p = __builtin_amdgcn_mbcnt_hi((uint32_t)(b >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)b, C));
                if (in && p < CAND) l.cand[p] = packed(z[j], at(j));
                C += __builtin_popcountll(b);
            } else {
                const bool in0 = key[2 * j] >= bound, in1 = key[2 * j + 1] >= bound;
                const unsigned long long b0 = __ballot(in0), b1 = __ballot(in1);
                if (!(b0 | b1)) continue;
                int p = __builtin_amdgcn_mbcnt_hi((uint32_t)(b0 >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)b0, C));
                p = __builtin_amdgcn_mbcnt_hi((uint32_t)(b1 >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)b1, p));
                if (in0 && p < CAND) l.cand[p] = packed(z[2 * j], at(2 * j));
                p += in0;
                if (in1 && p < CAND) l.cand[p] = packed(z[2 * j + 1], at(2 * j + 1));
                C += __builtin_popcountll(b0) + __builtin_popcountll(b1);
            }
        }
        again |= C > CAND;
        wave_sync();
        // candidates in order of their ids, one a lane
        C = C < CAND ? C : CAND;
        const float2 cd = lane < C ? l.cand[lane] : packed(-INFINITY, 0);
        const float zc = cd.x;
        const int id = __float_as_int(cd.y);
        int rank = 0;
        if (!SCORED || !a.bias) {
            for (int j = 0; j < C; ++j) {
                const float o = lane_of(zc, j);
                rank += o > zc || (o == zc && j < lane);
            }
        } else {
            double c = -INFINITY, rest;
            if (lane < C) c = (sigmoid ? sigmoid64(zc, rest) : soft64(zc, m) * rcp64((double)sum)) + (double)a.bias[id];
            for (int j = 0; j < C; ++j) rank += lane_of(c, j) > c;
            if (lane >= C) rank = lane;
            // equal choices share a rank: the logits, then the ids decide
            l.ordz[rank] = __int_as_float(lane);
            wave_sync();
            if (__any(__float_as_int(l.ordz[rank]) != lane)) {
                for (int j = 0; j < C; ++j) {
                    const float o = lane_of(zc, j);
                    if (lane < C) rank += lane_of(c, j) == c && (o > zc || (o == zc && j < lane));
                }
            }
            if (!sigmoid) {
                // the sum of the softmax is an fp32 one: neighbours that a sum as far off as that may order otherwise
                wave_sync();
                l.ord[rank] = c;
                l.ordz[rank] = zc;
                wave_sync();
                const bool near = lane < k && lane + 1 < C && l.ordz[lane] != l.ordz[lane + 1] &&
                                  l.ord[lane] - l.ord[lane + 1] <= (double)slack;
                again |= __any(near);
            }
        }
        if (again) choose64<ZD>(a, t, !SCORED, l, out);
        else if (lane < C && rank < k) out[rank] = cd;
    }
    wave_sync();
    // the weights, a segment of lanes a token
    const int i = mine, r = lane & (seg - 1);
    const bool here = i < n && r < k;
    const float2 p = l.pick[lane];
    float zp = p.x;
    int pick = __float_as_int(p.y);
    if (a.ids_in) {
        pick = -1;
        zp = -INFINITY;
        if (here && (!a.mask || a.mask[t0 + i])) {
            const int e = a.ids_in[(t0 + i) * k + r];
            if (e >= 0 && e < E) {
                zp = load_z<ZD>(a.z, (t0 + i) * E + e);
                if (zp > -INFINITY) pick = e;
            }
        }
    }
    const bool live = pick >= 0;
    double s = 0.0, rest;
    if (a.rule.renorm) s = share64(a.rule.score, zp, live, seg);
    else if (live) s = sigmoid ? sigmoid64(zp, rest) : soft64(zp, my_m) * rcp64((double)my_sum);
    if (here) {
        if (!a.ids_in) a.ids[(t0 + i) * k + r] = pick;
        a.w[(t0 + i) * k + r] = (float)((double)a.rule.scale * s);
    }
}

struct SelBwdArgs {
    const void* z;
    const int32_t* ids;
    const float* dw;
    int T, E, k;
    moe_select_rule rule;
    const void* add;
    void* dz;
    int batch, seg;  // as SelArgs'
};

// One wave a token at a time, its experts as k_select's lie.  The picks of up to
// eight tokens are looked at side by side; what each adds at its expert goes through
// a row of LDS, 0 elsewhere, to the lane that holds the expert.  DENSE: the raw
// softmax, whose gradient reaches every expert:
//   dz_e = p_e (h_e - sum h p), with h the row's
// in fp32: dz is an fp32 number or shorter, p is divided by its own sum, and h_e - sum
// h p loses what the formula loses.
template <int ZD, int VEC, int NE, bool DENSE>
__global__ void __launch_bounds__(64 * SEL_WAVES) k_select_bwd(SelBwdArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const int64_t t0 = ((int64_t)blockIdx.x * SEL_WAVES + wid) * a.batch;
    if (t0 >= a.T) return;
    const int E = a.E, k = a.k, seg = a.seg;
    const int n = a.T - t0 < a.batch ? (int)(a.T - t0) : a.batch;
    float* row = reinterpret_cast<float*>(smem) + (size_t)wid * E;
    const auto load = [&](const void* p, int64_t t, float (&v)[NE], float none) {
#pragma unroll
        for (int j = 0; j < NE / VEC; ++j) {
            const int e = (lane + 64 * j) * VEC;
            const int64_t i = t * E + e;
            if constexpr (VEC == 1) {
                v[j] = e < E ? load_z<ZD>(p, i) : none;
            } else {
                const uint32_t w = e < E ? *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint16_t*>(p) + i) : 0u;
                v[2 * j] = e < E ? moe::bf16_lo(w) : none;
                v[2 * j + 1] = e < E ? moe::bf16_hi(w) : none;
            }
        }
    };
    constexpr bool AHEAD = NE <= 16;  // the next token's rows while this one's are looked at
    float zn[DENSE ? NE : 1], an[NE];
    if (AHEAD) {
        if constexpr (DENSE) load(a.z, t0, zn, -INFINITY);
        if (a.add) load(a.add, t0, an, 0.0f);
    }
    for (int e = lane; e < E; e += 64) row[e] = 0.0f;
    const int mine = lane / seg, r = lane & (seg - 1);
    int e = -1;
    float zp = -INFINITY, part = 0.0f;
    double h = 0.0;
    if (mine < n && r < k) {
        const int64_t i = (t0 + mine) * k + r;
        e = a.ids[i];
        const float d = a.dw[i];
        if (e >= 0 && e < E) zp = load_z<ZD>(a.z, (t0 + mine) * E + e);
        if (zp > -INFINITY) h = (double)a.rule.scale * (double)d;
        else e = -1;
    }
    const bool live = e >= 0;
    if constexpr (DENSE) {
        part = (float)h;
    } else {
        const bool sigmoid = a.rule.score == MOE_SCORE_SIGMOID;
        double q = 1.0, rest = 1.0, dot = 0.0;
        if (sigmoid) q = sigmoid64(live ? zp : 0.0, rest);
        if (a.rule.renorm) {
            q = share64(a.rule.score, zp, live, seg);
            dot = seg_all(live ? h * q : 0.0, seg, [](double x, double y) { return x + y; });
        }
        if (live) part = (float)(q * rest * (h - dot));
    }
    // the parts of an expert picked more than once, together
    float sum = 0.0f;
    for (int o = 0; o < k; ++o) {
        const int oe = __shfl(e, mine * seg + o, moe::WAVE);
        const float op = __shfl(part, mine * seg + o, moe::WAVE);
        sum += oe == e ? op : 0.0f;
    }
    wave_sync();
    for (int i = 0; i < n; ++i) {
        const int64_t t = t0 + i;
        float d[NE], z[DENSE ? NE : 1], ad[NE];
        if (!AHEAD) {
            if constexpr (DENSE) load(a.z, t, zn, -INFINITY);
            if (a.add) load(a.add, t, an, 0.0f);
        }
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            if constexpr (DENSE) z[j] = zn[j] > -INFINITY ? zn[j] : -INFINITY;
            ad[j] = an[j];
        }
        if (AHEAD && i + 1 < n) {
            if constexpr (DENSE) load(a.z, t + 1, zn, -INFINITY);
            if (a.add) load(a.add, t + 1, an, 0.0f);
        }
        if (live && mine == i) row[e] = sum;
        wave_sync();
#pragma unroll
        for (int j = 0; j < NE / VEC; ++j) {
            const int at = min((lane + 64 * j) * VEC, E - VEC);
            if constexpr (VEC == 1) {
                d[j] = row[at];
            } else {
                const float2 v = *reinterpret_cast<const float2*>(row + at);
                d[2 * j] = v.x, d[2 * j + 1] = v.y;
            }
        }
        wave_sync();
        if (live && mine == i) row[e] = 0.0f;
        if constexpr (DENSE) {
            float m = z[0], s = 0.0f, dot = 0.0f;
#pragma unroll
            for (int j = 1; j < NE; ++j) m = fmaxf(m, z[j]);
            m = moe::wave_all_max(m);
#pragma unroll
            for (int j = 0; j < NE; ++j) {
                z[j] = z[j] > -INFINITY ? soft32(z[j], m) : 0.0f;
                s += z[j];
                dot = fmaf(z[j], d[j], dot);
            }
            s = moe::wave_all_sum(s);
            dot = moe::wave_all_sum(dot);
            const float f = s > 0.0f ? __builtin_amdgcn_rcpf(s) : 0.0f;
            dot *= f;
#pragma unroll
            for (int j = 0; j < NE; ++j) d[j] = z[j] * f * (d[j] - dot);
        }
        if (a.add) {
#pragma unroll
            for (int j = 0; j < NE; ++j) d[j] += ad[j];
        }
#pragma unroll
        for (int j = 0; j < NE / VEC; ++j) {
            const int at = (lane + 64 * j) * VEC;
            if (at >= E) continue;
            if constexpr (ZD == MOE_X_F32) reinterpret_cast<float*>(a.dz)[t * E + at] = d[j];
            else if constexpr (VEC == 1) reinterpret_cast<__bf16*>(a.dz)[t * E + at] = (__bf16)d[j];
            else reinterpret_cast<bf16x2*>(a.dz)[(t * E + at) / 2] = bf16x2{(__bf16)d[2 * j], (__bf16)d[2 * j + 1]};
        }
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

// Calls go with the number of experts a lane holds; bf16 rows of an even length are
// read in pairs.
template <int ZD, int VEC, typename Go>
void by_experts(int E, const Go& go) {
    using std::integral_constant;
    const auto with = [&](auto ne) { go(integral_constant<int, ZD>{}, integral_constant<int, VEC>{}, ne); };
    const int ne = (E + 64 * VEC - 1) / (64 * VEC) * VEC;
    if (ne <= 2) with(integral_constant<int, 2>{});
    else if (ne <= 4) with(integral_constant<int, 4>{});
    else if (ne <= 5 && VEC == 1) with(integral_constant<int, VEC == 1 ? 5 : 6>{});
    else if (ne <= 6) with(integral_constant<int, 6>{});
    else if (ne <= 8) with(integral_constant<int, 8>{});
    else if (ne <= 16) with(integral_constant<int, 16>{});
    else if (ne <= 32) with(integral_constant<int, 32>{});
    else with(integral_constant<int, 64>{});
}

template <typename Go>
void by_format(int z_dtype, int E, const Go& go) {
    if (z_dtype == MOE_X_F32) by_experts<MOE_X_F32, 1>(E, go);
    else if (E % 2 == 0) by_experts<MOE_X_BF16, 2>(E, go);
    else by_experts<MOE_X_BF16, 1>(E, go);
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

int seg_of(int k) { return k <= 8 ? 8 : k <= 16 ? 16 : 32; }

// Tokens a wave: as many as leave 16 waves a CU, and as have their picks side by side.
int batch_of(int T, int seg) {
    int n = 1;
    while (n < 64 / seg && T / (2 * n) >= 256 * 16) n *= 2;
    return n;
}

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
    SelArgs a{z, bias, mask, ids_in, T, E, k, *rule, ids, w, 1, seg_of(k)};
    a.batch = batch_of(T, a.seg);
    const int waves = E <= 1024 ? SEL_WAVES : 1;
    const int per = waves * a.batch;
    const bool scored = bias || rule->groups > 1;
    by_format(z_dtype, E, [&](auto zd, auto vec, auto ne) {
        constexpr int ZD = decltype(zd)::value, VEC = decltype(vec)::value, NE = decltype(ne)::value;
        const dim3 grid((T + per - 1) / per), block(64 * waves);
        if (scored) hipLaunchKernelGGL((k_select<ZD, VEC, NE, true>), grid, block, waves * sel_lds(E), stream, a);
        else hipLaunchKernelGGL((k_select<ZD, VEC, NE, false>), grid, block, waves * sel_lds(E), stream, a);
    });
    return moe_check_launch("moe_route_select");
}

int moe_route_select_bwd(const void* z, int z_dtype, const int32_t* ids, const float* dw, int T, int E, int k,
                         const moe_select_rule* rule, const void* dz_add, void* dz, hipStream_t stream) {
    if (int rc = check_rule("moe_route_select_bwd", z_dtype, T, E, k, rule)) return rc;
    MOE_REQUIRE(T == 0 || (z && ids && dw && dz), MOE_E_ARG, "moe_route_select_bwd: z, ids, dw and dz must be non-NULL");
    MOE_REQUIRE(moe_aligned16(z) && moe_aligned16(dz_add) && moe_aligned16(dz) && aligned4(ids) && aligned4(dw),
                MOE_E_ALIGN, "moe_route_select_bwd: z, dz_add and dz must start on 16 bytes; ids and dw on 4");
    if (T == 0) return moe_ok();
    SelBwdArgs a{z, ids, dw, T, E, k, *rule, dz_add, dz, 1, seg_of(k)};
    a.batch = batch_of(T, a.seg);
    const int per = SEL_WAVES * a.batch;
    const bool dense = rule->score == MOE_SCORE_SOFTMAX && !rule->renorm;
    by_format(z_dtype, E, [&](auto zd, auto vec, auto ne) {
        constexpr int ZD = decltype(zd)::value, VEC = decltype(vec)::value, NE = decltype(ne)::value;
        const dim3 grid((T + per - 1) / per), block(64 * SEL_WAVES);
        const size_t lds = (size_t)SEL_WAVES * 4 * E;
        if (dense) hipLaunchKernelGGL((k_select_bwd<ZD, VEC, NE, true>), grid, block, lds, stream, a);
        else hipLaunchKernelGGL((k_select_bwd<ZD, VEC, NE, false>), grid, block, lds, stream, a);
    });
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
