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
    int batch;  // tokens that a wave takes, 64 / seg at most
    int seg;    // lanes of a token's candidates and picks: 16, 32 or 64 (of the gradient's picks 8, 16 or 32)
};

template <int ZD>
__device__ __forceinline__ float load_z(const void* z, int64_t i) {
    if constexpr (ZD == MOE_X_F32) return reinterpret_cast<const float*>(z)[i];
    else return moe::bf16_to_f32(reinterpret_cast<const uint16_t*>(z)[i]);
}

// 1 / v to a double's last bits, v and 1 / v far inside the normal range (here 1 + exp and sums of 2^-8 to 2^16): the
// hardware's estimate and two Newton steps
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

// Reduction over segments of 8, 16, 32 or 64 lanes.
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
    if (seg > 32) {
        T x, y;
        moe::row_pair<true>(v, x, y);
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
    double* ord;   // [CAND + 2] choices in order
    float* ordz;   // [CAND + 2] and their logits
    float* candz;  // [CAND] candidates: logits
    int* candi;    // [CAND] and ids
    float* pickz;  // [CAND] picks
    int* picki;    // [CAND]
    uint32_t* kept;  // [2 * 4] lanes of the kept groups of a token
};

constexpr size_t SEL_LDS = (CAND + 2) * 12 + CAND * 16 + 40;

__device__ __forceinline__ SelLds sel_parts(unsigned char* p) {
    SelLds l;
    l.ord = reinterpret_cast<double*>(p);
    l.ordz = reinterpret_cast<float*>(l.ord + CAND + 2);
    l.candz = l.ordz + CAND + 2;
    l.candi = reinterpret_cast<int*>(l.candz + CAND);
    l.pickz = reinterpret_cast<float*>(l.candi + CAND);
    l.picki = reinterpret_cast<int*>(l.pickz + CAND);
    l.kept = reinterpret_cast<uint32_t*>(l.picki + CAND);
    return l;
}

// Which lanes hold experts of a kept group: every one of the `per` lanes of a group
// has that group's value.  some: the group has an open expert (two of the lowest biases
// add up to an fp32 -inf all the same; err is inf then).  unsure: values are off by up to
// err, and that may matter.
template <typename T>
__device__ __forceinline__ unsigned long long keep_groups(T value, bool some, T err, int G, int kept, int per, T* sorted,
                                                          bool& unsure) {
    const int lane = threadIdx.x & 63, g = lane / per;
    int rank = 0;
    for (int o = 0; o < G; ++o) {
        const T v = lane_of(value, o * per);
        rank += v > value || (v == value && o < g);
    }
    const bool open = g < G && some;
    unsure = false;
    if (err > 0 && kept < G) {
        if (g < G) sorted[rank] = value;
        wave_sync();
        const T last = sorted[kept - 1], next = sorted[kept];
        const T mid = next > (T)-INFINITY ? next + (T)0.5 * (last - next) : (T)-INFINITY;
        unsure = __any(open && !(rank < kept ? value - err > mid : value + err < mid));
        wave_sync();
    }
    return __ballot(open && rank < kept);
}

// The two largest of what was seen, and one more.
template <typename T>
__device__ __forceinline__ void top2(T v, T& best, T& second) {
    second = v > best ? best : v > second ? v : second;
    best = v > best ? v : best;
}

// A group's value from the two largest choices of each of its lanes (per: a power
// of two, neighbours), of which best and second become the group's.  size: the
// magnitudes of what was added.
template <typename T>
__device__ __forceinline__ T group_value(T& best, T& second, int per, int top, T& size) {
    const auto join = [&](T b, T c) {
        top2(b, best, second);
        top2(c, best, second);
    };
    if (per > 1) join(moe::dpp_of<moe::DPP_XOR1>(best), moe::dpp_of<moe::DPP_XOR1>(second));
    if (per > 2) join(moe::dpp_of<moe::DPP_XOR2>(best), moe::dpp_of<moe::DPP_XOR2>(second));
    if (per > 4) join(moe::dpp_of<moe::DPP_HALF_MIRROR>(best), moe::dpp_of<moe::DPP_HALF_MIRROR>(second));
    if (per > 8) join(moe::dpp_of<moe::DPP_MIRROR>(best), moe::dpp_of<moe::DPP_MIRROR>(second));
    if (per > 16) join(__shfl_xor(best, 16, moe::WAVE), __shfl_xor(second, 16, moe::WAVE));
    const bool two = top > 1 && second > (T)-INFINITY;
    size = two ? fabs(best) + fabs(second) : fabs(best);
    return two ? best + second : best;
}

__host__ __device__ __forceinline__ int lanes_per_group(int G) {
    int per = 64;
    while (per * G > 64) per >>= 1;
    return per;
}

// The sum of a softmax, in double, and the largest logit.
template <int ZD>
__device__ __forceinline__ double softmax64(const SelArgs& a, int64_t t, float& m) {
    const int lane = threadIdx.x & 63;
    m = -INFINITY;
    for (int e = lane; e < a.E; e += 64) m = fmaxf(m, load_z<ZD>(a.z, t * a.E + e));
    m = moe::wave_all_max(m);
    double sum = 0.0;
    for (int e = lane; e < a.E; e += 64) {
        const float z = load_z<ZD>(a.z, t * a.E + e);
        sum += z > -INFINITY ? soft64(z, m) : 0.0;
    }
    return moe::wave_all_sum(sum);
}

// A token's choices in double, an expert at a time.
template <int ZD>
struct Choice64 {
    const SelArgs& a;
    int64_t row;
    float m = 0.0f;
    double sum = 1.0, r = 1.0;
    __device__ __forceinline__ Choice64(const SelArgs& args, int64_t t) : a(args), row(t * args.E) {
        if (a.rule.score == MOE_SCORE_SOFTMAX) sum = softmax64<ZD>(a, t, m), r = rcp64(sum);
    }
    __device__ __forceinline__ double operator()(int e, float& z) const {
        z = load_z<ZD>(a.z, row + e);
        const float b = a.bias ? a.bias[e] : 0.0f;
        double rest;
        if (!(z > -INFINITY && b > -INFINITY)) return -INFINITY;
        return (a.rule.score == MOE_SCORE_SIGMOID ? sigmoid64(z, rest) : soft64(z, m) * r) + (double)b;
    }
};

// The lanes of the kept groups, in double: where fp32 does not tell the groups apart.
template <int ZD>
__device__ __forceinline__ unsigned long long groups64(const SelArgs& a, const Choice64<ZD>& choice, double* sorted) {
    const int lane = threadIdx.x & 63, G = a.rule.groups, gs = a.E / G, per = lanes_per_group(G), g = lane / per;
    double best = -INFINITY, second = -INFINITY, size;
    bool unsure;
    float z;
    if (g < G)
#pragma unroll 1
        for (int i = lane % per; i < gs; i += per) top2(choice(g * gs + i, z), best, second);
    const double value = group_value<double>(best, second, per, a.rule.group_top, size);
    return keep_groups<double>(value, best > -INFINITY, 0.0, G, a.rule.groups_kept, per, sorted, unsure);
}

// A token's picks, round by round, each the best behind the one before: where more
// candidates than lanes are nearly equal, or a group is larger than the registers.
// Picks go to places `to` and up.  m, sum: the softmax's largest logit and its sum, for
// the weights.
template <int ZD>
__device__ __forceinline__ void choose64(const SelArgs& a, int64_t t, const SelLds& l, int to, float& m, float& sum) {
    const int lane = threadIdx.x & 63, E = a.E, G = a.rule.groups, gs = E / G, per = lanes_per_group(G);
    const int first = lane / per * gs + lane % per, end = lane / per < G ? (lane / per + 1) * gs : 0;
    const Choice64<ZD> choice(a, t);
    m = choice.m, sum = (float)choice.sum;
    const bool kept = G == 1 || (groups64<ZD>(a, choice, l.ord) >> lane) & 1;
    double pc = INFINITY;
    float pz = INFINITY;
    int pe = -1;
    for (int i = 0; i < a.k; ++i) {
        double bc = -INFINITY;
        float bz = -INFINITY;
        int be = E;
        if (kept)
            for (int e = first; e < end; e += per) {
                float z;
                const double c = choice(e, z);
                if (c > pc || (c == pc && (z > pz || (z == pz && e <= pe)))) continue;  // taken
                if (c > bc || (c == bc && z > bz)) bc = c, bz = z, be = e;
            }
#pragma unroll
        for (int s = 32; s >= 1; s >>= 1) {
            const double oc = __shfl_xor(bc, s, moe::WAVE);
            const float oz = __shfl_xor(bz, s, moe::WAVE);
            const int oe = __shfl_xor(be, s, moe::WAVE);
            if (oc > bc || (oc == bc && (oz > bz || (oz == bz && oe < be)))) bc = oc, bz = oz, be = oe;
        }
        if (!(bc > -INFINITY)) break;
        if (lane == 0) l.pickz[to + i] = bz, l.picki[to + i] = be;
        pc = bc, pz = bz, pe = be;
    }
    wave_sync();
}

// How a token's experts are compared: by logits (PLAIN), or by choice scores, in a
// row of experts or in a group of lanes for each group of experts.
enum { PLAIN, SCORED, GROUPED };

// Largest of three; the instruction by itself, without the compiler's step that makes
// a signalling NaN quiet first.
__device__ __forceinline__ float max3(float x, float y, float z) {
    float d;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(x), "v"(y), "v"(z));
    return d;
}

// Largest of a lane's numbers, -inf without any.  A signalling NaN may hide some.
template <int NE>
__device__ __forceinline__ float lane_max(const float (&v)[NE]) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j + 1 < NE; j += 2) m = max3(m, v[j], v[j + 1]);
    if (NE & 1) m = max3(m, v[NE - 1], m);
    return max3(m, -INFINITY, -INFINITY);
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    return moe::wave_all(v, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
}

template <int N>
struct Int {
    static constexpr int value = N;
};
template <int N = 1, typename F>
__device__ __forceinline__ void rotations(const F& f) {  // f(1) .. f(15)
    if constexpr (N < 16) {
        f(Int<N>{});
        rotations<N + 1>(f);
    }
}
template <int N, typename T>
__device__ __forceinline__ T turned(T v) { return moe::dpp_of<0x120 + N>(v); }  // of the lane N below in the row of 16

// How far a share of k_select's fp32 softmax may be off, relative to it.  A term: 0.63
// |z| 2^-23 for the rounding of its argument, |z| up to 11 where no maximum is taken
// off and weighed to ln E at most otherwise, and its last bit; E / 64 + 6 additions, a
// quotient, a product.
__device__ __forceinline__ float share_error(int E) { return (2.0f * __logf((float)E) + (float)E * 0x1p-6f + 32.0f) * 0x1p-23f; }

// One wave takes `batch` tokens.
//
// One after the other: the k best of E without k rounds.  The lanes' largest keys
// bound the k-th best from below (there are k at least as good), by bisection
// between the smallest maximum of 8, 16 or 32 sets of lanes and the largest of all;
// whatever reaches that bound, some k + 3 experts, are the candidates.  Keys are the
// logits, or fp32 choices with a bound on how far they are from the 64-bit ones:
// candidates are then taken from twice that below the bound.  A logit or bias that
// closes an expert makes its key NaN or -inf, by 0 * -inf.  With groups each group
// has lanes of its own (as many as there are for all, a power of two), which hold its
// experts; what a token drops is dropped with the lane.
//
// Side by side, a segment of lanes a token: candidates are ranked, by 64-bit choices,
// and the picks weighed.
//
// A token whose candidates do not fit its segment (equal logits, or a bias so large
// that the scores vanish beside it) gets the same search over all its keys; if those
// next to the border still are too many and not all alike, choose64 takes it, k rounds
// over its experts.  Groups that fp32 does not tell apart are valued in double.
//
// What bounds it: instructions.  65537 tokens of 512 bf16 logits, k 10, softmax and a
// bias: 54 us, 312 vector and 260 scalar instructions a token, the vector units at work
// for 84 of 118 thousand clocks; the logits by themselves are 13 us of reading.  16384
// tokens of 288 fp32 logits in 8 groups, sigmoids, k 8: 21 us, 472 a token.  One token
// of 128 experts takes 3 us, a launch.
template <int ZD, int VEC, int NE, int HOW>
__global__ void __launch_bounds__(64 * SEL_WAVES) k_select(SelArgs a) {
    __shared__ __align__(16) unsigned char smem[SEL_WAVES * SEL_LDS];
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const int64_t t0 = ((int64_t)blockIdx.x * SEL_WAVES + wid) * a.batch;
    if (t0 >= a.T) return;
    const int E = a.E, k = a.k, G = a.rule.groups, gs = E / G, seg = a.seg;
    const int n = a.T - t0 < a.batch ? (int)(a.T - t0) : a.batch;
    const SelLds l = sel_parts(smem + wid * SEL_LDS);
    const bool sigmoid = a.rule.score == MOE_SCORE_SIGMOID;
    const bool sums = !sigmoid && (HOW != PLAIN || !a.rule.renorm);  // the softmax over all experts is needed
    // this lane's experts: first, first + stride, ... `own` of them (of pairs: of bf16 pairs)
    const int per = HOW == GROUPED ? lanes_per_group(G) : 64;
    const int first = HOW == GROUPED ? lane / per * gs + lane % per : lane * VEC, stride = HOW == GROUPED ? per : 64 * VEC;
    const int own = HOW == GROUPED ? (lane / per < G ? (gs - lane % per + per - 1) / per : 0) : (E - first + stride - 1) / stride;
    const auto at = [&](int j) { return first + j / VEC * stride + j % VEC; };
    l.pickz[lane] = -INFINITY;
    l.picki[lane] = -1;
    const int mine = lane / seg;  // the token whose candidates and picks this lane takes
    int my_c = 0;
    float my_m = 0.0f, my_sum = 1.0f;
    uint32_t slow = 0;  // tokens to be taken in double from the start
    unsigned long long todo = __ballot(lane < n && (!a.mask || a.mask[t0 + lane]));

    // The biases stay in registers, and the next token's logits are read while this one's are looked at, where registers
    // are left: 16384 tokens of 2048 fp32 logits 59 us so and 70 without.
    constexpr bool KEEP = NE <= 32;
    float bias[HOW != PLAIN && KEEP ? NE : 1];
    const auto bias_at = [&](int j) { return j / VEC < own ? (a.bias ? a.bias[at(j)] : 0.0f) : -INFINITY; };
    if constexpr (HOW != PLAIN && KEEP) {
#pragma unroll
        for (int j = 0; j < NE; ++j) bias[j] = bias_at(j);
    }
    float zn[NE];
    const auto load = [&](int64_t t) {
#pragma unroll
        for (int j = 0; j < NE / VEC; ++j) {
            const int64_t i = t * E + first + j * stride;
            if constexpr (VEC == 1) {
                zn[j] = j < own ? load_z<ZD>(a.z, i) : -INFINITY;
            } else {
                const uint32_t p = j < own ? *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint16_t*>(a.z) + i) : 0xFF80FF80u;
                zn[2 * j] = moe::bf16_lo(p);
                zn[2 * j + 1] = moe::bf16_hi(p);
            }
        }
    };
    const bool rows = !a.ids_in || sums;
    uint32_t close = 0;  // tokens whose groups fp32 does not tell apart
    for (bool exact = false; rows && todo; exact = true) {
        if (KEEP) load(t0 + __builtin_ctzll(todo));
        while (todo) {
            const int i = __builtin_ctzll(todo);
            todo &= todo - 1;
            const int64_t t = t0 + i;
            float z[NE];
            if (!KEEP) load(t);
#pragma unroll
            for (int j = 0; j < NE; ++j) z[j] = zn[j];
            if (KEEP && todo) load(t0 + __builtin_ctzll(todo));
            if (HOW == GROUPED && NE == 64 && gs > NE * per) {  // more than registers
                slow |= 1u << i;
                continue;
            }
            float key[NE], m = 0.0f, sum = 1.0f;
            bool careful = false;
            if (sums) {
                // the softmax needs no maximum taken off where its sum is neither large nor small
#pragma unroll
                for (int j = 0; j < NE; ++j) key[j] = __builtin_amdgcn_exp2f(z[j] * 1.44269504f);
                sum = 0.0f;
#pragma unroll
                for (int j = 0; j < NE; ++j) sum += key[j];
                sum = moe::wave_all_sum(sum);
                careful = __any(!(sum > 0x1p-8f && sum < 0x1p16f));  // or NaN, or nothing open; the same on every lane
                if (careful) {
#pragma unroll
                    for (int j = 0; j < NE; ++j) z[j] = z[j] > -INFINITY ? z[j] : -INFINITY;
                    m = of_code(wave_max_u32(code_of(lane_max(z))));
                    if (m == -INFINITY) continue;
                    sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < NE; ++j) {
                        key[j] = z[j] > -INFINITY ? soft32(z[j], m) : 0.0f;
                        sum += key[j];
                    }
                    sum = moe::wave_all_sum(sum);
                }
                if (mine == i) my_m = m, my_sum = sum;
            }
            if (a.ids_in) continue;
            float slack = 0.0f;  // how far a key may be from its 64-bit choice, but for the rounding of a sum with the bias
            unsigned long long in_kept = ~0ull;
            if constexpr (HOW == PLAIN) {
#pragma unroll
                for (int j = 0; j < NE; ++j) key[j] = z[j];
            } else {
                if (sigmoid) {
                    // |z| s (1 - s) 2^-23 < 2^-25 for the argument, 2^-25 for the exponential, 2^-24 + 2^-23 for sum and quotient
                    slack = 0x1p-22f;
#pragma unroll
                    for (int j = 0; j < NE; ++j) {
                        const float b = KEEP ? bias[KEEP ? j : 0] : bias_at(j);
                        key[j] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z[j] * -1.44269504f)) + fmaf(fminf(z[j], 0.0f), 0.0f, b);
                    }
                } else {
                    const float r = __builtin_amdgcn_rcpf(sum);
                    slack = share_error(E);
                    const auto b = [&](int j) { return KEEP ? bias[KEEP ? j : 0] : bias_at(j); };
                    if (careful) {
#pragma unroll
                        for (int j = 0; j < NE; ++j) key[j] = z[j] > -INFINITY ? fmaf(key[j], r, b(j)) : -INFINITY;
                    } else {
#pragma unroll
                        for (int j = 0; j < NE; ++j) key[j] = fmaf(key[j], r, fmaf(z[j], 0.0f, b(j)));
                    }
                }
            }
            float v = lane_max(key);
            if constexpr (HOW == GROUPED) {
                float best = -INFINITY, second = -INFINITY, size;
#pragma unroll
                for (int j = 0; j < NE; ++j) top2(key[j], best, second);
                const float value = group_value<float>(best, second, per, a.rule.group_top, size);
                // a choice is off by the slack and a rounding, a sum of two by a rounding more
                bool unsure;
                in_kept = keep_groups<float>(value, best > -INFINITY, 2.0f * slack + size * 0x1p-22f, G, a.rule.groups_kept, per,
                                             l.ordz, unsure);
                if (exact) {
                    in_kept = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)l.kept[2 * i]) |
                              ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)l.kept[2 * i + 1]) << 32);
                } else if (unsure) {
                    close |= 1u << i;
                    continue;
                }
                if (!((in_kept >> lane) & 1)) v = -INFINITY;
            }
            // a bound that k keys reach
            const uint32_t code = code_of(v);
            uint32_t lo, hi;
            {
                const auto up = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
                const auto down = [](uint32_t x, uint32_t y) { return x < y ? x : y; };
                // the sets' lanes lie in every row, and so in other groups
                uint32_t x, y, c, d;
                moe::row_pair<true>(code, x, y);
                c = up(x, y), d = c;  // 32 sets of two
                moe::row_pair<false>(c, x, y);
                c = up(x, y);
                d = k > 16 ? (moe::row_pair<false>(d, x, y), down(x, y)) : c;  // 16 of four
                c = up(c, moe::dpp_of<moe::DPP_MIRROR>(c));
                d = k > 8 ? down(d, moe::dpp_of<moe::DPP_MIRROR>(d)) : c;  // 8 of eight
                c = up(c, moe::dpp_of<moe::DPP_HALF_MIRROR>(c));
                d = down(d, moe::dpp_of<moe::DPP_HALF_MIRROR>(d));
                c = up(c, moe::dpp_of<moe::DPP_XOR2>(c));
                d = down(d, moe::dpp_of<moe::DPP_XOR2>(d));
                hi = __builtin_amdgcn_readfirstlane((int)up(c, moe::dpp_of<moe::DPP_XOR1>(c)));
                lo = __builtin_amdgcn_readfirstlane((int)down(d, moe::dpp_of<moe::DPP_XOR1>(d)));
            }
            int have = __builtin_popcountll(__ballot(code >= lo));
            const int enough = k + (seg - k) / 4;
            for (uint32_t step = hi > lo ? 0x80000000u >> __builtin_clz(hi - lo) : 0u; step && have > enough; step >>= 1) {
                const int c = step <= hi - lo ? __builtin_popcountll(__ballot(code >= lo + step)) : 0;
                if (c >= k) lo += step, have = c;
            }
            // the least key of an expert that may be better than one with this key; above -inf: whatever is open
            const auto least_of = [&](float kth) {
                if constexpr (HOW != PLAIN) kth = kth < INFINITY ? kth - (2.0f * slack + fabsf(kth) * 0x1p-22f) : kth;
                return fmaxf(kth, -3.402823466e38f);
            };
            float bound = least_of(of_code(lo));
            int C = 0;
            unsigned long long in[NE];
            const auto reach = [&](float least) {
                C = 0;
#pragma unroll
                for (int j = 0; j < NE; ++j) {
                    in[j] = __ballot(key[j] >= least) & in_kept;
                    C += __builtin_popcountll(in[j]);
                }
            };
            reach(bound);
            if (C > seg) {
                // lanes with several, or equals: the same search over every key.  Fewer than k reach hi: a signalling NaN
                // may have hidden a lane's best from the largest of all, then it is what lies above +inf
                reach(of_code(++hi));
                if (C >= k) hi = 0xFF800001u;
                for (C = seg + 1; hi - lo > 1 && C > seg;) {
                    const uint32_t mid = lo + (hi - lo) / 2;
                    const float kth = fmaxf(of_code(mid), -3.402823466e38f);
                    reach(kth);
                    if (C < k) {
                        hi = mid;
                        C = seg + 1;
                        continue;
                    }
                    lo = mid;
                    bound = least_of(kth);
                    reach(bound);
                }
                if (C > seg) {
                    // what lies above the k-th key for certain, and of the rest, if it is all alike, the lowest ids
                    const float kth = fmaxf(of_code(lo), -3.402823466e38f), over = kth + (kth - least_of(kth));
                    reach(least_of(kth));
                    unsigned long long sure[NE];
                    int n_sure = 0;
                    float z0 = 0.0f, b0 = 0.0f;
                    bool any = false, alike = true;
#pragma unroll
                    for (int j = 0; j < NE; ++j) {
                        sure[j] = in[j] & __ballot(key[j] > over);
                        n_sure += __builtin_popcountll(sure[j]);
                        const unsigned long long band = in[j] & ~sure[j];
                        if (!band) continue;
                        const float b = HOW == PLAIN ? 0.0f : KEEP ? bias[HOW != PLAIN && KEEP ? j : 0] : bias_at(j);
                        if (!any) z0 = lane_of(z[j], __builtin_ctzll(band)), b0 = lane_of(b, __builtin_ctzll(band));
                        any = true;
                        if (band & __ballot(!(z[j] == z0 && b == b0))) alike = false;
                    }
                    if (!alike) {
                        slow |= 1u << i;
                        continue;
                    }
                    int most = -1;  // the ids up to it number seg or fewer
                    for (int bit = 1 << 12; bit; bit >>= 1) {
                        int c = n_sure;
#pragma unroll
                        for (int j = 0; j < NE; ++j) c += __builtin_popcountll(in[j] & ~sure[j] & __ballot(at(j) <= most + bit));
                        if (c <= seg) most += bit;
                    }
                    C = 0;
#pragma unroll
                    for (int j = 0; j < NE; ++j) {
                        in[j] &= sure[j] | __ballot(at(j) <= most);
                        C += __builtin_popcountll(in[j]);
                    }
                }
            }
            if (mine == i) my_c = C;
            int base = i * seg;
#pragma unroll
            for (int j = 0; j < NE; ++j) {
                if (!in[j]) continue;
                if (__builtin_amdgcn_inverse_ballot_w64(in[j])) {
                    const int p = __builtin_amdgcn_mbcnt_hi((uint32_t)(in[j] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)in[j], base));
                    l.candz[p] = z[j];
                    l.candi[p] = at(j);
                }
                base += __builtin_popcountll(in[j]);
            }
        }
        if constexpr (HOW == GROUPED) {  // their groups in double, then once more
            for (uint32_t c = close; c; c &= c - 1) {
                const int i = __builtin_ctz(c);
                const Choice64<ZD> choice(a, t0 + i);
                const unsigned long long kept = groups64<ZD>(a, choice, l.ord);
                if (lane < 2) l.kept[2 * i + lane] = (uint32_t)(kept >> (32 * lane));
                wave_sync();
            }
        }
        todo = close;
        close = 0;
    }
    wave_sync();
    const int r = lane & (seg - 1);
    if (!a.ids_in) {
        const bool live = r < my_c;
        const float zc = live ? l.candz[lane] : -INFINITY;
        const int id = live ? l.candi[lane] : 0x7FFFFFFF;
        int rank = 0;
        if (HOW == PLAIN || !a.bias) {
            // by logits, then ids
            for (int x = 0; x < seg; x += 16) {
                const float oz = x ? __shfl_xor(zc, x, moe::WAVE) : zc;
                const int oi = x ? __shfl_xor(id, x, moe::WAVE) : id;
                if (x) rank += oz > zc || (oz == zc && oi < id);
                rotations([&](auto by) {
                    constexpr int N = decltype(by)::value;
                    const float tz = turned<N>(oz);
                    const int ti = turned<N>(oi);  // by every lane, whatever tz is
                    rank += (tz > zc) | ((tz == zc) & (ti < id));
                });
            }
        } else {
            double c, rest, share = rcp64((double)my_sum);
            float top = my_m;  // what was taken off the logits under `share`
            for (bool exact = sigmoid;; exact = true) {
                const double p = !live ? 0.0 : sigmoid ? sigmoid64(zc, rest) : soft64(zc, top) * share;
                c = live ? p + (double)a.bias[id] : -INFINITY;
                rank = 0;
                for (int x = 0; x < seg; x += 16) {
                    const double o = x ? __shfl_xor(c, x, moe::WAVE) : c;
                    if (x) rank += o > c;
                    rotations([&](auto by) { rank += turned<decltype(by)::value>(o) > c; });
                }
                // equal choices share a rank: the logits, then the ids decide
                int* who = reinterpret_cast<int*>(l.ordz) + mine * seg;
                if (live) who[rank] = lane;
                wave_sync();
                if (__any(live && who[rank] != lane)) {
                    for (int x = 0; x < seg; ++x) {
                        const int src = mine * seg + x;
                        const double o = __shfl(c, src, moe::WAVE);
                        const float oz = __shfl(zc, src, moe::WAVE);
                        const int oi = __shfl(id, src, moe::WAVE);
                        if (live) rank += o == c && (oz > zc || (oz == zc && oi < id));
                    }
                }
                if (exact) break;
                // the sum of the softmax is an fp32 one: where two are so close that it may have put them the wrong way round,
                // one in double.  Each pick against the next (what holds for neighbours adds up for others), and the last one
                // against every candidate behind it: of these a near one may stand behind others that are far enough.  Equal
                // logits have equal scores, and their order stands
                wave_sync();
                if (live) l.ord[mine * seg + rank] = c, l.ordz[mine * seg + rank] = zc, l.candz[mine * seg + rank] = (float)p * share_error(E);
                wave_sync();
                const int o = r < k - 1 ? lane + 1 : mine * seg + k - 1;
                unsigned long long near = __ballot(r != k - 1 && (r < k - 1 ? r + 1 : r) < my_c && l.ordz[lane] != l.ordz[o] &&
                                                   fabs(l.ord[lane] - l.ord[o]) <= (double)(l.candz[lane] + l.candz[o]));
                if (!near) break;
                while (near) {
                    const int i = __builtin_ctzll(near) / seg;
                    float m;
                    const double s = rcp64(softmax64<ZD>(a, t0 + i, m));
                    if (mine == i) share = s, top = m;
                    near &= ~__ballot(mine == i);
                }
                wave_sync();
            }
        }
        if (live && rank < k && !((slow >> mine) & 1)) l.pickz[mine * seg + rank] = zc, l.picki[mine * seg + rank] = id;
        wave_sync();
        for (; slow && HOW != PLAIN; slow &= slow - 1) {
            const int i = __builtin_ctz(slow);
            float m, sum;
            choose64<ZD>(a, t0 + i, l, i * seg, m, sum);
            if (mine == i) my_m = m, my_sum = sum;
        }
    }
    // the weights
    const bool here = mine < n && r < k;
    const int64_t o = (t0 + mine) * k + r;
    float zp = l.pickz[lane];
    int pick = l.picki[lane];
    if (a.ids_in && here && (!a.mask || a.mask[t0 + mine])) {
        const int e = a.ids_in[o];
        if (e >= 0 && e < E) {
            zp = load_z<ZD>(a.z, (t0 + mine) * E + e);
            if (zp > -INFINITY) pick = e;
        }
    }
    const bool live = pick >= 0;
    double s = 0.0, rest;
    if (a.rule.renorm) s = share64(a.rule.score, zp, live, seg);
    else if (live) s = sigmoid ? sigmoid64(zp, rest) : soft64(zp, my_m) * rcp64((double)my_sum);
    if (here) {
        if (!a.ids_in) a.ids[o] = pick;
        a.w[o] = (float)((double)a.rule.scale * s);
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
//
// What bounds it: the rows.  65537 tokens of 512 bf16 logits, dense: 31 us, 134 MB are
// 26 at a large copy's rate (203 vector instructions a token); 16384 of 288 in fp32, the
// picks alone and another gradient added: 9 us, 38 MB are 7.
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
    constexpr bool AHEAD = NE <= 32;  // the next token's rows while this one's are looked at (16384 x 2048 fp32: 45 us, 47 without)
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
            if constexpr (DENSE) z[j] = zn[j];
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
            float s = 0.0f, dot = 0.0f, ex[NE];  // the softmax as in k_select
#pragma unroll
            for (int j = 0; j < NE; ++j) {
                ex[j] = __builtin_amdgcn_exp2f(z[j] * 1.44269504f);
                s += ex[j];
                dot = fmaf(ex[j], d[j], dot);
            }
            s = moe::wave_all_sum(s);
            if (__any(!(s > 0x1p-8f && s < 0x1p16f))) {
#pragma unroll
                for (int j = 0; j < NE; ++j) z[j] = z[j] > -INFINITY ? z[j] : -INFINITY;
                const float m = of_code(wave_max_u32(code_of(lane_max(z))));
                s = dot = 0.0f;
#pragma unroll
                for (int j = 0; j < NE; ++j) {
                    ex[j] = z[j] > -INFINITY ? soft32(z[j], m) : 0.0f;
                    s += ex[j];
                    dot = fmaf(ex[j], d[j], dot);
                }
                s = moe::wave_all_sum(s);
            }
            dot = moe::wave_all_sum(dot);
            const float f = s > 0.0f ? __builtin_amdgcn_rcpf(s) : 0.0f;
            dot *= f;
#pragma unroll
            for (int j = 0; j < NE; ++j) d[j] = ex[j] * f * (d[j] - dot);
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

// One workgroup a layer: 48 layers of 512 experts are 300 KB, and the time, 4 us, is a
// launch and two passes of waiting for them.  Whole numbers: C - n c is exact.
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

// Calls go with the number of experts a lane holds (64: what is more is taken in
// double from the start); bf16 rows of an even length are read in pairs.  Five and six
// have kernels of their own, where 8 instead costs most in groups: 65536 tokens of 288
// experts 67 us and 88, of 384 71 and 90, in a row 27.5 and 30.  Three and seven have
// none, they would gain 4 %: of 192 experts 56 us and 53.5, of 448 91 and 87.
template <typename Go>
void by_count(int ne, const Go& go) {
    using std::integral_constant;
    if (ne <= 2) go(integral_constant<int, 2>{});
    else if (ne <= 4) go(integral_constant<int, 4>{});
    else if (ne <= 5) go(integral_constant<int, 5>{});
    else if (ne <= 6) go(integral_constant<int, 6>{});
    else if (ne <= 8) go(integral_constant<int, 8>{});
    else if (ne <= 16) go(integral_constant<int, 16>{});
    else if (ne <= 32) go(integral_constant<int, 32>{});
    else go(integral_constant<int, 64>{});
}

template <typename Go>
void by_format(int z_dtype, int E, const Go& go) {
    using std::integral_constant;
    const integral_constant<int, 1> one;
    const int ne = (E + 63) / 64;
    if (z_dtype == MOE_X_F32) by_count(ne, [&](auto c) { go(integral_constant<int, MOE_X_F32>{}, one, c); });
    else if (E % 2) by_count(ne, [&](auto c) { go(integral_constant<int, MOE_X_BF16>{}, one, c); });
    else
        by_count((E + 127) / 128 * 2, [&](auto c) {
            constexpr int NE = decltype(c)::value == 5 ? 6 : decltype(c)::value;
            go(integral_constant<int, MOE_X_BF16>{}, integral_constant<int, 2>{}, integral_constant<int, NE>{});
        });
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
// Lanes of a token's candidates: k, some equal ones and a few for the bound's sake.  The
// fewer, the more tokens side by side, and the sooner equal logits have to be searched
// for one by one.  65537 tokens of 512 bf16 logits, us by 16, 32 and 64 lanes, a bias and
// logits that differ: k 10 50, 61 and 94, k 12 52, 61 and 95, k 14 96, 62 and 97, k 22 by
// 32 72 and by 64 108, k 28 88 and 112.  No bias, logits in steps of a quarter (many
// equals): k 8 50 and 40 by 32, k 10 74 and 43, k 12 107 and 45, k 22 by 32 85 and by 64 70,
// k 28 164 and 71.  The cuts lie where both kinds are well served.
int cand_of(int k) { return k <= 10 ? 16 : k <= 22 ? 32 : 64; }

// Tokens a wave: as many as leave 16 waves a CU, and as have their picks side by side.
// Several at a time save the second half of the work (65537 tokens of 512: 50 us by four
// and 75 one by one; 8192 12.4 by two, 14.4 one by one, 15.0 by four), one at a time fills
// the card (4096 tokens: 9.7 us, 13.1 by four; 1024 7.6 and 12.0).
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
    SelArgs a{z, bias, mask, ids_in, T, E, k, *rule, ids, w, 1, cand_of(k)};
    a.batch = batch_of(T, a.seg);
    const int per = SEL_WAVES * a.batch, G = rule->groups;
    const dim3 grid((T + per - 1) / per), block(64 * SEL_WAVES);
    using std::integral_constant;
    const auto go = [&](auto zd, auto vec, auto ne, auto how) {
        hipLaunchKernelGGL((k_select<decltype(zd)::value, decltype(vec)::value, decltype(ne)::value, decltype(how)::value>), grid,
                           block, 0, stream, a);
    };
    if (G > 1 && !ids_in) {
        const int per_group = lanes_per_group(G), ne = (E / G + per_group - 1) / per_group;
        const integral_constant<int, GROUPED> how;
        const integral_constant<int, 1> one;
        if (z_dtype == MOE_X_F32) by_count(ne, [&](auto c) { go(integral_constant<int, MOE_X_F32>{}, one, c, how); });
        else by_count(ne, [&](auto c) { go(integral_constant<int, MOE_X_BF16>{}, one, c, how); });
    } else {
        by_format(z_dtype, E, [&](auto zd, auto vec, auto ne) {
            if (bias && !ids_in) go(zd, vec, ne, integral_constant<int, SCORED>{});
            else go(zd, vec, ne, integral_constant<int, PLAIN>{});
        });
    }
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
