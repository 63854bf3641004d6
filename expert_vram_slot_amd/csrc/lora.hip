// Low-rank adapters of many requests beside a shared product:
//   y_t = base_t + scale_i B_i (A_i x_t), i = ids_t
// in two passes: h = A x (each token with its own adapter's rows), then y = base
// + B (scale h).
//
// Both run on the matrix cores, v_mfma_f32_16x16x32_bf16, 16 rows of A or B
// against 16 tokens.  Tokens that share an adapter share its rows: they are taken in
// order of their adapters (up to 64 sorted inside each wave, more by k_lora_order, in
// windows of 1024), in tiles of 16, or of 64 where there are many.  The adapters of a
// tile are taken each by itself: nothing of one, an infinity or a NaN, reaches
// another's tokens.  fp32 x and h are cut into three bf16 planes (8 + 8 + 8 bits,
// exact) and take three products: A x keeps its 24 bits, and the products are no bound.
//
// The inputs of A x are split over waves and workgroups; the partial sums (one of
// each split in the workspace) are added in a fixed order.
#include <type_traits>

#include "common.hpp"

namespace {

using v4u = uint32_t __attribute__((ext_vector_type(4)));
using v2u = uint32_t __attribute__((ext_vector_type(2)));
using v4f = float __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef v4f v4f_loose __attribute__((aligned(4)));
typedef v2u v2u_loose __attribute__((aligned(2)));

constexpr int WINDOW = 1024;     // tokens sorted together
// Up to so many are sorted in a wave, without a kernel for it (4096 x 4096, us with and without: 64 tokens of 32
// adapters 17.7 and 15.7, 40 of 16 14.5 and 13.9).
constexpr int WAVE_TOKENS = 64;
// More tokens than this go in tiles of 64.  Tiles of 16 and of 64, us, 4096 x 4096, bf16: 512 tokens of one adapter of
// rank 16 16.5 and 17.1, of 64 in no order 21.9 and 36.9; 1024 of rank 64, of one 30.8 and 31.2, of 8 in a row 32.9 and
// 30.2, of 64 in no order 46.0 and 51.1; 2048 of rank 16, of one 27.9 and 26.0, of 8 in a row 31.7 and 25.9, of 64 in no
// order 41.5 and 53.7, of rank 64 of 8 62.8 and 41.4.
constexpr int MANY = 1024;
constexpr int DOWN_WAVES = 4;    // of a workgroup of the first pass
constexpr int MAX_SPLITS = 4;    // of the inputs, between workgroups
constexpr int STEP = 64;         // rows of B of a step of the second pass
constexpr int RANKS = 64;        // rows of A that a workgroup of the first pass takes

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
    float* h;        // [splits][T][r]
    int32_t* order;  // [T], or NULL: up to WAVE_TOKENS tokens
    int splits;
    int parts;       // workgroups a tile in the second pass
    int steps;       // of STEP rows of B that a wave of the second pass takes
};

__device__ __forceinline__ int adapter_of(const LoraArgs& a, int t) {
    if (t < 0) return -1;
    const int i = a.ids[t];
    return i >= 0 && i < a.n ? i : -1;
}

__device__ __forceinline__ int rank_of(const LoraArgs& a, int i) {
    return i < 0 ? 0 : a.ranks ? min(max(a.ranks[i], 0), a.r) : a.r;
}

// The token (-1: none) and adapter (-1: none) of this lane in a tile of TM
// places: lane l holds place l % TM.
template <int TM>
__device__ __forceinline__ void member(const LoraArgs& a, int tile, int lane, int& tok, int& ad) {
    const int place = tile * TM + (lane & (TM - 1));
    if (a.order) {
        tok = place < a.T ? a.order[place] : -1;
        ad = adapter_of(a, tok);
        return;
    }
    tok = lane < a.T ? lane : -1;
    ad = adapter_of(a, tok);
    const uint32_t key = tok < 0 ? ~0u : ((uint32_t)(ad + 1) << 6) | (uint32_t)lane;
    int rank = 0;
    for (int j = 0; j < a.T; ++j) rank += (uint32_t)__builtin_amdgcn_readlane((int)key, j) < key;
    if (tok < 0) rank = lane;  // behind the others
    const int from = __builtin_amdgcn_ds_permute(4 * rank, lane);  // the lane whose rank this one's number is
    const int src = __shfl(from, place & 63, moe::WAVE);
    tok = __shfl(tok, src, moe::WAVE);
    ad = __shfl(ad, src, moe::WAVE);
}

// Places of the tokens of a window in order of their adapters, then of their
// numbers: each counts the window's smaller keys.  One workgroup for 64 tokens,
// four threads a token: no workgroup waits for another, and nothing depends on the
// order of atomics.  3.5 us for 257 tokens, 6 for 16384: a launch, the ids, and 64
// reads of LDS a thread.
__global__ void __launch_bounds__(256) k_lora_order(LoraArgs a) {
    __shared__ __align__(16) uint32_t key[WINDOW];
    __shared__ int part[4][64];
    const int tid = threadIdx.x, q = tid >> 6;
    const int first = blockIdx.x * 64, w0 = first / WINDOW * WINDOW, n = min(WINDOW, a.T - w0);
    for (int i = tid; i < WINDOW; i += 256)
        key[i] = i < n ? ((uint32_t)(adapter_of(a, w0 + i) + 1) << 10) | (uint32_t)i : ~0u;
    __syncthreads();
    const int at = first - w0 + (tid & 63);
    const uint32_t mine = key[at];
    const int len = (n + 15) / 16 * 4;  // a quarter, in fours
    const v4u* k4 = reinterpret_cast<const v4u*>(key) + q * (len / 4);
    int smaller = 0;
    for (int i = 0; i < len / 4; ++i) {
        const v4u v = k4[i];
        smaller += (v[0] < mine) + (v[1] < mine) + (v[2] < mine) + (v[3] < mine);
    }
    part[q][tid & 63] = smaller;
    __syncthreads();
    if (q == 0 && at < n) a.order[w0 + part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid]] = w0 + at;
}

// Eight floats as three planes of bf16, cut, not rounded.
__device__ __forceinline__ void cut8(float (&v)[8], bf16x8 (&out)[3]) {
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        v4u w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (__float_as_uint(v[2 * i]) >> 16) | (__float_as_uint(v[2 * i + 1]) & 0xFFFF0000u);
        out[p] = __builtin_bit_cast(bf16x8, w);
        if (p < 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] -= __uint_as_float(__float_as_uint(v[i]) & 0xFFFF0000u);
        }
    }
}

// Eight inputs of x, in planes.
template <int XD>
struct Piece {
    v4u raw[XD == MOE_X_F32 ? 2 : 1];
    static constexpr int PLANES = XD == MOE_X_F32 ? 3 : 1;
    __device__ __forceinline__ void get(const char* p) {
        raw[0] = *reinterpret_cast<const v4u*>(p);
        if constexpr (XD == MOE_X_F32) raw[1] = *reinterpret_cast<const v4u*>(p + 16);
    }
    __device__ __forceinline__ void planes(bf16x8 (&out)[PLANES]) const {
        if constexpr (XD == MOE_X_F32) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(raw[i >> 2][i & 3]);
            cut8(v, out);
        } else {
            out[0] = __builtin_bit_cast(bf16x8, raw[0]);
        }
    }
};

// h of a tile of 16 NT tokens, RB blocks of 16 rows of A, a share of the inputs.
// A product takes 32 inputs: lane (m, q) brings inputs 8q.. of row m of A and of
// token m, and holds h of rows 4q.. of token m.  Rows of A past the rank are read
// where there are any and change nothing but h of those rows, which the second
// pass does not use.
//
// What bounds it: the way of x and A to the registers.  16384 tokens of 4096 inputs,
// rank 64: 48 us, x alone (134 MB) takes 37-41 so, A alone (512 KB a workgroup, from the
// caches) 22, the products with no loads 13.  Two groups of loads on their way, not one
// (63 us); of few tokens it is waiting: 257 tokens of 4096 inputs, rank 32, 12 us, one
// token of 2048 3 us.
template <int XD, int NT, int RB>
__global__ void __launch_bounds__(64 * DOWN_WAVES, 2) k_lora_down(LoraArgs a) {
    // products of 32 inputs loaded together: as many as leave room for two waves a SIMD
    constexpr int U = NT == 1 ? (XD == MOE_X_F32 && RB == 4 ? 2 : 4) : XD == MOE_X_BF16 ? 2 : 1;
    constexpr int XB = XD == MOE_X_F32 ? 4 : 2;
    __shared__ __align__(16) v4f red[DOWN_WAVES][NT * RB][64];
    __shared__ int s_tok[16 * NT], s_ad[16 * NT];
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, m = lane & 15, q = lane >> 4;
    // workgroups go to the eight dies in turn: those of a tile, with other rows of A, go to one, where its inputs then are
    // (257 x 8192 x 4096 of rank 64 23 us so, 27 in the tiles' own order)
    const int parts = a.splits * ((a.r + RANKS - 1) / RANKS), part = (blockIdx.x >> 3) % parts;
    const int at_tile = (blockIdx.x >> 3) / parts * 8 + (blockIdx.x & 7), split = part % a.splits, row0 = part / a.splits * RANKS;
    if ((int64_t)at_tile * 16 * NT >= a.T) return;
    int tok, ad;
    member<16 * NT>(a, at_tile, lane, tok, ad);
    if (wid == 0 && lane < 16 * NT) s_tok[lane] = tok, s_ad[lane] = ad;
    const int units = (a.K + 31) / 32, waves = a.splits * DOWN_WAVES, wi = split * DOWN_WAVES + wid;
    const int u0 = (int)((int64_t)units * wi / waves), u1 = (int)((int64_t)units * (wi + 1) / waves);
    const char* xp[NT];
#pragma unroll
    for (int s = 0; s < NT; ++s) {
        const int t = __shfl(tok, NT == 1 ? lane : 16 * s + m, moe::WAVE);
        xp[s] = reinterpret_cast<const char*>(a.x) + (int64_t)max(t, 0) * a.ldx * XB;
    }
    unsigned long long rest = __ballot(ad >= 0);
    for (int pass = 0; rest; ++pass) {
        const int d = __builtin_amdgcn_readlane(ad, __builtin_ctzll(rest));
        rest &= ~__ballot(ad == d);
        if (pass % gridDim.y != blockIdx.y || row0 >= rank_of(a, d)) continue;
        const uint16_t* ap[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) ap[b] = a.a + ((int64_t)d * a.r + min(row0 + 16 * b + m, a.r - 1)) * a.K;
        v4f acc[NT][RB] = {};
        v4u af[2][U][RB];
        Piece<XD> xf[2][U][NT];
        const auto fetch = [&](int buf, int u) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int un = min(u + i, u1 - 1), k = min(32 * un + 8 * q, a.K - 8);
#pragma unroll
                for (int b = 0; b < RB; ++b) af[buf][i][b] = *reinterpret_cast<const v4u*>(ap[b] + k);
#pragma unroll
                for (int s = 0; s < NT; ++s) xf[buf][i][s].get(xp[s] + (int64_t)k * XB);
            }
        };
        const auto multiply = [&](int buf, int u) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (u + i >= u1) break;
                bf16x8 av[RB];
#pragma unroll
                for (int b = 0; b < RB; ++b) {
                    // past the last inputs: a product with 0
                    if (32 * (u + i) + 32 > a.K && 32 * (u + i) + 8 * q >= a.K) af[buf][i][b] = v4u{};
                    av[b] = __builtin_bit_cast(bf16x8, af[buf][i][b]);
                }
#pragma unroll
                for (int s = 0; s < NT; ++s) {
                    bf16x8 xv[Piece<XD>::PLANES];
                    xf[buf][i][s].planes(xv);
#pragma unroll
                    for (int b = 0; b < RB; ++b)
#pragma unroll
                        for (int p = 0; p < Piece<XD>::PLANES; ++p)
                            acc[s][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[b], xv[p], acc[s][b], 0, 0, 0);
                }
            }
        };
        if (u0 < u1) {
            fetch(0, u0);
            for (int u = u0; u < u1; u += 2 * U) {
                if (u + U < u1) fetch(1, u + U);
                multiply(0, u);
                if (u + U < u1) {
                    if (u + 2 * U < u1) fetch(0, u + 2 * U);
                    multiply(1, u + U);
                }
            }
        }
        __syncthreads();  // the tokens are there, and the last adapter's sums are read
#pragma unroll
        for (int s = 0; s < NT; ++s)
#pragma unroll
            for (int b = 0; b < RB; ++b) red[wid][s * RB + b][lane] = acc[s][b];
        __syncthreads();
        for (int i = threadIdx.x; i < NT * RB * 64; i += 64 * DOWN_WAVES) {
            const int sb = i >> 6, l = i & 63, at = 16 * (sb / RB) + (l & 15), j = row0 + 16 * (sb % RB) + 4 * (l >> 4);
            if (s_ad[at] != d || s_tok[at] < 0 || j >= a.r) continue;
            v4f sum = red[0][sb][l];
#pragma unroll
            for (int w = 1; w < DOWN_WAVES; ++w) sum += red[w][sb][l];
            *reinterpret_cast<v4f*>(a.h + ((int64_t)split * a.T + s_tok[at]) * a.r + j) = sum;
        }
    }
}

// The second pass takes a tile of tokens by 64 rows of B a step, in four products (times
// three planes of h):
// lane (m, q) brings columns 8q.. of rows 4m.., a row a product, and of token m's h,
// and holds outputs 4m.. of tokens 4q.., so that a load of the base or a store takes
// 256 bytes of fp32 or 128 of bf16 in a row.
template <int YD>
struct Outputs {
    using Out = std::conditional_t<YD == MOE_X_F32, float, __bf16>;
    using Piece = std::conditional_t<YD == MOE_X_F32, v4f, v2u>;  // four outputs
    using Loose = std::conditional_t<YD == MOE_X_F32, v4f_loose, v2u_loose>;

    static __device__ __forceinline__ Piece get(const void* base, int64_t at) {
        return *reinterpret_cast<const Loose*>(reinterpret_cast<const Out*>(base) + at);
    }
    static __device__ __forceinline__ void put(void* y, int64_t at, const Piece& b, const v4f& v) {
        Loose* to = reinterpret_cast<Loose*>(reinterpret_cast<Out*>(y) + at);
        if constexpr (YD == MOE_X_F32) {
            *to = v + b;
        } else {
            const bf16x4 o = {(__bf16)(moe::bf16_lo(b[0]) + v[0]), (__bf16)(moe::bf16_hi(b[0]) + v[1]),
                              (__bf16)(moe::bf16_lo(b[1]) + v[2]), (__bf16)(moe::bf16_hi(b[1]) + v[3])};
            *to = __builtin_bit_cast(v2u, o);
        }
    }
    static __device__ __forceinline__ void put_one(void* y, int64_t at, const void* base, int64_t at_base, float v) {
        reinterpret_cast<Out*>(y)[at] = (Out)(base ? (float)reinterpret_cast<const Out*>(base)[at_base] + v : v);
    }
};

// Columns j.. of a row of B; those past the rank may hold anything.
__device__ __forceinline__ v4u within(v4u w, int j, int rank) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] &= (j + 2 * k < rank ? 0xFFFFu : 0u) | (j + 2 * k + 1 < rank ? 0xFFFF0000u : 0u);
    return w;
}

// Rows 4m + h of step `step` of adapter d, columns 32c + 8q..
template <int RC>
struct Rows {
    v4u w[RC][4];
    __device__ __forceinline__ void fetch(const LoraArgs& a, int d, int step) {
        const int lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
#pragma unroll
        for (int c = 0; c < RC; ++c)
#pragma unroll
            for (int h = 0; h < 4; ++h)
                w[c][h] = *reinterpret_cast<const v4u*>(a.b + ((int64_t)d * a.N + min(STEP * step + 4 * m + h, a.N - 1)) * a.r +
                                                        min(32 * c + 8 * q, a.r - 8));
    }
    __device__ __forceinline__ void cut(int rank) {
        const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int c = 0; c < RC; ++c) {
            if (32 * c + 32 <= rank) continue;
#pragma unroll
            for (int h = 0; h < 4; ++h) w[c][h] = within(w[c][h], 32 * c + 8 * q, rank);
        }
    }
    // sum += rows times h, as it lies in LDS
    __device__ __forceinline__ void multiply(const v4u (&hs)[RC][3][64], int at, v4f (&sum)[4]) const {
#pragma unroll
        for (int c = 0; c < RC; ++c)
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                const bf16x8 hv = __builtin_bit_cast(bf16x8, hs[c][p][at]);
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    sum[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hv, __builtin_bit_cast(bf16x8, w[c][h]), sum[h], 0, 0, 0);
            }
    }
};

// The same for four waves that share a step: each brings one of the four rows, and all
// read them from LDS.
template <int RC>
struct SharedRows {
    v4u w[RC];
    __device__ __forceinline__ void fetch(const LoraArgs& a, int d, int step) {
        const int lane = threadIdx.x & 63, h = threadIdx.x >> 6, m = lane & 15, q = lane >> 4;
#pragma unroll
        for (int c = 0; c < RC; ++c)
            w[c] = *reinterpret_cast<const v4u*>(a.b + ((int64_t)d * a.N + min(STEP * step + 4 * m + h, a.N - 1)) * a.r +
                                                 min(32 * c + 8 * q, a.r - 8));
    }
    __device__ __forceinline__ void share(int rank, v4u (&rows)[RC][4][64]) {
        const int lane = threadIdx.x & 63, h = threadIdx.x >> 6, q = lane >> 4;
        __syncthreads();  // the last step's are read
#pragma unroll
        for (int c = 0; c < RC; ++c) {
            v4u v = w[c];
            if (32 * c + 32 > rank) v = within(v, 32 * c + 8 * q, rank);
            rows[c][h][lane] = v;
        }
        __syncthreads();
    }
    static __device__ __forceinline__ void multiply(const v4u (&rows)[RC][4][64], const v4u (&hs)[RC][3][64], int at, v4f (&sum)[4]) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int c = 0; c < RC; ++c) {
            bf16x8 w[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) w[h] = __builtin_bit_cast(bf16x8, rows[c][h][lane]);
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                const bf16x8 hv = __builtin_bit_cast(bf16x8, hs[c][p][at]);
#pragma unroll
                for (int h = 0; h < 4; ++h) sum[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hv, w[h], sum[h], 0, 0, 0);
            }
        }
    }
};

// Up to 16 tokens of one adapter, list[0 .. cnt), and their y; rank 0: y = base.
// Token j stands in row 4 (j % 4) + j / 4 of h, so that outputs i of the lanes are
// tokens 4i..4i + 3: with few tokens most loads and stores are left out whole.  The next
// step's rows and base are on their way before this one's y is stored: loads and stores
// count as one, and a wait for loads behind stores would wait for those too.  For the
// same reason no lane is without a token: the places behind the last are the first's.
// FULL: no place is.  SHARED: the workgroup's waves go through the steps together, also
// those that are left without a token.
template <int YD, int RC, bool BASE, bool FULL, bool SHARED>
__device__ __forceinline__ void up_steps(const LoraArgs& a, const v4u (&hs)[RC][3][64], v4u (*shared)[RC][4][64], const int* list,
                                         int cnt, int d, int rank, int first, int last) {
    using O = Outputs<YD>;
    const int lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4, whole = min(last, a.N / STEP);
    const int own = (4 * (m & 3) + (m >> 2) < cnt ? m : 0) + 16 * q;
    int tok[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) tok[i] = list[4 * i + q < cnt ? 4 * i + q : 0];
    // (a wave by itself has a token: known, so that the loop's waits count on its load)
    const auto used = [&](int i) { return FULL || (!SHARED && i == 0) || 4 * i < cnt; };
    std::conditional_t<SHARED, SharedRows<RC>, Rows<RC>> rows;
    typename O::Piece base[4] = {};
    const auto fetch_base = [&](int step) {
        if constexpr (BASE)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (used(i)) base[i] = O::get(a.base, tok[i] * a.ldb + (STEP * step + 4 * m));
    };
    const auto start = [&](v4f (&acc)[4]) {
        const float zero = rank || !BASE ? 0.0f : -0.0f;  // of base plus -0 the bits are base's
#pragma unroll
        for (int h = 0; h < 4; ++h) acc[h] = v4f{zero, zero, zero, zero};
    };
    // sums of a step; the next one's rows are on their way as soon as this one's are out of their registers
    const auto multiply = [&](v4f (&acc)[4], int next) {
        if constexpr (SHARED) {
            rows.share(rank, *shared);
            rows.fetch(a, d, next);
            if (used(0)) rows.multiply(*shared, hs, own, acc);
        } else {
            rows.cut(rank);
            rows.multiply(hs, own, acc);
            rows.fetch(a, d, next);
        }
    };
    if (rank) rows.fetch(a, d, first);
    if (first < whole) fetch_base(first);
    for (int step = first; step < whole; ++step) {
        if constexpr (RC >= (SHARED ? 2 : 4)) asm volatile("" ::: "memory");  // h is read from LDS where it is used: it does not fit registers
        // nor are addresses kept from step to step
#pragma unroll
        for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(tok[i]));
        v4f acc[4];
        start(acc);
        if (rank) multiply(acc, min(step + 1, last - 1));
        typename O::Piece b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = base[i];
        fetch_base(min(step + 1, whole - 1));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (used(i))
                O::put(a.y, tok[i] * a.ldy + (STEP * step + 4 * m), b[i], v4f{acc[0][i], acc[1][i], acc[2][i], acc[3][i]});
    }
    if (whole >= last) return;
    // the last rows, fewer than STEP
    v4f acc[4];
    start(acc);
    if (rank) multiply(acc, last - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (4 * i + q >= cnt) continue;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int n = STEP * whole + 4 * m + h;
            if (n < a.N) O::put_one(a.y, tok[i] * a.ldy + n, BASE ? a.base : nullptr, tok[i] * a.ldb + n, acc[h][i]);
        }
    }
}

// Waves a SIMD: as many as LDS (64) and registers (16) have room for.  Tiles of 64 by
// four, three and two, us: 16384 x 4096 x 4096 of rank 64 112, 112 and 124 (now 109 by four), of rank 16
// 97, 99 and 117.
constexpr int up_resident(int tm, int rc) { return rc == 8 ? 1 : rc == 4 ? 2 : tm == 64 ? 4 : rc == 1 ? 3 : 2; }

// A workgroup takes a tile of tokens, some of its adapters (those without one are one
// more) and some steps.  h of an adapter's tokens, added up, scaled and cut, lies in
// LDS as the products want it.  Of 16 tokens each wave takes steps of its own; of 64
// the four waves share theirs, each with 16 of the tokens, and B passes through LDS once
// for all (16384 x 4096 x 4096 of rank 64: 121 us where two pairs of waves took steps of
// their own and B from the caches; 4096 x 4096 x 4096 of rank 128 80 and 61).
//
// What bounds it: base, y and B.  16384 tokens of 4096 outputs, bf16, rank 64: 61 us,
// 268 MB are 52 at a large copy's rate (92 us where a store took 64 bytes of a row, not
// 128; loads and stores past the caches 99-108).  64 tokens of 131072 outputs, fp32, 16
// adapters of rank 16: 38 us, 134 MB are 26; the base is loaded a step ahead, and at the
// ends of a wave's steps there is nothing else to do.
template <int YD, int TM, int RC, bool BASE>
__global__ void __launch_bounds__(256, up_resident(TM, RC)) k_lora_up(LoraArgs a) {
    constexpr bool SHARED = TM == 64;
    __shared__ __align__(16) v4u hs[TM / 16][RC][3][64];
    __shared__ __align__(16) v4u shared[SHARED ? RC : 1][4][64];
    __shared__ int s_tok[TM];
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, quarter = SHARED ? wid : 0;
    const int at_tile = blockIdx.x / a.parts, part = blockIdx.x - at_tile * a.parts, wave = SHARED ? part : part * (blockDim.x >> 6) + wid;
    const int first = wave * a.steps, last = min(first + a.steps, (a.N + STEP - 1) / STEP);
    int tok, ad;
    member<TM>(a, at_tile, lane, tok, ad);
    if (threadIdx.x < TM) s_tok[lane] = tok;
    int group = 0;
    for (unsigned long long rest = __ballot(tok >= 0 && lane < TM); rest; ++group) {
        const int at = __builtin_ctzll(rest), d = __builtin_amdgcn_readlane(ad, at);
        const unsigned long long here = rest & __ballot(ad == d);  // neighbours: the tile is in order of its adapters
        rest &= ~here;
        if (group % gridDim.y != blockIdx.y) continue;
        const int cnt = __builtin_popcountll(here), rank = rank_of(a, d);
        if (rank == 0 && BASE && a.base == a.y) continue;
        __syncthreads();  // the tokens are there, and the last adapter's h is read
        for (int i = threadIdx.x; i < cnt * RC * 4 && rank; i += blockDim.x) {
            const int k = i / (RC * 4), j = i % (RC * 4) * 8, t = s_tok[at + k];
            float v[8] = {};
            if (j < rank) {
                v4f part[MAX_SPLITS][2];  // on their way together
#pragma unroll
                for (int sp = 0; sp < MAX_SPLITS; ++sp) {
                    const v4f* p = reinterpret_cast<const v4f*>(a.h + ((int64_t)min(sp, a.splits - 1) * a.T + t) * a.r + j);
                    part[sp][0] = p[0], part[sp][1] = p[1];
                }
#pragma unroll
                for (int sp = 0; sp < MAX_SPLITS; ++sp)
                    if (sp < a.splits)
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] += part[sp][e >> 2][e & 3];
                const float f = a.scale ? a.scale[d] : 1.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = j + e < rank ? f * v[e] : 0.0f;
            }
            bf16x8 w[3];
            cut8(v, w);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                hs[k >> 4][j >> 5][p][4 * (k & 3) + (k >> 2 & 3) + 16 * (j >> 3 & 3)] = __builtin_bit_cast(v4u, w[p]);
        }
        __syncthreads();
        const int mine = max(0, min(cnt - 16 * quarter, 16));
        if (first >= last) continue;
        const int* list = s_tok + at + (mine ? 16 * quarter : 0);
        if constexpr (SHARED) {
            if (cnt == TM) up_steps<YD, RC, BASE, true, true>(a, hs[quarter], &shared, list, 16, d, rank, first, last);
            else up_steps<YD, RC, BASE, false, true>(a, hs[quarter], &shared, list, mine, d, rank, first, last);
        } else {
            if (mine == 16) up_steps<YD, RC, BASE, true, false>(a, hs[0], nullptr, list, mine, d, rank, first, last);
            else up_steps<YD, RC, BASE, false, false>(a, hs[0], nullptr, list, mine, d, rank, first, last);
        }
    }
}

bool on_elements(const void* p, int dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == MOE_X_F32 ? 3u : 1u)) == 0;
}

int tile_tokens(int T) { return T > MANY ? 64 : 16; }

// Parts that the inputs are split in between workgroups: enough for one a CU where
// every token has the same adapter, none shorter than 256 inputs.  Four at most and
// none, us: 512 x 4096 x 4096 of rank 16 16.5 and 20.2, 8 x 4096 x 8192 12.4 and 19.4.
int most_splits(int K) {
    const int s = K / 256;
    return s < 1 ? 1 : s > MAX_SPLITS ? MAX_SPLITS : s;
}

int down_splits(int T, int K) {
    const int tm = tile_tokens(T), tiles = (T + tm - 1) / tm, most = most_splits(K);
    const int s = 256 / (tiles > 0 ? tiles : 1);
    return s < 1 ? 1 : s > most ? most : s;
}

size_t h_bytes(int T, int K, int r) { return (size_t)down_splits(T, K) * (T > 0 ? T : 1) * r * 4; }

// The most that up to T tokens need: s parts where they are at most 256 / s tiles.
size_t h_bytes_to(int T, int K, int r) {
    int64_t rows = 1;
    for (int s = 1; s <= most_splits(K); ++s) {
        const int64_t to = s == 1 ? T : 64 * (256 / s), n = (T < to ? T : to) * s;
        if (n > rows) rows = n;
    }
    return (size_t)rows * r * 4;
}

template <int XD, int NT>
void launch_down(const LoraArgs& g, int tiles, int spread, hipStream_t stream) {
    const dim3 grid((tiles + 7) / 8 * 8 * g.splits * ((g.r + RANKS - 1) / RANKS), spread), block(64 * DOWN_WAVES);
    if (g.r <= 16) hipLaunchKernelGGL((k_lora_down<XD, NT, 1>), grid, block, 0, stream, g);
    else if (g.r <= 32) hipLaunchKernelGGL((k_lora_down<XD, NT, 2>), grid, block, 0, stream, g);
    else hipLaunchKernelGGL((k_lora_down<XD, NT, 4>), grid, block, 0, stream, g);
}

template <int YD, int TM, int RC>
void launch_up(const LoraArgs& g, const dim3& grid, const dim3& block, hipStream_t stream) {
    if (g.base) hipLaunchKernelGGL((k_lora_up<YD, TM, RC, true>), grid, block, 0, stream, g);
    else hipLaunchKernelGGL((k_lora_up<YD, TM, RC, false>), grid, block, 0, stream, g);
}

template <int YD, int TM>
void launch_up(const LoraArgs& g, const dim3& grid, const dim3& block, hipStream_t stream) {
    if (g.r <= 32) launch_up<YD, TM, 1>(g, grid, block, stream);
    else if (g.r <= 64) launch_up<YD, TM, 2>(g, grid, block, stream);
    else if (g.r <= 128) launch_up<YD, TM, 4>(g, grid, block, stream);
    else launch_up<YD, TM, 8>(g, grid, block, stream);
}

}  // namespace

extern "C" {

size_t moe_lora_workspace_bytes(int T, int K, int r) {
    if (T < 0 || T > MOE_LINEAR_MAX_T || K < 8 || K > MOE_LINEAR_MAX_NK || r < 8 || r > MOE_LORA_MAX_R) return 0;
    return h_bytes_to(T, K, r) + (T > WAVE_TOKENS ? (size_t)T * 4 : 0);
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
    LoraArgs g{x, ldx, reinterpret_cast<const uint16_t*>(a), reinterpret_cast<const uint16_t*>(b), ranks, scale, ids, n, r,
               T, N, K, base, ldb, y, ldy, reinterpret_cast<float*>(ws), nullptr, down_splits(T, K), 1, 1};
    if (T > WAVE_TOKENS) {
        g.order = reinterpret_cast<int32_t*>(reinterpret_cast<char*>(ws) + h_bytes(T, K, r));
        hipLaunchKernelGGL(k_lora_order, dim3((T + 63) / 64), dim3(256), 0, stream, g);
        if (int rc = moe_check_launch("moe_lora_add/order")) return rc;
    }
    const int tm = tile_tokens(T), tiles = (T + tm - 1) / tm;
    const int most = n < tm ? n : tm;  // adapters of a tile
    // workgroups that share a tile's adapters.  A tile of 16 has seldom more than 8 (first pass, 257 tokens of 64 adapters:
    // 13.1 us by 16, 10.4 by 8, 11.1 by 4; both passes, 40 tokens of 16: 13.9 by 8, 26.0 by one); one of 64 of a prompt
    // has one or two (2048 tokens of 64 adapters in no order 53.7 us by 4, 68.9 by one; 16384 of 8 in a row 117 either way)
    const int spread = most < (tm == 16 ? 8 : 4) ? most : tm == 16 ? 8 : 4;
    if (x_dtype == MOE_X_F32) {
        if (tm == 16) launch_down<MOE_X_F32, 1>(g, tiles, spread, stream);
        else launch_down<MOE_X_F32, 4>(g, tiles, spread, stream);
    } else {
        if (tm == 16) launch_down<MOE_X_BF16, 1>(g, tiles, spread, stream);
        else launch_down<MOE_X_BF16, 4>(g, tiles, spread, stream);
    }
    if (int rc = moe_check_launch("moe_lora_add/down")) return rc;
    // Of a tile of 64 the second pass shares out adapters by two: no difference where a tile has one or two (16384 tokens of
    // 8 in a row 111 us by one, two and four; 2048 35.8, 34.9 and 36.7), more where it has many (1200 x 30000 x 1024 of 64
    // in no order 300, 225 and 183 us; 1025 x 7337 x 2936 of 31 in a row 44, 40 and 40), and by four large ranks lose (4096 x
    // 4096 x 4096 of rank 128 60.6, 60.6 and 62.3)
    const int groups = n + 1 < tm ? n + 1 : tm, up_spread = groups < (tm == 16 ? 8 : 2) ? groups : tm == 16 ? 8 : 2;
    const int resident = up_resident(tm, r <= 32 ? 1 : r <= 64 ? 2 : r <= 128 ? 4 : 8);
    const int64_t at_once = 256 * resident * (tm == 64 ? 1 : 4);
    // adapters of a tile, as far as the numbers tell
    const int64_t units = tm == 64 ? tiles : (int64_t)tiles + (n < T ? n : T - 1);
    // waves a tile (the four that share as one): as many as fill the card a whole number of times, what comes before a
    // wave's first step being as long as START steps.  1, 3 and 6 are alike to 2 %; 0 makes short waves of prompts (3000 x
    // 4096 x 4096 of rank 16 47 us, 41 with 3) and more of them of long rows (1388 x 51862 x 1464 of rank 128 in fp32 221 us, 271)
    constexpr int START = 3;
    const int steps = (N + STEP - 1) / STEP;
    int need = 1;
    int64_t best = INT64_MAX;
    for (int rounds = 1; rounds <= 8; ++rounds) {
        int64_t w = at_once * rounds / units;
        w = w < 1 ? 1 : w > steps ? steps : w;
        const int64_t each = (steps + w - 1) / w, long_ = (units * ((steps + each - 1) / each) + at_once - 1) / at_once * (each + START);
        if (long_ < best) best = long_, need = (int)((steps + each - 1) / each), g.steps = (int)each;
    }
    // waves a workgroup (those that share as one).  Few stand alone, to lie on more CUs (16 x 8192 x 4096 10.8 us, by four
    // 12.6; 7 x 5001 x 1536 10.7 and 12.3); of many, four share a workgroup's start, the adding up and cutting
    // of h: as fast as alone (512 x 4096 x 4096 19.6 us both ways) or up to 6 % slower (64 x 131072 x 4096 43.6 and 41.0)
    const int per = tm == 64 || units * need <= 1024 ? 1 : 4;
    g.parts = (need + per - 1) / per;
    const dim3 grid(g.parts * tiles, up_spread), block(tm == 64 ? 256 : 64 * per);
    if (y_dtype == MOE_X_F32) {
        if (tm == 16) launch_up<MOE_X_F32, 16>(g, grid, block, stream);
        else launch_up<MOE_X_F32, 64>(g, grid, block, stream);
    } else {
        if (tm == 16) launch_up<MOE_X_BF16, 16>(g, grid, block, stream);
        else launch_up<MOE_X_BF16, 64>(g, grid, block, stream);
    }
    return moe_check_launch("moe_lora_add/up");
}

}  // extern "C"
