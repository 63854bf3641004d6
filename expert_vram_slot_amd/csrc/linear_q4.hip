// Dense 4-bit product: y = x W^T (+ bias), W in 4-bit blocks with one fp16
// scale for each group of inputs of a row.
//
// y[t][n] = bias[n] + sum over groups b of d[n][b] * (sum over k in b of
// x[t][k] * q[n][k] - 8 * sum over k in b of x[t][k]).  The codes lie as in a
// slab's Q4B32 plane (blocks of 32 inputs, byte j of a block: input j low,
// input j + 16 high), whatever the group.
//
// Every batch size runs on the matrix cores: v_mfma_f32_16x16x32_bf16 takes
// 16 tokens against 16 rows of W over one block of 32 inputs.
//  - Codes 0..15 are whole numbers a bf16 holds.  A code in a byte read as
//    fp8 e4m3 is code * 2^-9 (the subnormals and the first binade are one
//    line), so the fp8 -> bf16 conversion with scale 2^9 makes two codes at a
//    time: 7 vector instructions for 8 codes, masks included.
//  - The correction by 8 goes in as the product's C operand, -8 * sum of x
//    over the group, and each group's result is scaled in fp32: no weight is
//    rounded.  fp32 activations are split into three bf16 planes (8 + 8 + 8
//    bits, exact) and take three products.
//  - A lane loads 16 bytes of codes: lane (row i, quarter q) the whole block q
//    of a chunk of 128 inputs, so a load instruction takes 64 bytes of each of
//    16 rows.  A product wants one block's codes over the four quarters: a
//    4 x 4 transpose between quarters and registers, four lane swaps.
//  - x is staged in LDS in the order the product takes it (block, quarter,
//    token, the quarter's eight inputs), with the group sums beside it.
#include <type_traits>

#include "common.hpp"

namespace {

using v4u = uint32_t __attribute__((ext_vector_type(4)));
using v2u = uint32_t __attribute__((ext_vector_type(2)));
using v4f = float __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int CH = 128;  // inputs of a chunk: one 16-byte load of each lane

struct LinArgs {
    const void* x;
    int64_t ldx;
    const v4u* wq;
    const _Float16* scales;
    const float* bias;
    void* y;
    int64_t ldy;
    int T, N, K;
    int y_dtype;
    int wk;          // waves that share a row tile, each with every wk-th chunk
    int tp;          // token rows staged per tile: a power of two up to 16
    int kc;          // inputs staged at a time
};

// Eight codes of a dword (low nibbles, then high) as bf16.
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t d) {
    const uint32_t lo = d & 0x0F0F0F0Fu, hi = (d >> 4) & 0x0F0F0F0Fu;
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false);
    const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
}

// Register i of quarter q <-> register q of quarter i.
__device__ __forceinline__ v4u transpose4(v4u w) {
    const auto a = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
    const auto c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
    return v4u{c[0], d[0], c[1], d[1]};
}

template <int XD>
constexpr int PLANES = XD == MOE_X_F32 ? 3 : 1;

// Eight consecutive inputs of a token, as bf16 planes.
template <int XD>
struct Piece {
    v4u raw[XD == MOE_X_F32 ? 2 : 1];

    __device__ __forceinline__ void zero() {
        for (auto& r : raw) r = v4u{0, 0, 0, 0};
    }
    __device__ __forceinline__ void load(const LinArgs& a, int64_t t, int k) {
        const char* p = reinterpret_cast<const char*>(a.x) + (t * a.ldx + k) * (XD == MOE_X_F32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < (XD == MOE_X_F32 ? 2 : 1); ++i) raw[i] = reinterpret_cast<const v4u*>(p)[i];
    }
    __device__ __forceinline__ float sum() const {
        float s = 0.0f;
        if constexpr (XD == MOE_X_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s += __uint_as_float(raw[i >> 2][i & 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) s += moe::bf16_lo(raw[0][i]) + moe::bf16_hi(raw[0][i]);
        }
        return s;
    }
    // Plane p: the eight inputs less what the planes before it hold, cut to
    // bf16 (cut, not rounded: three cuts of 8 bits take a whole significand).
    __device__ __forceinline__ v4u plane(int p) const {
        if constexpr (XD != MOE_X_F32) {
            return raw[0];
        } else {
            v4u out;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t h[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v = __uint_as_float(raw[i >> 1][2 * (i & 1) + j]);
                    for (int c = 0; c < p; ++c) v -= __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
                    h[j] = __float_as_uint(v) >> 16;
                }
                out[i] = h[0] | (h[1] << 16);
            }
            return out;
        }
    }
};

// LDS: planes of x [plane][block of 32][tile][quarter][tp tokens][8 bf16],
// then the group sums [group][16 * NT] fp32.
template <int XD, int G, int NT>
struct Stage {
    char* base;
    int tp, kc;
    __device__ __forceinline__ int plane_bytes() const { return kc / 32 * NT * 64 * tp; }
    __device__ __forceinline__ char* piece(int p, int block, int nt, int q, int tok) const {
        return base + p * plane_bytes() + (((block * NT + nt) * 4 + q) * tp + tok) * 16;
    }
    __device__ __forceinline__ float* sums(int group) const {
        return reinterpret_cast<float*>(base + PLANES<XD> * plane_bytes()) + group * 16 * NT;
    }
    static __host__ __device__ size_t bytes(int tp, int kc) {
        return (size_t)PLANES<XD> * (kc / 32) * NT * 64 * tp + (size_t)(kc / G) * 16 * NT * 4;
    }
    // inputs 8j .. 8j + 7 of token `tok` of the stage
    __device__ __forceinline__ void put(const Piece<XD>& v, int tok, int j, int lane) const {
        const int block = j >> 2, part = j & 3, nt = tok / 16, t = tok & 15;
        const int half = part >> 1, q = (part & 1) * 2;
#pragma unroll
        for (int p = 0; p < PLANES<XD>; ++p) {
            const v4u b = v.plane(p);
            *reinterpret_cast<v2u*>(piece(p, block, nt, q, t) + 8 * half) = v2u{b[0], b[1]};
            *reinterpret_cast<v2u*>(piece(p, block, nt, q + 1, t) + 8 * half) = v2u{b[2], b[3]};
        }
        float s = v.sum();
#pragma unroll
        for (int m = 1; m < G / 8; m <<= 1) s += __shfl_xor(s, m, moe::WAVE);
        if (j % (G / 8) == 0) sums(j / (G / 8))[tok] = -8.0f * s;
    }
};

// A wave's R row tiles: what its lanes add to a scalar base for their codes
// and scales.  Rows from N on read the last row.
template <int G, int R>
struct Rows {
    static constexpr int NS = CH / G;  // scales of a row in a chunk
    uint32_t code[R], code_end[R], scale[R];
    __device__ __forceinline__ Rows(const LinArgs& a, int64_t n0, int lane) {
        const int q = lane >> 4, nb = a.K >> 5, ng = a.K / G;
        const int end = nb - 1 - (nb - 1) / 4 * 4;  // the last chunk's last block
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t left = a.N - 1 - n0;
            const int i = 16 * r + (lane & 15) < left ? 16 * r + (lane & 15) : (int)left;
            code[r] = (uint32_t)i * nb * 16 + 16 * q;
            code_end[r] = (uint32_t)i * nb * 16 + 16 * (q < end ? q : end);
            scale[r] = (uint32_t)i * ng * 2;
        }
    }
};

// One chunk of codes and its scales, as loaded.  EVEN: K is whole chunks and
// the scales of a row's chunk are one aligned load.  Otherwise that load starts
// on any scale, ends with the matrix at the latest, and what lies past the
// row's end becomes the scale 0 (x is staged as 0 there).
template <int G, int R, bool EVEN>
struct Codes {
    static constexpr int NS = CH / G;
    using S = std::conditional_t<NS == 4, uint64_t, std::conditional_t<NS == 2, uint32_t, uint16_t>>;
    typedef S Loose __attribute__((aligned(2)));
    v4u w[R];
    S s[R];

    // c: chunk, at most the last one (the same in the wave)
    __device__ __forceinline__ void load(const LinArgs& a, const char* codes, const char* scales, const Rows<G, R>& rows,
                                         int c, int chunks) {
        const char* cp = codes + (int64_t)c * 64;
        const bool whole = EVEN || c + 1 < chunks || a.K % CH == 0;
#pragma unroll
        for (int r = 0; r < R; ++r) w[r] = *reinterpret_cast<const v4u*>(cp + (whole ? rows.code[r] : rows.code_end[r]));
        const char* sp = scales + (int64_t)c * (2 * NS);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if constexpr (EVEN) {
                s[r] = *reinterpret_cast<const S*>(sp + rows.scale[r]);
            } else {
                const int ng = a.K / G, left = ng - c * NS;
                const char* end = reinterpret_cast<const char*>(a.scales) + (int64_t)a.N * ng * 2;
                const char* at = sp + rows.scale[r];
                if ((int64_t)a.N * ng >= NS) {
                    const int64_t over = at + sizeof(S) - end;
                    const int back = over > 0 ? (int)over : 0;
                    s[r] = *reinterpret_cast<const Loose*>(at - back) >> (8 * back);
                } else {  // fewer scales than a load in the whole matrix
                    s[r] = 0;
                    for (int i = 0; i < NS; ++i)
                        if (i < left) s[r] |= (S)((S)reinterpret_cast<const uint16_t*>(at)[i] << (16 * i));
                }
                if (left < NS) s[r] &= (S)(((S)1 << (16 * left)) - 1);
            }
        }
    }
};

// Takes a chunk out of its buffer (which is free for the next load from then
// on) into the order the product wants.
template <int G, int R, bool EVEN>
struct Chunk {
    v4u w[R];
    typename Codes<G, R, EVEN>::S s[R];
    __device__ __forceinline__ explicit Chunk(const Codes<G, R, EVEN>& c) {
#pragma unroll
        for (int r = 0; r < R; ++r) w[r] = transpose4(c.w[r]), s[r] = c.s[r];
    }
    __device__ __forceinline__ float scale(int r, int i) const {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)(s[r] >> (16 * i)));
    }
};

template <int XD, int G, int NT, int R, bool EVEN>
__device__ __forceinline__ void multiply(const Chunk<G, R, EVEN>& cw, const Stage<XD, G, NT>& st, int block0, int lane,
                                         v4f (&acc)[R][NT]) {
    const int q = lane >> 4, tok = lane & (st.tp - 1);
    const int step = NT * 64 * st.tp;
    const char* at = st.piece(0, block0, 0, q, tok);
    const float* sums = st.sums(block0 * 32 / G) + 4 * q;
    v4f d[R][NT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        constexpr int BG = G / 32;  // blocks of a group
        bf16x8 b[R];
#pragma unroll
        for (int r = 0; r < R; ++r) b[r] = codes_bf16(cw.w[r][i]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (i % BG == 0) {
                const v4f c = *reinterpret_cast<const v4f*>(sums + (i / BG * NT + nt) * 16);
#pragma unroll
                for (int r = 0; r < R; ++r) d[r][nt] = c;
            }
#pragma unroll
            for (int p = 0; p < PLANES<XD>; ++p) {
                const bf16x8 x = *reinterpret_cast<const bf16x8*>(at + p * st.plane_bytes() + nt * 64 * st.tp);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    d[r][nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, b[r], d[r][nt], 0, 0, 0);
            }
            if (i % BG == BG - 1) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float s = cw.scale(r, i / BG);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[r][nt][e] = fmaf(s, d[r][nt][e], acc[r][nt][e]);
                }
            }
        }
        at += step;
    }
}

// NW waves; wave = (row tiles of R * 16 rows) x (every wk-th chunk).  x is
// staged kc inputs at a time in one buffer; D chunks a wave are on their way.
template <int XD, int G, int NT, int R, int NW, int D, bool EVEN>
__global__ void __launch_bounds__(64 * NW) k_linear_q4(LinArgs a) {
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4;
    const int wk = wave % a.wk, wn = wave / a.wk;
    int64_t n0 = ((int64_t)blockIdx.x * (NW / a.wk) + wn) * (16 * R);
    const bool none = n0 >= a.N;  // this wave only helps to stage x
    if (none) n0 = 0;
    const int64_t t0 = (int64_t)blockIdx.y * (16 * NT);
    const Stage<XD, G, NT> st{smem, a.tp, a.kc};
    const char* codes = reinterpret_cast<const char*>(a.wq) + n0 * (a.K / 2);
    const char* scales = reinterpret_cast<const char*>(a.scales) + n0 * (a.K / G) * 2;
    const Rows<G, R> rows(a, n0, lane);
    v4f acc[R][NT] = {};
    const int chunks = (a.K + CH - 1) / CH;
    const int toks = NT == 1 ? a.tp : 16 * NT;
    const auto clamp = [&](int c) { return c < chunks ? c : chunks - 1; };
    Codes<G, R, EVEN> buf[D];
#pragma unroll
    for (int i = 0; i < D; ++i) buf[i].load(a, codes, scales, rows, clamp(i * a.wk + wk), chunks);
    int c = wk;
    for (int k0 = 0; k0 < a.K; k0 += a.kc) {
        const int pieces = toks * (a.kc / 8), per = a.kc / 8;
        if (k0) __syncthreads();
        for (int p = threadIdx.x; p < pieces; p += 64 * NW) {
            const int tok = p / per, j = p % per;
            Piece<XD> v;
            v.zero();
            if (t0 + tok < a.T && k0 + 8 * j < a.K) v.load(a, t0 + tok, k0 + 8 * j);
            st.put(v, tok, j, lane);
        }
        __syncthreads();
        if (none) continue;
        const int end = (k0 + a.kc < a.K ? k0 + a.kc : a.K + CH - 1) / CH;
        const int b0 = k0 / 32;
        while (c + (D - 1) * a.wk < end) {
#pragma unroll
            for (int i = 0; i < D; ++i) {
                const Chunk<G, R, EVEN> cur(buf[i]);
                buf[i].load(a, codes, scales, rows, clamp(c + D * a.wk), chunks);
                multiply<XD, G, NT, R, EVEN>(cur, st, 4 * c - b0, lane, acc);
                c += a.wk;
            }
        }
        if (c < end) {  // fewer than D are left, of all inputs
#pragma unroll
            for (int i = 0; i < D - 1; ++i) {
                if (c < end) multiply<XD, G, NT, R, EVEN>(Chunk<G, R, EVEN>(buf[i]), st, 4 * c - b0, lane, acc);
                c += a.wk;
            }
        }
    }
    // waves of one row tile: summed in wave order
    if (a.wk == 1) {
        if (none) return;
    } else {
        __syncthreads();
        v4f* part = reinterpret_cast<v4f*>(smem);
        if (wk > 0) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) part[(wave * R * NT + r * NT + nt) * 64 + lane] = acc[r][nt];
        }
        __syncthreads();
        if (wk > 0 || none) return;
        for (int w = 1; w < a.wk; ++w)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) acc[r][nt] += part[((wave + w) * R * NT + r * NT + nt) * 64 + lane];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t n = n0 + 16 * r + (lane & 15);
        if (n >= a.N) continue;
        const float b = a.bias ? a.bias[n] : 0.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t t = t0 + 16 * nt + 4 * q + e;
                if (t >= a.T) continue;
                const float v = acc[r][nt][e] + b;
                if (a.y_dtype == MOE_X_F32) reinterpret_cast<float*>(a.y)[t * a.ldy + n] = v;
                else reinterpret_cast<__bf16*>(a.y)[t * a.ldy + n] = (__bf16)v;
            }
    }
}

constexpr size_t LIN_LDS = 64 << 10;

template <int XD, int G, int NT, int R, int D>
int launch(LinArgs a, hipStream_t st) {
    constexpr int NW = 8;
    const int pad = (a.K + CH - 1) / CH * CH;
    const int chunks = pad / CH;
    // row tiles enough for the card's 256 CUs go to waves of their own; fewer
    // share their inputs among several waves
    const int64_t tiles = ((int64_t)a.N + 16 * R - 1) / (16 * R) * ((a.T + 16 * NT - 1) / (16 * NT));
    a.wk = 1;
    while (a.wk < NW && a.wk * 2 <= chunks && tiles * a.wk < 2048) a.wk *= 2;
    a.kc = pad;
    if (D < 4 || Stage<XD, G, NT>::bytes(a.tp, a.kc) > LIN_LDS) {
        while (a.wk > 1 && Stage<XD, G, NT>::bytes(a.tp, CH * D * a.wk) > LIN_LDS) a.wk /= 2;
        a.kc = CH * D * a.wk;
    }
    size_t lds = Stage<XD, G, NT>::bytes(a.tp, a.kc);
    const size_t red = (size_t)NW * R * NT * 1024;
    if (a.wk > 1 && lds < red) lds = red;
    const int rows = 16 * R * (NW / a.wk);
    const dim3 grid((unsigned)((a.N + rows - 1) / rows), (unsigned)((a.T + 16 * NT - 1) / (16 * NT)));
    const bool even = a.K % CH == 0 && reinterpret_cast<uintptr_t>(a.scales) % (2 * CH / G) == 0;
    const auto kern = even ? k_linear_q4<XD, G, NT, R, NW, D, true> : k_linear_q4<XD, G, NT, R, NW, D, false>;
    hipLaunchKernelGGL(kern, grid, dim3(64 * NW), lds, st, a);
    return moe_check_launch("moe_linear_q4");
}

template <int XD, int G>
int pick(LinArgs a, hipStream_t st) {
    const int pad = (a.K + CH - 1) / CH * CH;
    a.tp = 1;
    while (a.tp < 16 && a.tp < a.T) a.tp *= 2;
    if (a.T <= 16) {
        if (Stage<XD, G, 1>::bytes(a.tp, pad) <= LIN_LDS) return launch<XD, G, 1, 1, 4>(a, st);
        return launch<XD, G, 1, 1, 2>(a, st);
    }
    if (a.T <= 32) return launch<XD, G, 2, 2, 2>(a, st);
    return launch<XD, G, 4, 2, XD == MOE_X_F32 ? 1 : 2>(a, st);
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
    LinArgs a{};
    a.x = x, a.ldx = ldx, a.wq = reinterpret_cast<const v4u*>(wq), a.scales = reinterpret_cast<const _Float16*>(scales);
    a.bias = bias, a.y = y, a.ldy = ldy, a.T = T, a.N = N, a.K = K, a.y_dtype = y_dtype;
    const auto go = [&](auto xd) {
        constexpr int XD = decltype(xd)::value;
        return group == 32 ? pick<XD, 32>(a, stream) : group == 64 ? pick<XD, 64>(a, stream) : pick<XD, 128>(a, stream);
    };
    return x_dtype == MOE_X_F32 ? go(std::integral_constant<int, MOE_X_F32>{})
                                : go(std::integral_constant<int, MOE_X_BF16>{});
}
