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
//  - The correction by 8 is a product of its own, x against a constant -8,
//    shared by the rows of a wave, and each group's result is scaled in fp32:
//    no weight is rounded.  fp32 activations are split into three bf16 planes
//    (8 + 8 + 8 bits, exact) and take three products.
//  - Two chunks of 128 inputs are loaded together, so that a load instruction
//    takes whole 128-byte lines, one of each of 8 rows (64 bytes of 16 rows
//    each: the more loads on their way, the more lines left the caches between
//    their halves; one token, 131072 x 2048: 45 us).  An exchange between lanes
//    8 apart gives each chunk 16 rows by four blocks, and a 4 x 4 transpose
//    between quarters of the wave and registers (four lane swaps) gives each
//    block's four dwords to the four quarters, as a product wants them.
//  - x lies in LDS, all of it where that fits (workgroups then stay and take
//    one row tile after the other, the codes' loads running on across tiles),
//    else a stretch of inputs at a time in two buffers.
// That is k_linear_q4.  One token, 131072 x 2048 in groups of 32: 34 us, 4.5 TB/s, 65
// vector instructions for a chunk of 16 rows (8 of them products), the vector unit
// busy half of the time: the waits for loads bound it.  Its launch and one tile's
// latencies bound it where it is small (one token, 2048 x 2048: 5.5 us), the staging
// of x before the first product in between (16 x 8192 x 4096: 9.4 us).
// Many bf16 tokens by many rows go to k_linear_q4_tile, below.
#include <atomic>
#include <type_traits>

#include "common.hpp"

namespace {

using v4u = uint32_t __attribute__((ext_vector_type(4)));
using v2u = uint32_t __attribute__((ext_vector_type(2)));
using v4f = float __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int CH = 128;  // inputs of a chunk: one 16-byte piece of each lane
constexpr int UNIT = 2 * CH;  // inputs loaded together

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
    int wk;  // waves that share a row tile, each with every wk-th chunk
    int kc;  // inputs staged at a time
};

// Eight codes in bytes as bf16.
__device__ __forceinline__ bf16x8 bytes_bf16(uint32_t lo, uint32_t hi) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false);
    const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
}

// Eight codes of a dword (low nibbles, then high) as bf16.
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t d) { return bytes_bf16(d & 0x0F0F0F0Fu, (d >> 4) & 0x0F0F0F0Fu); }

// Register i of quarter q <-> register q of quarter i.
__device__ __forceinline__ v4u transpose4(v4u w) {
    const auto a = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
    const auto c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
    return v4u{c[0], d[0], c[1], d[1]};
}

// Registers a and b of lanes 8 apart: a keeps its lower eight lanes of each row
// of 16 and takes b's lower for its upper; b the other way round.
__device__ __forceinline__ void exchange8(v4u& a, v4u& b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = (int)a[i];
        a[i] = (uint32_t)__builtin_amdgcn_update_dpp((int)a[i], (int)b[i], 0x128, 0xF, 0xC, false);  // row_ror:8
        b[i] = (uint32_t)__builtin_amdgcn_update_dpp((int)b[i], t, 0x128, 0xF, 0x3, false);
    }
}

constexpr int PIECES = 2;  // fp32 pieces of a stage that a thread holds on their way

template <int XD>
constexpr int PLANES = XD == MOE_X_F32 ? 3 : 1;

// x in LDS: [plane][block of 32][token][64 bytes], the row's four 16-byte units
// turned by (token / 4) % 4: a product's lanes read 8 bytes of 16 tokens, which
// then lie in different banks.
template <int XD, int NT, int TP>
struct Stage {
    static constexpr int TOKS = NT * TP;    // token rows (TP: of a tile)
    static constexpr int BLOCK = TOKS * 64;  // bytes of a block of a plane
    char* base;
    int plane;  // bytes

    __device__ __forceinline__ static int turn(int tok) { return (tok >> 2) & 3; }
    static __host__ __device__ size_t bytes(int kc) { return (size_t)PLANES<XD> * (kc / 32) * BLOCK; }
    // Where unit u of the stage comes from.  Tokens and inputs past the end
    // read the last ones: such tokens are not stored, such inputs meet the
    // scale 0.
    __device__ __forceinline__ static const char* source(const LinArgs& a, int64_t t0, int k0, int u) {
        const int block = u / (TOKS * 4), tok = u / 4 % TOKS, k = k0 + 32 * block + 8 * ((u & 3) ^ turn(tok));
        const int64_t t = t0 + tok < a.T ? t0 + tok : a.T - 1;
        return reinterpret_cast<const char*>(a.x) + (t * a.ldx + (k < a.K ? k : a.K - 8)) * (XD == MOE_X_F32 ? 4 : 2);
    }
    // Unit u of eight fp32 inputs, cut (not rounded) into planes: three cuts of
    // 8 bits take a whole significand.
    __device__ __forceinline__ void put(int u, const v4u (&raw)[2]) const {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(raw[i >> 2][i & 3]);
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            v4u out;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                out[i] = (__float_as_uint(v[2 * i]) >> 16) | (__float_as_uint(v[2 * i + 1]) & 0xFFFF0000u);
            *reinterpret_cast<v4u*>(base + p * plane + u * 16) = out;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] -= __uint_as_float(__float_as_uint(v[i]) & 0xFFFF0000u);
        }
    }
    // The wave's units first, first + 64, ... below end straight into LDS
    // (bf16; whole waves of units).
    __device__ __forceinline__ void fetch(const LinArgs& a, int64_t t0, int k0, int first, int step, int end) const {
        typedef __attribute__((address_space(1))) const void* gptr;
        typedef __attribute__((address_space(3))) void* lptr;
        for (int u = first; u < end; u += step)
            __builtin_amdgcn_global_load_lds((gptr)source(a, t0, k0, u + (int)(threadIdx.x & 63)),
                                             (lptr)(base + u * 16), 16, 0, 0);
    }
};

// A wave's R row tiles: what its lanes add to a scalar base for their codes
// (pieces of rows l % 8 and 8 + l % 8 of a tile) and scales (of row l % 16).
// Rows from N on read the last row.
template <int G, int R>
struct Rows {
    uint32_t code[R][2], code_end[R][2], scale[R];
    __device__ __forceinline__ Rows(const LinArgs& a, int64_t n0, int lane) {
        const int piece = (lane >> 4) + 4 * ((lane >> 3) & 1), nb = a.K >> 5, ng = a.K / G;
        const int end = (nb - 1) % 8;  // the last unit's last piece
        const int64_t left = a.N - 1 - n0;
        const auto row = [&](int i) { return (uint32_t)(i < left ? i : (int)left); };
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = row(16 * r + 8 * h + (lane & 7)) * nb * 16;
                code[r][h] = at + 16 * piece;
                code_end[r][h] = at + 16 * (piece < end ? piece : end);
            }
            scale[r] = row(16 * r + (lane & 15)) * ng * 2;
        }
    }
};

// The scales of a wave's rows for one unit, as loaded.  EVEN: K is whole units
// and the scales of a row's unit are one aligned load.  Otherwise a chunk's
// scales are a load that starts on any scale, ends with the matrix at the
// latest, and what lies past the row's end becomes the scale 0.
template <int G, int R, bool EVEN>
struct Scales {
    static constexpr int NS = CH / G;  // scales of a row in a chunk
    using S = std::conditional_t<NS == 4, uint64_t, std::conditional_t<NS == 2, uint32_t, uint16_t>>;
    typedef S Loose __attribute__((aligned(2)));
    S s[R][2];

    __device__ __forceinline__ void load(const LinArgs& a, const char* scales, const Rows<G, R>& rows, int u) {
        const char* sp = scales + (int64_t)u * (4 * NS);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if constexpr (EVEN && NS == 4) {
                const v4u v = *reinterpret_cast<const v4u*>(sp + rows.scale[r]);
                s[r][0] = v[0] | (uint64_t)v[1] << 32, s[r][1] = v[2] | (uint64_t)v[3] << 32;
            } else if constexpr (EVEN && NS == 2) {
                const v2u v = *reinterpret_cast<const v2u*>(sp + rows.scale[r]);
                s[r][0] = v[0], s[r][1] = v[1];
            } else if constexpr (EVEN) {
                const uint32_t v = *reinterpret_cast<const uint32_t*>(sp + rows.scale[r]);
                s[r][0] = (uint16_t)v, s[r][1] = (uint16_t)(v >> 16);
            } else {
                const int ng = a.K / G;
                const char* end = reinterpret_cast<const char*>(a.scales) + (int64_t)a.N * ng * 2;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int left = ng - (2 * u + h) * NS;
                    const char* at = sp + rows.scale[r] + 2 * NS * h;
                    s[r][h] = 0;
                    if (left <= 0) continue;  // the unit's second chunk is past the row
                    if ((int64_t)a.N * ng >= NS) {
                        const int64_t over = at + sizeof(S) - end;
                        const int back = over > 0 ? (int)over : 0;
                        s[r][h] = *reinterpret_cast<const Loose*>(at - back) >> (8 * back);
                    } else {  // fewer scales than a load in the whole matrix
                        for (int i = 0; i < NS; ++i)
                            if (i < left) s[r][h] |= (S)((S)reinterpret_cast<const uint16_t*>(at)[i] << (16 * i));
                    }
                    if (left < NS) s[r][h] &= (S)(((S)1 << (16 * left)) - 1);
                }
            }
        }
    }
    // as fp32, here and now: kept as they were loaded, or folded into a later
    // step, they stay in the load's registers and the next load waits
    __device__ __forceinline__ void take(float (&out)[2][R][NS]) const {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    out[h][r][i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(s[r][h] >> (16 * i)));
                    asm volatile("" : "+v"(out[h][r][i]));
                }
    }
};

// One unit of codes and its scales, as loaded.
template <int G, int R, bool EVEN>
struct Codes {
    v4u w[R][2];
    Scales<G, R, EVEN> s;

    // u: unit, at most the last one (the same in the wave)
    __device__ __forceinline__ void load(const LinArgs& a, const char* codes, const char* scales, const Rows<G, R>& rows,
                                         int u, int units) {
        const char* cp = codes + (int64_t)u * (UNIT / 2);
        const bool whole = EVEN || u + 1 < units || a.K % UNIT == 0;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[r][h] = *reinterpret_cast<const v4u*>(cp + (whole ? rows.code[r][h] : rows.code_end[r][h]));
        s.load(a, scales, rows, u);
    }
};

// Takes a unit's two chunks out of their buffer (which is free for the next
// load from then on) into the order the product wants.
template <int G, int R, bool EVEN>
struct Chunks {
    v4u w[2][R];
    float scale[2][R][CH / G];
    __device__ __forceinline__ explicit Chunks(const Codes<G, R, EVEN>& c) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            v4u lo = c.w[r][0], hi = c.w[r][1];
            exchange8(lo, hi);
            w[0][r] = transpose4(lo), w[1][r] = transpose4(hi);
        }
        c.s.take(scale);
    }
};

// Values of a lane's column of a product that are tokens: all four, one of a
// single token.
template <int NT, int TP>
constexpr int TOK4 = NT == 1 && TP == 1 ? 1 : 4;

// One chunk: R row tiles against the NT token tiles, token tile by token tile,
// so that R + 1 products at a time depend on nothing but their own sums.  at0,
// at1: this lane's two halves of its inputs of the chunk's first block, token
// tile 0.
template <int XD, int G, int NT, int TP, int R>
__device__ __forceinline__ void multiply(const v4u (&w)[R], const float (&scale)[R][CH / G], const char* at0,
                                         const char* at1, int plane, v4f (&acc)[R][NT]) {
    using St = Stage<XD, NT, TP>;
    constexpr uint32_t M8 = 0xC100C100u;  // bf16 -8 twice
    const bf16x8 minus8 = __builtin_bit_cast(bf16x8, v4u{M8, M8, M8, M8});
    constexpr int BG = G / 32;  // blocks of a group
    constexpr bool AS_C = BG == 1 && PLANES<XD> == 1;  // the correction goes in as the product's C
    bf16x8 b[4][R];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) b[i][r] = codes_bf16(w[r][i]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        v4f d[R], eight;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int p = 0; p < PLANES<XD>; ++p) {
                const int off = i * St::BLOCK + nt * 1024;
                const v2u lo = *reinterpret_cast<const v2u*>(at0 + p * plane + off);
                const v2u hi = *reinterpret_cast<const v2u*>(at1 + p * plane + off);
                const bf16x8 x = __builtin_bit_cast(bf16x8, v4u{lo[0], lo[1], hi[0], hi[1]});
                const bool first = i % BG == 0 && p == 0;
                eight = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, minus8, first ? v4f{} : eight, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    d[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, b[i][r], AS_C ? eight : first ? v4f{} : d[r], 0, 0, 0);
            }
            if (i % BG == BG - 1) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int e = 0; e < TOK4<NT, TP>; ++e)
                        acc[r][nt][e] = fmaf(scale[r][i / BG], AS_C ? d[r][e] : d[r][e] + eight[e], acc[r][nt][e]);
            }
        }
    }
}

// Stores the rows n0 .. n0 + 16 R - 1 of the tokens t0 .. t_end - 1, as far as they exist.
template <typename Y, int NT, int R>
__device__ __forceinline__ void store_as(const LinArgs& a, int64_t n0, int64_t t0, int64_t t_end, int lane,
                                         const float (&bias)[R], const v4f (&acc)[R][NT]) {
    Y* y = reinterpret_cast<Y*>(a.y) + (t0 + 4 * (lane >> 4)) * a.ldy + n0 + (lane & 15);
    const bool all = t0 + 16 * NT <= t_end && n0 + 16 * R <= a.N;  // no lane has to be looked at
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            Y* row = y + (int64_t)(16 * nt + e) * a.ldy;
            const bool in_t = t0 + 4 * (lane >> 4) + 16 * nt + e < t_end;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (all || (in_t && n0 + 16 * r + (lane & 15) < a.N)) row[16 * r] = (Y)(acc[r][nt][e] + bias[r]);
        }
}
template <int NT, int R>
__device__ __forceinline__ void store_rows(const LinArgs& a, int64_t n0, int64_t t0, int64_t t_end, int lane,
                                           const float (&bias)[R], const v4f (&acc)[R][NT]) {
    if (a.y_dtype == MOE_X_F32) store_as<float>(a, n0, t0, t_end, lane, bias, acc);
    else store_as<__bf16>(a, n0, t0, t_end, lane, bias, acc);
}

// Adds up the waves of a row group (in wave order, through `part` in LDS) and
// stores its rows.
template <int NT, int R>
__device__ __forceinline__ void store_tile(const LinArgs& a, char* part_, int64_t group, int64_t groups, int64_t t0,
                                           int64_t t_end, int wk, int wave, int lane, const float (&bias)[R], v4f (&acc)[R][NT]) {
    if (a.wk > 1) {
        v4f* part = reinterpret_cast<v4f*>(part_);
        if (wk > 0) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) part[(wave * R * NT + r * NT + nt) * 64 + lane] = acc[r][nt];
        }
        __syncthreads();
        if (wk == 0) {
            for (int w = 1; w < a.wk; ++w)
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) acc[r][nt] += part[((wave + w) * R * NT + r * NT + nt) * 64 + lane];
        }
        __syncthreads();
    }
    if (wk > 0 || group >= groups) return;
    store_rows<NT, R>(a, group * (16 * R), t0, t_end, lane, bias, acc);
}

// NW waves.  A wave takes R row tiles of 16 rows (NW / wk such groups a workgroup)
// and every wk-th unit of them; the workgroup goes on to the groups gridDim.x
// further.  A wave's units come D at a time: while D are multiplied the next D
// are on their way, those of the next tile after a tile's last.
// ALL: x is staged whole, once; else kc = D * wk units at a time.
template <int XD, int G, int NT, int TP, int R, int D, bool ALL, bool EVEN, int NW>
__global__ void __launch_bounds__(64 * NW) k_linear_q4(LinArgs a) {
    using St = Stage<XD, NT, TP>;
    extern __shared__ __align__(16) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), q = lane >> 4;
    const int wk = wave % a.wk, wn = wave / a.wk, per = NW / a.wk;
    const int64_t t0 = (int64_t)blockIdx.y * St::TOKS, t_end = t0 + St::TOKS < a.T ? t0 + St::TOKS : a.T;
    const int64_t groups = ((int64_t)a.N + 16 * R - 1) / (16 * R);
    const int stage_bytes = (int)St::bytes(a.kc);
    const int chunks = (a.K + CH - 1) / CH, units = (chunks + 1) / 2;
    const int rounds = ((units + a.wk - 1) / a.wk + D - 1) / D;  // of D units a wave, for one group
    const int pieces = a.kc / 32 * St::TOKS * 4;                 // of 16 bytes, of a plane of a stage

    // this lane's two 8-byte halves in a block
    const int tok = lane & (TP - 1);
    const int at0 = tok * 64 + (((q >> 1) ^ St::turn(tok)) * 16) + (q & 1) * 8, at1 = at0 ^ 32;

    int64_t group = (int64_t)blockIdx.x * per + wn;
    const auto group_at = [&](int64_t g) { return g < groups ? g : groups - 1; };
    Rows<G, R> rows(a, group_at(group) * (16 * R), lane);
    const char* codes = reinterpret_cast<const char*>(a.wq) + group_at(group) * (16 * R) * (a.K / 2);
    const char* scales = reinterpret_cast<const char*>(a.scales) + group_at(group) * (16 * R) * (a.K / G) * 2;
    const auto unit_at = [&](int round, int i) {
        const int u = (round * D + i) * a.wk + wk;
        return u < units ? u : units - 1;
    };
    Codes<G, R, EVEN> buf[D];
#pragma unroll
    for (int i = 0; i < D; ++i) buf[i].load(a, codes, scales, rows, unit_at(0, i), units);

    // stage 0
    if constexpr (XD == MOE_X_BF16 && TP == 16) {
        St{smem, stage_bytes}.fetch(a, t0, 0, wave * 64, NW * 64, pieces);
        __builtin_amdgcn_s_waitcnt(0x0F70);  // all loads are there (the barrier waits for LDS writes alone)
    } else {
        const St st{smem, stage_bytes / PLANES<XD>};
#pragma unroll 4
        for (int u = tid; u < pieces; u += 64 * NW) {
            const v4u* p = reinterpret_cast<const v4u*>(St::source(a, t0, 0, u));
            if constexpr (XD == MOE_X_F32) {
                const v4u raw[2] = {p[0], p[1]};
                st.put(u, raw);
            } else {
                *reinterpret_cast<v4u*>(smem + u * 16) = p[0];
            }
        }
    }
    __syncthreads();

    v4f acc[R][NT] = {};
    int now = 0;  // the stage's buffer
    // every workgroup's waves take as many rounds, so that they meet at the barriers
    const int64_t turns = (groups + per - 1) / per;
    for (int64_t turn = blockIdx.x; turn < turns; turn += gridDim.x) {
        const int64_t mine = group;
        // fetched before the chunks: loads come back in order, and at a tile's end this one would wait for all of
        // the next tile's (and where the compiler sees it pending, so would every round)
        float bias[R] = {};
        if (a.bias) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t n = group_at(mine) * (16 * R) + 16 * r + (lane & 15);
                bias[r] = a.bias[n < a.N ? n : a.N - 1];
            }
        }
        for (int round = 0; round < rounds; ++round) {
            const bool last = round + 1 == rounds;
            const bool more = !last || turn + gridDim.x < turns;
            v4u raw[XD == MOE_X_F32 && !ALL ? PIECES : 1][2];
            const int k_next = last ? 0 : (round + 1) * a.kc;
            if constexpr (!ALL) {
                // the next stage goes into the other buffer, which nobody reads since the last barrier
                char* other = smem + (now ^ 1) * stage_bytes;
                if (more) {
                    if constexpr (XD == MOE_X_BF16) {
                        St{other, stage_bytes}.fetch(a, t0, k_next, wave * 64, NW * 64, pieces);
                    } else {
#pragma unroll
                        for (int i = 0; i < PIECES; ++i) {
                            if (tid + i * 64 * NW >= pieces) break;
                            const v4u* p = reinterpret_cast<const v4u*>(St::source(a, t0, k_next, tid + i * 64 * NW));
                            raw[i][0] = p[0], raw[i][1] = p[1];
                        }
                    }
                }
            }
            if (last) {  // the loads go on with the next group
                group += (int64_t)gridDim.x * per;
                const int64_t g = group_at(group);
                rows = Rows<G, R>(a, g * (16 * R), lane);
                codes = reinterpret_cast<const char*>(a.wq) + g * (16 * R) * (a.K / 2);
                scales = reinterpret_cast<const char*>(a.scales) + g * (16 * R) * (a.K / G) * 2;
            }
            const int next = last ? 0 : round + 1;
            const char* x = smem + (ALL ? 0 : now * stage_bytes);
            const int u0 = round * D * a.wk + wk, k0 = ALL ? 0 : round * a.kc;
            const int plane = stage_bytes / PLANES<XD>;
#pragma unroll
            for (int i = 0; i < D; ++i) {
                // the load goes out before the product of the unit it replaces; left to itself the compiler
                // lets it wait for free registers
                const Chunks<G, R, EVEN> cur(buf[i]);
                buf[i].load(a, codes, scales, rows, unit_at(next, i), units);
                __builtin_amdgcn_sched_barrier(0);
                const int c = 2 * (u0 + i * a.wk);
                const char* at = x + (4 * c - k0 / 32) * St::BLOCK;
                if (c < chunks) multiply<XD, G, NT, TP, R>(cur.w[0], cur.scale[0], at + at0, at + at1, plane, acc);
                at += 4 * St::BLOCK;
                if (c + 1 < chunks) multiply<XD, G, NT, TP, R>(cur.w[1], cur.scale[1], at + at0, at + at1, plane, acc);
            }
            if constexpr (!ALL) {
                if constexpr (XD == MOE_X_F32) {
                    if (more) {
                        const St st{smem + (now ^ 1) * stage_bytes, plane};
#pragma unroll
                        for (int i = 0; i < PIECES; ++i)
                            if (tid + i * 64 * NW < pieces) st.put(tid + i * 64 * NW, raw[i]);
                    }
                } else {
                    __builtin_amdgcn_s_waitcnt(0x0F70);
                }
                __syncthreads();
                now ^= 1;
            }
        }
        store_tile<NT, R>(a, smem + (ALL ? 1 : 2) * stage_bytes, mine, groups, t0, t_end, wk, wave, lane, bias, acc);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[r][nt] = v4f{};
    }
}

// Many tokens of bf16: a workgroup of NW waves takes NT token tiles against
// NW * R row tiles, a unit of 256 inputs at a time in two buffers, codes and x
// both brought into LDS by direct loads, which take no registers while they are
// on their way.
//  - Codes: each wave's own R * 16 rows of 128 bytes, the 16-byte pieces of row i
//    turned (xor) by i / 2 % 8; x: rows of 512 bytes, the pieces of token t turned
//    by t % 16.  A load instruction takes whole lines, and the lanes of a read lie
//    in different banks.
//  - A quarter of the wave supplies eight inputs in a row, 16 bytes of x, against
//    the low or the high nibbles of 8 bytes of codes.
//  - The corrections -8 * (sum of x over a group) are computed once per workgroup:
//    each wave one (chunk, token tile) of the unit, and go into the products as
//    their C.
// 64 x 131072 x 4096 in groups of 128: 102 us, 670 TFLOP/s; 61 us without the
// products and the stores, 78 us with the same few lines loaded over and over.  A
// unit takes 5400 clocks of its CU: x from LDS eight times over 2560, products
// 2176, vector instructions 1870, two barriers; they overlap in part.  Four row
// tiles a wave would read half of that LDS: in eight waves 45 registers are
// spilled (121 us), in four nobody fills the waits (113 us).
template <int G, int NT, int R, bool EVEN, int NW>
struct Tile {
    static constexpr int ROWS = NW * R * 16;
    static constexpr int CODES = ROWS * (UNIT / 2), X = NT * 16 * UNIT * 2, STAGE = CODES + X;
    static constexpr int NS = CH / G;
    static constexpr int CORR = 2 * NS * NT * 16 * 4;
    static constexpr size_t LDS = 2 * STAGE + CORR;
    static_assert(2 * NT <= NW, "one (chunk, token tile) a wave");
};

template <int G, int NT, int R, bool EVEN, int NW>
__global__ void __launch_bounds__(64 * NW) k_linear_q4_tile(LinArgs a) {
    using Ti = Tile<G, NT, R, EVEN, NW>;
    constexpr int NS = Ti::NS, BG = G / 32;
    typedef __attribute__((address_space(1))) const void* gptr;
    typedef __attribute__((address_space(3))) void* lptr;
    extern __shared__ __align__(16) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), q = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.y * (16 * NT);
    const int64_t tiles = ((int64_t)a.N + Ti::ROWS - 1) / Ti::ROWS;
    const int units = (a.K + UNIT - 1) / UNIT;
    const int64_t wrow = (int64_t)wave * (R * 16);  // of the tile
    // rows from N on read the last row, in whatever wave they are
    const auto first_row = [&](int64_t tile) {
        const int64_t n = tile * Ti::ROWS + wrow;
        return n < a.N ? n : (int64_t)a.N - 1;
    };
    // What this lane brings: pieces of the wave's rows of codes (offsets from the first row's start, those of the
    // row's last unit besides) and of tokens (addresses of their starts, pieces).
    constexpr int XJ = NT * 8 / NW;
    uint32_t code[2 * R], code_end[2 * R];
    const auto code_rows = [&](int64_t n0) {
        const int nb = a.K >> 5, end = (nb - 1) % 8;
#pragma unroll
        for (int j = 0; j < 2 * R; ++j) {
            const int i = 8 * j + (lane >> 3), piece = (lane & 7) ^ ((i >> 1) & 7);
            const uint32_t at = (uint32_t)(n0 + i < a.N ? i : (int)(a.N - 1 - n0)) * nb * 16;
            code[j] = at + 16 * piece, code_end[j] = at + 16 * (piece < end ? piece : end);
        }
    };
    const char* xrow[XJ];
    int xk[XJ];
#pragma unroll
    for (int j = 0; j < XJ; ++j) {
        const int tok = (wave * XJ + j) * 2 + (lane >> 5);
        xrow[j] = reinterpret_cast<const char*>(a.x) + (t0 + tok < a.T ? t0 + tok : a.T - 1) * a.ldx * 2;
        xk[j] = 16 * ((lane & 31) ^ (tok & 15));
    }
    // bring unit u of the rows from n0 on, of x into buffer b
    const auto whole = [&](int u) { return EVEN || u + 1 < units || a.K % UNIT == 0; };
    const auto fetch_codes = [&](int64_t n0, int u, int b, uint32_t mask) {
        const char* from = reinterpret_cast<const char*>(a.wq) + n0 * (a.K / 2) + (int64_t)u * (UNIT / 2);
        char* to = smem + b * Ti::STAGE + wave * (R * 16 * 128);
#pragma unroll
        for (int j = 0; j < 2 * R; ++j)
            __builtin_amdgcn_global_load_lds((gptr)(from + ((whole(u) ? code[j] : code_end[j]) & mask)),
                                             (lptr)(to + j * 1024), 16, 0, 0);
    };
    const auto fetch_x = [&](int u, int b) {
        char* to = smem + b * Ti::STAGE + Ti::CODES + wave * (XJ * 1024);
#pragma unroll
        for (int j = 0; j < XJ; ++j) {
            int k = xk[j] + u * (UNIT * 2);
            if (!whole(u) && k >= 2 * a.K) k = 2 * a.K - 16;
            __builtin_amdgcn_global_load_lds((gptr)(xrow[j] + k), (lptr)(to + j * 1024), 16, 0, 0);
        }
    };

    // This lane's reads: code piece and x piece of a chunk's first product (the others are an xor away).  Groups of
    // two blocks and more: a pair of products takes 8 bytes of two blocks, the low and the high nibbles; else a product
    // takes one block, its quarters the low (q < 2) or the high nibbles.
    constexpr int CB = BG >= 2 ? 2 : 4;  // code reads of a chunk
    const int row16 = lane & 15;
    const int code_at = wave * (R * 16 * 128) + row16 * 128 + (((CB == 2 ? q >> 1 : 0) ^ ((row16 >> 1) & 7)) * 16) + (q & 1) * 8;
    const int x_at = Ti::CODES + row16 * 512 + (((CB == 2 ? 4 * (q >> 1) + (q & 1) : q) ^ row16) * 16);
    const auto x_block = [](int i) { return CB == 2 ? (i >> 1) * 128 + (i & 1) * 32 : i * 64; };
    const int shift = (q >> 1) * 4;
    float* corr = reinterpret_cast<float*>(smem + 2 * Ti::STAGE);
    constexpr uint32_t M8 = 0xC100C100u;  // bf16 -8 twice
    const bf16x8 minus8 = __builtin_bit_cast(bf16x8, v4u{M8, M8, M8, M8});

    // A unit's codes are asked for two units ahead, its scales and x one ahead: behind the last unit too (the codes
    // then one piece for all lanes), so that the number of loads on their way is known.
    int64_t tile = blockIdx.x, code_tile = tile;
    int code_u = 0;
    const auto ask_codes = [&](int b) {
        const bool more = code_tile < tiles;
        const int64_t n0 = first_row(more ? code_tile : 0);
        if (code_u == 0) code_rows(n0);
        fetch_codes(n0, code_u, b, more ? ~0u : 0u);
        if (++code_u == units) code_u = 0, code_tile += gridDim.x;
    };
    Rows<G, R> rows(a, first_row(tile), lane);
    const char* scales = reinterpret_cast<const char*>(a.scales) + first_row(tile) * (a.K / G) * 2;
    Scales<G, R, EVEN> loaded;
    loaded.load(a, scales, rows, 0);
    // (asked for with the scales, before the tile: with loads of the next unit behind it alone, each store would wait
    // for those)
    float next_bias[R] = {};
    const auto ask_bias = [&](int64_t t) {
        if (a.bias) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t n = t * Ti::ROWS + wrow + 16 * r + row16;
                next_bias[r] = a.bias[n < a.N ? n : (int64_t)a.N - 1];
            }
        }
    };
    ask_bias(tile);
    ask_codes(0);
    fetch_x(0, 0);
    __builtin_amdgcn_sched_barrier(0);  // the codes waited for last go out last
    ask_codes(1);
    // Waits for the next unit, all but the 2 R loads of the one behind it: at a unit's end, so that the stores of a tile
    // go out after the wait and have a unit's time.
    float scale[2][R][NS];
    const auto arrive = [&] {
        __builtin_amdgcn_s_waitcnt(0x0F70 | 2 * R);
        loaded.take(scale);
    };
    arrive();
    int now = 0;
    for (; tile < tiles; tile += gridDim.x) {
        const int64_t n0 = tile * Ti::ROWS + wrow;
        float bias[R];
#pragma unroll
        for (int r = 0; r < R; ++r) bias[r] = next_bias[r];
        v4f acc[R][NT] = {};
        int u = 0;
        do {
            // the unit is there, of every wave, and nobody reads the other buffer of x any more (__syncthreads would
            // wait for all loads)
            asm volatile("s_barrier" ::: "memory");
            const bool last = u + 1 == units;
            if (last) {
                const int64_t to = tile + gridDim.x < tiles ? tile + gridDim.x : tile, next = first_row(to);
                ask_bias(to);
                rows = Rows<G, R>(a, next, lane);
                scales = reinterpret_cast<const char*>(a.scales) + next * (a.K / G) * 2;
            }
            loaded.load(a, scales, rows, last ? 0 : u + 1);
            fetch_x(last ? 0 : u + 1, now ^ 1);
            __builtin_amdgcn_sched_barrier(0);
            const char* stage = smem + now * Ti::STAGE;
            // A step is a chunk's token tile.  Its reads go out a step ahead, and what it adds up, and the second
            // chunk's codes as bf16, lie between the products (groups of one block have no registers for all of that:
            // their corrections are read in the step, the second chunk's codes taken at its start).
            const auto x_of = [&](int step, bf16x8(&x)[4]) {
                const int h = step / NT, nt = step % NT;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[i] = *reinterpret_cast<const bf16x8*>(stage + (x_at ^ x_block(i)) + nt * 8192 + h * 256);
            };
            const auto corr_of = [&](int step, v4f(&c)[NS]) {
                const int h = step / NT, nt = step % NT;
#pragma unroll
                for (int g = 0; g < NS; ++g)
                    c[g] = *reinterpret_cast<const v4f*>(corr + ((h * NS + g) * NT + nt) * 16 + 4 * q);
            };
            v2u w[2][CB][R];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < CB; ++i)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        w[h][i][r] = *reinterpret_cast<const v2u*>(stage + (code_at ^ ((4 * h + 4 / CB * i) * 16)) + r * 2048);
            bf16x8 b[2][4][R];
            const auto unpack = [&](int h, int i) {  // the codes of chunk h that product i takes
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const v2u v = w[h][CB == 4 ? i : i / 2][r];
                    const int by = CB == 4 ? shift : 4 * (i % 2);
                    b[h][i][r] = bytes_bf16((v[0] >> by) & 0x0F0F0F0Fu, (v[1] >> by) & 0x0F0F0F0Fu);
                }
            };
            if (wave < 2 * NT) {
                bf16x8 mine[4];
                x_of(wave, mine);
                v4f sum[NS];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum[i / BG] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mine[i], minus8, i % BG ? sum[i / BG] : v4f{}, 0, 0, 0);
                if (row16 == 0) {
#pragma unroll
                    for (int g = 0; g < NS; ++g)
                        *reinterpret_cast<v4f*>(corr + ((wave / NT * NS + g) * NT + wave % NT) * 16 + 4 * q) = sum[g];
                }
            }
            bf16x8 x[2][4];
            v4f c[2][NS], d[2][NS][R];
            x_of(0, x[0]);
#pragma unroll
            for (int i = 0; i < 4; ++i) unpack(0, i);
            __builtin_amdgcn_sched_barrier(0);
            // the corrections are there, the codes out of their buffer
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            ask_codes(now);
            if (CB == 2) corr_of(0, c[0]);
            __builtin_amdgcn_sched_barrier(0);
            const auto add_up = [&](int step) {
                const int h = step / NT, nt = step % NT;
#pragma unroll
                for (int g = 0; g < NS; ++g)
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[r][nt][e] = fmaf(scale[h][r][g], d[step & 1][g][r][e], acc[r][nt][e]);
            };
#pragma unroll
            for (int step = 0; step < 2 * NT; ++step) {
                const int h = step / NT;
                if (step + 1 < 2 * NT) x_of(step + 1, x[(step + 1) & 1]);
                if (CB == 4) corr_of(step, c[step & 1]);
                else if (step + 1 < 2 * NT) corr_of(step + 1, c[(step + 1) & 1]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (CB == 4 ? step == NT : h == 0 && i * NT / 4 == step) unpack(1, i);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        d[step & 1][i / BG][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            x[step & 1][i], b[h][i][r], i % BG == 0 ? c[step & 1][i / BG] : d[step & 1][i / BG][r], 0, 0, 0);
                if (CB == 4) add_up(step);
                else if (step) add_up(step - 1);
                __builtin_amdgcn_sched_group_barrier(0x100, 4 + NS, 0);  // LDS reads
#pragma unroll
                for (int i = 0; i < 4 * R; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);  // a product
                    __builtin_amdgcn_sched_group_barrier(0x2, 3, 0);  // vector instructions
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (CB == 2) add_up(2 * NT - 1);
            __builtin_amdgcn_sched_barrier(0);
            arrive();
            now ^= 1;
        } while (++u < units);
        store_rows<NT, R>(a, n0, t0, a.T, lane, bias, acc);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // nothing may come into LDS after the workgroup's end
}

constexpr size_t LDS_MAX = 160 << 10;

// More than 64 KB of LDS for `kern` is asked for once per kernel (`asked`: its
// devices) and device.
int ask_lds(const void* kern, size_t lds, std::atomic<uint64_t>& asked) {
    if (lds <= 64 << 10) return moe_ok();
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess && !(dev < 64 && (asked.load() >> dev & 1))) {
        e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)LDS_MAX);
        if (e == hipSuccess && dev < 64) asked.fetch_or((uint64_t)1 << dev);
    }
    if (e != hipSuccess) return moe_fail(MOE_E_HIP, "moe_linear_q4: %zu bytes of LDS: %s", lds, hipGetErrorString(e));
    return moe_ok();
}

template <int XD, int G, int NT, int TP, int R, int D, bool ALL, bool EVEN, int NW>
int launch(LinArgs a, hipStream_t st) {
    using St = Stage<XD, NT, TP>;
    const auto kern = k_linear_q4<XD, G, NT, TP, R, D, ALL, EVEN, NW>;
    const int units = (a.K + UNIT - 1) / UNIT;
    // row groups enough for the card go to waves of their own; fewer share
    // their inputs among several waves
    const int64_t groups = ((int64_t)a.N + 16 * R - 1) / (16 * R), tiles = ((int64_t)a.T + St::TOKS - 1) / St::TOKS;
    a.wk = 1;
    while (a.wk < NW && a.wk * 2 <= units && groups * tiles * a.wk < 2048 &&
           (ALL || 2 * St::bytes(UNIT * D * a.wk * 2) + (size_t)NW * R * NT * 1024 <= LDS_MAX) &&
           (ALL || XD == MOE_X_BF16 || UNIT * D * a.wk * 2 / 32 * St::TOKS * 4 <= PIECES * 64 * NW))
        a.wk *= 2;
    a.kc = ALL ? (a.K + CH - 1) / CH * CH : UNIT * D * a.wk;
    const size_t lds = (ALL ? 1 : 2) * St::bytes(a.kc) + (a.wk > 1 ? (size_t)NW * R * NT * 1024 : 0);
    static std::atomic<uint64_t> asked{0};
    const int rc = ask_lds(reinterpret_cast<const void*>(kern), lds, asked);
    if (rc != MOE_OK) return rc;
    // with x staged once, workgroups stay: as many as the card holds at a time, the same number for each tile of
    // tokens.  That number is cut down, so that with many tiles CUs may idle: fp32, 4096 rows, 4096 tokens 618 us (128
    // tiles, 2 each), 4097 tokens 1213 us (129 tiles, 1 each).
    const int per = NW / a.wk;
    int64_t blocks = (groups + per - 1) / per;
    const int64_t most = 256 * (lds > 80 << 10 ? 1 : 2);
    if (blocks * tiles > most) blocks = tiles >= most ? 1 : most / tiles;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks, (unsigned)tiles), dim3(64 * NW), lds, st, a);
    return moe_check_launch("moe_linear_q4");
}

template <int G, int NT, bool EVEN>
int launch_tile(const LinArgs& a, hipStream_t st) {
    using Ti = Tile<G, NT, 2, EVEN, 8>;
    static_assert(Ti::LDS <= LDS_MAX, "LDS");
    const auto kern = k_linear_q4_tile<G, NT, 2, EVEN, 8>;
    static std::atomic<uint64_t> asked{0};
    const int rc = ask_lds(reinterpret_cast<const void*>(kern), Ti::LDS, asked);
    if (rc != MOE_OK) return rc;
    const int64_t tiles = ((int64_t)a.T + 16 * NT - 1) / (16 * NT);
    int64_t blocks = ((int64_t)a.N + Ti::ROWS - 1) / Ti::ROWS;
    // one workgroup a CU, the same number for each tile of tokens, cut down: 8192 tokens by 4096 x 4096 378 us (128
    // tiles, 2 each, 727 TFLOP/s), 8193 tokens 625 us (129 tiles, 1 each: half of the CUs idle)
    if (blocks * tiles > 256) blocks = tiles >= 256 ? 1 : 256 / tiles;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks, (unsigned)tiles), dim3(512), Ti::LDS, st, a);
    return moe_check_launch("moe_linear_q4");
}

template <int XD, int G, bool EVEN>
int pick(const LinArgs& a, hipStream_t st) {
    const int pad = (a.K + CH - 1) / CH * CH;
    // x whole in LDS: as long as two workgroups share a CU, and bf16 as long as one has room (8 x 4000 x 6144: 8.5 us,
    // in stages 10 us; 5 x 20000 x 8192 33 and 40 us; but fp32, 8 x 40000 x 2688: 59 and 49 us)
    const size_t most = XD == MOE_X_BF16 ? 128 << 10 : 80 << 10;
    if (a.T == 1 && Stage<XD, 1, 1>::bytes(pad) <= most) return launch<XD, G, 1, 1, 1, 2, true, EVEN, 8>(a, st);
    if (a.T <= 4 && Stage<XD, 1, 4>::bytes(pad) <= most) return launch<XD, G, 1, 4, 1, 2, true, EVEN, 8>(a, st);
    if (a.T <= 8 && Stage<XD, 1, 8>::bytes(pad) <= most) return launch<XD, G, 1, 8, 1, 2, true, EVEN, 8>(a, st);
    // More tokens.  bf16: tiles of 64 tokens by 256 rows or of 32 by 256, one a CU at a time, of which the first take
    // half as long again (2.6 and 1.75 us a unit): whichever ends sooner (131072 x 4096: 64 tokens 102 and 124 us, 32
    // tokens 96 and 75 us), as long as half the CUs get one (64 x 24576 x 4096: 32 us, by 16 tokens a wave 48; 64 x
    // 8192 x 4096: 28 and 18).  fp32: tiles of 32 by 256 where every CU gets one (32 x 65536 x 2048: 51 us, by 16 tokens
    // 63; 64 x 16384 x 2048: 41 and 33), although all forms of that kernel spill 4 to 19 vector registers.  Else 16 tokens
    // by 16 rows a wave, the codes read again for each 16 tokens.
    if (a.T > 16) {
        const int64_t by64 = ((int64_t)a.N + 255) / 256 * ((a.T + 63) / 64), by32 = ((int64_t)a.N + 255) / 256 * ((a.T + 31) / 32);
        if constexpr (XD == MOE_X_BF16) {
            if (by32 >= 128) {
                if (3 * ((by64 + 255) / 256) <= 2 * ((by32 + 255) / 256)) return launch_tile<G, 4, EVEN>(a, st);
                return launch_tile<G, 2, EVEN>(a, st);
            }
        } else if (by32 >= 256) {
            return launch<XD, G, 2, 16, 2, 1, false, EVEN, 8>(a, st);
        }
    }
    if (Stage<XD, 1, 16>::bytes(pad) <= 128 << 10) return launch<XD, G, 1, 16, 1, 2, true, EVEN, 8>(a, st);
    if constexpr (XD == MOE_X_F32) {
        // Long rows of fp32: the fewer tokens a stage holds, the more inputs, and the more waves share a row tile; each
        // tile of tokens reads the codes again.  By 4, 8 and 16 tokens: 16 x 300 x 8192 13, 21 and 39 us; 16 x 2000 x
        // 8192 24, 23 and 40 us; 64 x 2000 x 8192 53, 43 and 43 us; 64 x 8192 x 4096 97, 54 and 39 us.
        const int64_t groups = ((int64_t)a.N + 15) / 16;
        if (a.T <= 4 || groups * ((a.T + 3) / 4) <= 256) return launch<XD, G, 1, 4, 1, 1, false, EVEN, 8>(a, st);
        if (a.T <= 8 || groups * ((a.T + 7) / 8) <= 1024) return launch<XD, G, 1, 8, 1, 1, false, EVEN, 8>(a, st);
    }
    return launch<XD, G, 1, 16, 1, 1, false, EVEN, 8>(a, st);
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
        const bool even = K % UNIT == 0 && reinterpret_cast<uintptr_t>(scales) % (2 * UNIT / group) == 0;
        const auto by_group = [&](auto g) {
            constexpr int G = decltype(g)::value;
            return even ? pick<XD, G, true>(a, stream) : pick<XD, G, false>(a, stream);
        };
        return group == 32   ? by_group(std::integral_constant<int, 32>{})
               : group == 64 ? by_group(std::integral_constant<int, 64>{})
                             : by_group(std::integral_constant<int, 128>{});
    };
    return x_dtype == MOE_X_F32 ? go(std::integral_constant<int, MOE_X_F32>{})
                                : go(std::integral_constant<int, MOE_X_BF16>{});
}
