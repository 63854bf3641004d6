// One token id for each row of logits, from a given random number.
//
// With m the row's largest logit and w_i = exp((l_i - m) / temperature), the
// candidates are the logits above -inf.  Three cuts follow one another, each
// keeping a prefix of the order (logit falling, then id rising):
//   min-p  w_i >= min_p
//   top-k  the first k of what min-p left
//   top-p  the shortest prefix of what is left whose mass reaches top_p times
//          the mass of what is left
// and the draw takes, in ascending id, the first kept token whose running
// mass exceeds u times the kept mass Z.
//
// Masses are whole numbers: w_i, computed in double, rounded to a multiple of
// 2^-S with S = 62 - ceil(log2 V) (51 at most), so a row's mass stays below
// 2^63.  Sums of whole numbers do not depend on their order: the result is one
// of the inputs alone, with integer atomics wherever they are handy.
//
// What is kept is always a prefix, so one pair (key, id) says it, and no row
// is ever sorted.  A row is cut into BINS of equal width in the logit (over
// the span where masses are not 0); counts and masses per bin tell in which
// bin a cut falls, and only the ids of those bins (a few hundred, whatever the
// row) are listed and searched for the place.
//   rows of up to ROW_MAX ids   one workgroup a row, the row in LDS
//   longer rows                 k_top (largest and smallest candidate of each
//                               segment of 1024 ids) -> k_bins (counts and
//                               masses per bin) -> k_list (ids of the cut bins,
//                               mass of each segment above them) -> k_draw (one
//                               workgroup a row: the cuts, the draw's segment,
//                               the draw)
// A row whose cut bins hold more than LIST ids takes a radix selection instead,
// eight bits of the logit's key a pass over the whole row by one workgroup: the
// same result, but 1.8 ms for a row of 131072 and 2.2 ms for 64 of them, against 26
// and 58 us.  Many equal logits lead there, or one far outlier under a high
// temperature; so may bf16 logits far from 0, where a step is wide (131072 of
// spread 2 around 24 lie on steps of 1/8, some 3000 on each: any top-p whose cut
// falls among the many).
//
// 64 x 131072 fp32: k_top 7.5 us (4.5 TB/s), k_bins 17, k_list 13.5, k_draw 11.7 us;
// k_bins and k_list are bound by the vector unit (a mass costs about 24 double
// instructions; 200 and 140 for 256 ids, 225 in both with bf16 and top-p, the unit
// busy for 64 to 88 hundredths of the time), k_draw and a single row (3 + 5.5 + 7 +
// 6.7 us) by the steps that wait for one another.  17 x 5003 bf16 in k_row: 15.5 us,
// about 25 barriers.
#include <math.h>

#include <type_traits>

#include "common.hpp"
#include "exp64.hpp"
#include "wave.hpp"

namespace {

using u64 = unsigned long long;
using v4u = uint32_t __attribute__((ext_vector_type(4)));
using v2u = uint32_t __attribute__((ext_vector_type(2)));

constexpr int CHUNK_NT = 256;         // threads of a workgroup of k_top, k_bins and k_list
constexpr int ROW_NT = 512;           // of k_row (17 x 5003: 256 threads 22 us, 512 15.2 us, 1024 19.9 us)
constexpr int DRAW_NT = 256;          // of k_draw (512 threads: 1 to 2 us more)
constexpr int BINS = 1024;
constexpr int LIST = 2048;            // listed ids of a longer row
constexpr int ROW_LIST = 1024;        // and of a short one
constexpr int SEG = 1024;             // ids a wave takes at a time: four groups of 64 x 4
constexpr int GROUPS = SEG / 256;
constexpr int ROW_MAX = 8 * SEG;      // ids of a row one workgroup holds
constexpr int MAX_SEGS = MOE_SAMPLE_MAX_V / SEG;

// A logit as the kernels hold it: -inf for NaN and past a row's end.
using v4f = float __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float held(float l) { return fmaxf(l, -INFINITY); }

// Rising with the value; -0 and +0 alike.  Not of -inf.
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t b = __float_as_uint(l + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// An id in the order of the cuts: larger comes first.
__device__ __forceinline__ u64 entry_of(float l, int id) { return ((u64)key_of(l) << 32) | (uint32_t)~id; }
__device__ __forceinline__ float entry_value(u64 e) { return value_of((uint32_t)(e >> 32)); }
__device__ __forceinline__ int entry_id(u64 e) { return (int)~(uint32_t)e; }

struct SmpArgs {
    const void* logits;
    int64_t ldl;
    int T, V, S;
    int segs;   // segments of a row
    int share;  // segments of a wave (longer rows)
    const float* temperature;
    const float* min_p;
    const int32_t* top_k;
    const float* top_p;
    const float* u;
    int32_t* ids;
    float* prob;
};

// Where the cuts fall.  Ids of bins below `sure` are kept whatever happens
// inside the cut bins: bins p0 .. p1 (top-p; the last one is open as long as
// the mass that top-k leaves is) and bin `bk` (top-k).
struct Cuts {
    int sure, p0, p1, bk;
    u64 rank, mass_bk;  // ids of bin bk that top-k keeps; mass above bin bk (no such bin: the row's)
    u64 mass_sure;      // mass above bin p0
    u64 pad;
    __device__ __forceinline__ bool lists(int b) const { return (b >= p0 && b <= p1) || b == bk; }
    __device__ __forceinline__ bool any() const { return sure < BINS; }
};

// Per row of the workspace (longer rows).
struct Head {
    Cuts cuts;
    float top, low;  // the row's largest and smallest candidate; top -inf: none
    uint32_t listed, pad;
};

struct RowWs {
    Head* head;
    u64* bin_mass;       // [BINS]
    u64* list;           // [LIST] entries
    u64* seg_mass;       // [segs] mass of the segment's ids above the cut bins
    uint32_t* bin_count;  // [BINS]
    float* seg_max;      // [segs] largest and smallest candidate
    float* seg_min;      // [segs]

    static __host__ __device__ size_t bytes(int segs) {
        return sizeof(Head) + (size_t)BINS * 12 + (size_t)LIST * 8 + (size_t)((segs + 1) & ~1) * 16;
    }
    __host__ __device__ RowWs(void* ws, int64_t row, int segs) {
        const int c = (segs + 1) & ~1;
        char* p = reinterpret_cast<char*>(ws) + row * bytes(segs);
        head = reinterpret_cast<Head*>(p);
        bin_mass = reinterpret_cast<u64*>(p + sizeof(Head));
        list = bin_mass + BINS;
        seg_mass = list + LIST;
        bin_count = reinterpret_cast<uint32_t*>(seg_mass + c);
        seg_max = reinterpret_cast<float*>(bin_count + BINS);
        seg_min = seg_max + c;
    }
};
static_assert(sizeof(Head) % 16 == 0, "rows of the workspace start on 16 bytes");

template <int LD>
__device__ __forceinline__ float load_one(const SmpArgs& a, int row, int i) {
    const int64_t at = (int64_t)row * a.ldl + i;
    if constexpr (LD == MOE_X_F32) return held(reinterpret_cast<const float*>(a.logits)[at]);
    else return held(moe::bf16_to_f32(reinterpret_cast<const uint16_t*>(a.logits)[at]));
}

// Four logits of a row as they lie in memory: rows start on any logit, which
// the wide loads allow.
template <int LD>
struct Raw {
    using U = std::conditional_t<LD == MOE_X_F32, v4u, v2u>;
    typedef U Loose __attribute__((aligned(LD == MOE_X_F32 ? 4 : 2)));
    U v;
    // Of ids i .. i + 3; past V - 4 the row's last four (V at least 4).
    __device__ __forceinline__ void load(const SmpArgs& a, int row, int i) {
        const int64_t at = (int64_t)row * a.ldl + (i < a.V - 4 ? i : a.V - 4);
        v = *reinterpret_cast<const Loose*>(reinterpret_cast<const char*>(a.logits) + at * (LD == MOE_X_F32 ? 4 : 2));
    }
    // Those of ids i .. i + 3; -inf from the row's end on.
    __device__ __forceinline__ v4f logits(const SmpArgs& a, int i) const {
        v4f k;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (LD == MOE_X_F32) k[j] = held(__uint_as_float(v[j]));
            else k[j] = held(j & 1 ? moe::bf16_hi(v[j >> 1]) : moe::bf16_lo(v[j >> 1]));
        }
        const int over = i - (a.V - 4);  // ids that the load went back by
        const float no = -INFINITY;
        if (over > 0) k = over == 1 ? v4f{k[1], k[2], k[3], no} : over == 2 ? v4f{k[2], k[3], no, no}
                        : over == 3 ? v4f{k[3], no, no, no} : v4f{no, no, no, no};
        return k;
    }
};

// Logits of ids i .. i + 3 (-inf from the row's end on).
template <int LD>
__device__ __forceinline__ v4f load_four(const SmpArgs& a, int row, int i) {
    if (a.V < 4) {
        v4f k = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        for (int j = 0; j < 4; ++j)
            if (i + j < a.V) k[j] = load_one<LD>(a, row, i + j);
        return k;
    }
    Raw<LD> r;
    r.load(a, row, i);
    return r.logits(a, i);
}

// A row's settings as they lie in memory: fetched at once, before anything waits.
struct Settings {
    float temperature, min_p, top_p, u;
    int k;
    __device__ __forceinline__ Settings(const SmpArgs& a, int row) {
        temperature = a.temperature ? a.temperature[row] : 1.0f;
        min_p = a.min_p ? a.min_p[row] : 0.0f;
        k = a.top_k ? a.top_k[row] : 0;
        top_p = a.top_p ? a.top_p[row] : 1.0f;
        u = a.u[row];
    }
};

// The mass and the bin of a logit under a row's settings.
struct Row {
    double top, least, scale, shift;
    float topf, width;  // width: bins per unit of the logit
    float p, u;
    int k;
    bool greedy, cut_k, cut_p, inf;

    __device__ __forceinline__ Row(const SmpArgs& a, const Settings& s, float top_, float low) {
        greedy = !(s.temperature > 0.0f);
        // a row with +inf: those alone, as if they were 0
        inf = top_ == INFINITY;
        topf = inf ? 0.0f : top_;
        top = topf;
        const double t = s.temperature;
        scale = 1.4426950408889634 / t;  // 1 / ln 2
        shift = 0x1.8p52 + a.S;
        // min-p's cut as a logit; masses are 0 from (S + 1) ln 2 temperatures below the top on
        double cut = -1000.0 * t;
        if (s.min_p > 0.0f) cut = log(s.min_p < 1.0f ? (double)s.min_p : 1.0) * t;
        const double zero = -(a.S + 1) * 0.6931471805599454 * t;
        least = fmax(fmax(cut, zero), -0x1p1000);
        k = s.k;
        p = s.top_p;
        u = s.u;
        cut_k = k > 0 && k < a.V;
        cut_p = p < 1.0f;
        const float span = inf ? 0.0f : fminf(topf - low, -(float)zero);
        width = span > 0.0f ? (float)BINS / span : 0.0f;
    }
    __device__ __forceinline__ float norm(float l) const { return inf ? (l == INFINITY ? 0.0f : -INFINITY) : l; }
    // 2^S exp((l - top) / temperature) to the nearest whole number; 0 for what
    // is no candidate or min-p drops.  2^y, y = n + r with |r| <= 1/2: the
    // polynomial of degree 10 through 2^r's values at the 11 Chebyshev nodes
    // (relative error below 2^-51.6, 1 at 0), with n + S, from the low word of
    // y + 1.5 * 2^52 + S, added to its exponent; added to 2^52 the result is
    // rounded into the low bits.
    __device__ __forceinline__ u64 mass(float l) const {
#pragma clang fp contract(off)
        const double d = (double)norm(l) - top;
        const double t = fma(d, scale, shift);
        const double r = fma(d, scale, shift - t);
        double p = moe::fma_s(0x1.e6063f7a40c36p-28, r, 0x1.b675bcadc429ap-24);
        p = moe::fma_s(p, r, 0x1.62bfd4776f20bp-20);
        p = moe::fma_s(p, r, 0x1.ffcb540625945p-17);
        p = moe::fma_s(p, r, 0x1.430913096fdb5p-13);
        p = moe::fma_s(p, r, 0x1.5d87fe9d7a5b2p-10);
        p = moe::fma_s(p, r, 0x1.3b2ab6fba1ddap-7);
        p = moe::fma_s(p, r, 0x1.c6b08d703ce48p-5);
        p = moe::fma_s(p, r, 0x1.ebfbdff82c598p-3);
        p = moe::fma_s(p, r, 0x1.62e42fefa3a19p-1);
        p = fma(p, r, 1.0);
        const u64 b = __builtin_bit_cast(u64, p);
        const uint32_t hi = (uint32_t)(b >> 32) + ((uint32_t)__builtin_bit_cast(u64, t) << 20);
        const double w = __builtin_bit_cast(double, (u64)(uint32_t)b | ((u64)hi << 32));
        const u64 m = __builtin_bit_cast(u64, w + 0x1p52) & ((1ull << 52) - 1);
        return d >= least ? m : 0;
    }
    // of a candidate; never falls as the logit falls: each step rounds monotonically
    __device__ __forceinline__ int bin(float l) const {
        const float b = (topf - norm(l)) * width;
        return b < (float)(BINS - 1) ? (int)b : BINS - 1;
    }
    // the mass a prefix must reach, of a mass z that is left
    __device__ __forceinline__ u64 want(u64 z) const {
        const double w = ceil((double)(p > 0.0f ? p : 0.0f) * (double)z);
        return w < 1.0 ? 1 : (u64)w < z ? (u64)w : z;
    }
    // where the draw falls in a kept mass z
    __device__ __forceinline__ u64 target(u64 z) const {
        const double f = u > 0.0f ? u < 1.0f ? u : 1.0f : 0.0f;
        const u64 t = (u64)(f * (double)z);
        return t < z ? t : z - 1;
    }
};

// ------------------------------------------------------------- block helpers

__device__ __forceinline__ u64 lane_value(u64 v, int lane) {  // lane: the same in the wave
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane), hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), lane);
    return lo | ((u64)hi << 32);
}

// Reductions and running sums over a workgroup of NT threads, one barrier
// each: they write to two halves of `at` in turn, so a half is free again once
// the other has had its barrier.
template <int NT>
struct Block {
    static constexpr int NW = NT / 64;
    u64* at;  // LDS, [2 * NW]
    int half;

    __device__ __forceinline__ explicit Block(u64* scratch) : at(scratch), half(0) {}
    __device__ __forceinline__ u64* next() {
        half ^= NW;
        return at + half;
    }
    // op(v, v) is v: a largest or smallest
    template <typename T, typename Op>
    __device__ __forceinline__ T reduce(T v, Op op) {
        T* s = reinterpret_cast<T*>(next());
        v = moe::wave_all(v, op);
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
        __syncthreads();
        if constexpr (NW <= 4) {
            v = s[0];
#pragma unroll
            for (int w = 1; w < NW; ++w) v = op(v, s[w]);
            return v;
        } else {
            return moe::wave_all(s[(threadIdx.x & 63) % NW], op);
        }
    }
    __device__ __forceinline__ u64 sum(u64 v) {
        u64* s = next();
        const int lane = threadIdx.x & 63;
        v = moe::wave_all_sum(v);
        if (lane == 0) s[threadIdx.x >> 6] = v;
        __syncthreads();
        return moe::wave_all_sum(lane < NW ? s[lane] : 0);
    }
    // the largest of a and the smallest of b
    __device__ __forceinline__ void ends(float& a, float& b) {
        float* s = reinterpret_cast<float*>(next());
        a = moe::wave_all_max(a);
        b = moe::wave_all_max(-b);
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = a, s[NW + (threadIdx.x >> 6)] = b;
        __syncthreads();
        a = moe::wave_all_max(s[(threadIdx.x & 63) % NW]);
        b = -moe::wave_all_max(s[NW + (threadIdx.x & 63) % NW]);
    }
    // inclusive, in thread order; total: of all threads
    __device__ __forceinline__ u64 scan(u64 v, u64& total) {
        u64* s = next();
        const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        v = moe::wave_upto(v);
        if (lane == 63) s[wid] = v;
        __syncthreads();
        if constexpr (NW <= 4) {
            u64 all = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                if (w == wid) v += all;
                all += s[w];
            }
            total = all;
            return v;
        } else {
            const u64 mine = lane < NW ? s[lane] : 0, upto = moe::wave_upto(mine);
            total = lane_value(upto, 63);
            return v + lane_value(upto - mine, wid);
        }
    }
};

struct UMin { __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a < b ? a : b; } };
struct U64Max { __device__ u64 operator()(u64 a, u64 b) const { return a > b ? a : b; } };
struct U64Min { __device__ u64 operator()(u64 a, u64 b) const { return a < b ? a : b; } };

__device__ __forceinline__ void finish(const SmpArgs& a, int row, int id, u64 w, u64 z) {
    a.ids[row] = id;
    if (a.prob) a.prob[row] = z ? (float)((double)w / (double)z) : 0.0f;
}

// ------------------------------------------------------ cuts: bins, then ids

// From the row's counts and masses per bin (counts only where top-k cuts,
// masses only where top-p does).  s_cuts and scratch in LDS.
template <int NT>
__device__ __forceinline__ void find_cuts(const Row& r, const uint32_t* count, const u64* mass, Cuts* s_cuts,
                                          u64* s_z, Block<NT>& block) {
    constexpr int NB = BINS / NT;  // bins a thread looks after
    const int b0 = threadIdx.x * NB;
    if (threadIdx.x == 0) {
        s_cuts->sure = BINS, s_cuts->p0 = BINS, s_cuts->p1 = -1, s_cuts->bk = -1;
        s_cuts->rank = 0, s_cuts->mass_bk = 0, s_cuts->mass_sure = 0;
    }
    u64 m[NB], before = 0, total = 0;
    if (r.cut_p) {
        u64 sum = 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) sum += m[i] = mass[b0 + i];
        before = block.scan(sum, total) - sum;
    }
    if (threadIdx.x == 0) s_z[0] = s_z[1] = s_cuts->mass_bk = total;  // the mass that top-k leaves lies between the two
    __syncthreads();
    if (r.cut_k) {
        u64 c[NB], sum = 0, all;
#pragma unroll
        for (int i = 0; i < NB; ++i) sum += c[i] = count[b0 + i];
        const u64 upto = block.scan(sum, all);
        u64 at = upto - sum, mb = before;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            if (all > (u64)r.k && at < (u64)r.k && at + c[i] >= (u64)r.k) {
                s_cuts->bk = s_cuts->sure = b0 + i;
                s_cuts->rank = (u64)r.k - at;
                s_cuts->mass_bk = mb;
                if (r.cut_p) s_z[0] = mb, s_z[1] = mb + m[i];
            }
            at += c[i];
            if (r.cut_p) mb += m[i];
        }
    }
    __syncthreads();
    if (r.cut_p) {
        const u64 lo = r.want(s_z[0] ? s_z[0] : 1), hi = r.want(s_z[1]);
        u64 mb = before;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            if (mb < lo && mb + m[i] >= lo) s_cuts->p0 = s_cuts->sure = b0 + i, s_cuts->mass_sure = mb;
            if (mb < hi && mb + m[i] >= hi) s_cuts->p1 = b0 + i;
            mb += m[i];
        }
        __syncthreads();
    }
}

// Of a wave's n entries (falling order, all different), the one that ends the
// shortest prefix whose weight reaches `want`; entries of weight 0 are not there.
__device__ __forceinline__ u64 select_lanes(u64 entry, u64 weight, int n, u64 want) {
    u64 cum = 0;
    for (int i = 0; i < n; ++i) {
        const u64 e = lane_value(entry, i), w = lane_value(weight, i);
        cum += e >= entry ? w : 0;
    }
    const unsigned long long hit = __ballot(weight && cum >= want && cum - weight < want);
    return lane_value(entry, hit ? __ffsll(hit) - 1 : 0);
}

// The entry of list[0 .. n) that ends the shortest prefix (falling order, all
// entries different) whose weight reaches `want` (at least 1, at most all of
// it); entries of weight 0 are not there.  weight(i): entry i's, of any thread.
// The span of the entries is cut into 256 by its leading bits, again and again,
// until a wave can hold what is left: a lane an entry, each summing the weights
// of the entries at least as large.
template <int NT, typename W>
__device__ __forceinline__ u64 select_list(const u64* list, int n, const W& weight, u64 want, u64* hist, u64* few,
                                           Block<NT>& block, u64* s_out, int* s_n) {
    u64 lo = ~0ull, hi = 0;
    for (int i = threadIdx.x; i < n; i += NT)
        if (weight(i)) lo = list[i] < lo ? list[i] : lo, hi = list[i] > hi ? list[i] : hi;
    lo = block.reduce(lo, U64Min());
    hi = block.reduce(hi, U64Max());
    int left = n;
    while (left > 64 && lo < hi) {
        const int top = 63 - __clzll((long long)(lo ^ hi));
        const int shift = top > 7 ? top - 7 : 0;
        const u64 base = lo >> shift & ~255ull;  // the bits above the digit, the same in all
        __syncthreads();
        for (int i = threadIdx.x; i < 256; i += NT) hist[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += NT) {
            const u64 v = list[i], w = weight(i);
            if (w && v >= lo && v <= hi) atomicAdd(&hist[v >> shift & 255], w);
        }
        __syncthreads();
        if (threadIdx.x < 64) {  // falling digits: four a lane
            u64 h[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += h[i] = hist[255 - 4 * threadIdx.x - i];
            u64 before = moe::wave_upto(sum) - sum;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (before < want && before + h[i] >= want) s_out[0] = 255 - 4 * threadIdx.x - i, s_out[1] = want - before;
                before += h[i];
            }
        }
        if (threadIdx.x == 0) *s_n = 0;
        __syncthreads();
        lo = (base | s_out[0]) << shift;
        hi = lo | ((1ull << shift) - 1);
        want = s_out[1];
        int mine = 0;
        u64 l = ~0ull, h = 0;
        for (int i = threadIdx.x; i < n; i += NT) {
            const u64 v = list[i];
            if (v >= lo && v <= hi && weight(i)) ++mine, l = v < l ? v : l, h = v > h ? v : h;
        }
        if (mine) atomicAdd(s_n, mine);
        lo = block.reduce(l, U64Min());
        hi = block.reduce(h, U64Max());
        left = *s_n;
    }
    __syncthreads();
    if (threadIdx.x == 0) *s_n = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += NT) {
        const u64 v = list[i], w = weight(i);
        if (w && v >= lo && v <= hi) {
            const int at = atomicAdd(s_n, 1);
            if (at < 64) few[at] = v, few[64 + at] = w;
        }
    }
    __syncthreads();
    n = *s_n < 64 ? *s_n : 64;
    const int lane = threadIdx.x & 63;
    return select_lanes(lane < n ? few[lane] : 0, lane < n ? few[64 + lane] : 0, n, want);
}

// The last kept entry of a row whose cut bins' ids are list[0 .. n), with their
// masses beside them.  Where a wave holds them all, each wave works it out for
// itself.
template <int NT>
__device__ __forceinline__ u64 resolve(const Row& r, const Cuts& c, int n, const u64* list,
                                       const u64* mass, u64* hist, u64* few, Block<NT>& block, u64* s_out, int* s_n) {
    u64 bound = 0, z = c.mass_bk;  // the mass that top-k leaves
    const auto in_bk = [&](u64 e) { return r.bin(entry_value(e)) == c.bk; };
    const auto left = [&](u64 want) { return want > c.mass_sure ? want - c.mass_sure : 1; };
    if (n <= 64) {
        const int lane = threadIdx.x & 63;
        const u64 e = lane < n ? list[lane] : 0;
        u64 m = lane < n ? mass[lane] : 0;
        if (c.bk >= 0) {
            const bool in = lane < n && in_bk(e);
            bound = select_lanes(e, in ? 1 : 0, n, c.rank);
            if (!r.cut_p) return bound;
            z += moe::wave_all_sum(in && e >= bound ? m : 0);
        }
        m = e >= bound ? m : 0;
        return select_lanes(e, m, n, left(r.want(z)));
    }
    if (c.bk >= 0) {
        bound = select_list<NT>(list, n, [&](int i) { return (u64)(in_bk(list[i]) ? 1 : 0); }, c.rank, hist, few, block,
                                s_out, s_n);
        if (!r.cut_p) return bound;
        u64 part = 0;
        for (int i = threadIdx.x; i < n; i += NT)
            if (list[i] >= bound && in_bk(list[i])) part += mass[i];
        z += block.sum(part);
    }
    return select_list<NT>(list, n, [&](int i) { return list[i] >= bound ? mass[i] : 0; }, left(r.want(z)), hist, few,
                           block, s_out, s_n);
}

// ------------------------------------------------ the whole row, bit by bit

// Radix selection over the row in memory: for rows whose cut bins hold more
// ids than a list.  hist: 256 u64.
template <int LD, int NT>
__device__ __attribute__((noinline)) void select_row(const SmpArgs& a, const Row& r, int row, u64* hist, u64* scratch,
                                                     u64* s_left, uint32_t* s_key, int* s_at) {
    Block<NT> block(scratch);
    __syncthreads();
    const int tid = threadIdx.x, V = a.V;
    // 0: no candidate
    const auto key_at = [&](int i) {
        const float l = load_one<LD>(a, row, i);
        return l > -INFINITY ? key_of(l) : 0u;
    };
    uint32_t tkey = 0;
    int last = V;  // kept: key > tkey, or key == tkey and id <= last
    const auto kept = [&](uint32_t kk, int i) { return kk > tkey || (kk == tkey && i <= last); };
    const auto total_of = [&](auto weight) {
        u64 v = 0;
        for (int i = tid; i < V; i += NT) {
            const uint32_t kk = key_at(i);
            if (kk && kept(kk, i)) v += weight(value_of(kk));
        }
        return block.sum(v);
    };
    // the shortest prefix whose weight reaches `want` (at least 1, at most all of it)
    const auto select = [&](auto weight, u64 want) {
        uint32_t prefix = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += NT) hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < V; i += NT) {
                const uint32_t kk = key_at(i);
                if (kk == 0 || !kept(kk, i)) continue;
                if (shift < 24 && (kk >> (shift + 8)) != (prefix >> (shift + 8))) continue;
                const u64 w = weight(value_of(kk));
                if (w) atomicAdd(&hist[(kk >> shift) & 255], w);
            }
            __syncthreads();
            if (tid == 0) {
                int d = 255;
                while (d > 0 && hist[d] < want) want -= hist[d--];
                *s_key = prefix | ((uint32_t)d << shift);
                *s_left = want;
            }
            __syncthreads();
            prefix = *s_key;
            want = *s_left;
            __syncthreads();
        }
        // how many of the equal ones: all weigh the same
        const u64 each = weight(value_of(prefix));
        u64 need = each ? (want + each - 1) / each : 0;
        int found = V;
        for (int i0 = 0; i0 < V; i0 += NT) {
            const int i = i0 + tid;
            const uint32_t kk = i < V ? key_at(i) : 0;
            const bool is = kk == prefix && kept(kk, i);
            u64 total;
            const u64 at = block.scan(is ? 1 : 0, total);
            if (tid == 0) *s_at = V;
            __syncthreads();
            if (is && at == need) *s_at = i;
            __syncthreads();
            if (*s_at < V) {
                found = *s_at;
                break;
            }
            need -= total;
        }
        tkey = prefix;
        last = found;
        __syncthreads();
    };
    const auto mass = [&](float l) { return r.mass(l); };
    const auto count = [&](float l) { return (u64)(r.mass(l) ? 1 : 0); };
    if (r.cut_k && total_of(count) > (u64)r.k) select(count, (u64)r.k);
    u64 z = total_of(mass);
    if (r.cut_p) {
        select(mass, r.want(z));
        z = total_of(mass);
    }
    u64 target = r.target(z);
    for (int i0 = 0; i0 < V; i0 += NT) {
        const int i = i0 + tid;
        const uint32_t kk = i < V ? key_at(i) : 0;
        const u64 w = kk && kept(kk, i) ? r.mass(value_of(kk)) : 0;
        u64 total;
        const u64 cum = block.scan(w, total);
        if (w && cum > target && cum - w <= target) finish(a, row, i, w, z);
        if (total > target) break;
        target -= total;
    }
}

// ------------------------------------------------------------ segments

// Where a wave's segments come from.  Lane l holds ids seg * SEG + g * 256 +
// 4 l .. + 3 of group g.
template <int LD>
struct FromRow {
    using Held = Raw<LD>;
    const SmpArgs& a;
    int row;
    __device__ __forceinline__ static int id(int seg, int g) { return seg * SEG + g * 256 + 4 * (int)(threadIdx.x & 63); }
    __device__ __forceinline__ void load(int seg, Held (&h)[GROUPS]) const {
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) h[g].load(a, row, id(seg, g));
    }
    __device__ __forceinline__ v4f logits(const Held& h, int id) const { return h.logits(a, id); }
};

// f(seg, id of the first, four logits, group) over the groups of segments first,
// first + step, ... below end, of this wave; a segment is fetched while the one
// before is worked on.  What is held moves through one register group, so f's
// code is there once.
template <typename From, typename F>
__device__ __forceinline__ void each_group(int first, int step, int end, const From& from, const F& f) {
    if (first >= end) return;
    typename From::Held next[GROUPS];
    from.load(first, next);
    for (int seg = first; seg < end; seg += step) {
        typename From::Held held[GROUPS];
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) held[g] = next[g];
        if (seg + step < end) from.load(seg + step, next);
#pragma unroll 1
        for (int g = 0; g < GROUPS; ++g) {
            const int id = seg * SEG + g * 256 + 4 * (int)(threadIdx.x & 63);
            const v4f l = from.logits(held[0], id);
#pragma unroll
            for (int i = 0; i + 1 < GROUPS; ++i) held[i] = held[i + 1];
            f(seg, id, l, g);
        }
    }
}

__device__ __forceinline__ void ends(const v4f& l, float& top, float& low) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        top = fmaxf(top, l[v]);
        low = fminf(low, l[v] > -INFINITY ? l[v] : INFINITY);
    }
}

// Counts and masses into the bins.
__device__ __forceinline__ void to_bins(const Row& r, const v4f& l, uint32_t* count, u64* mass) {
    u64 m[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) m[v] = r.mass(l[v]);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        if (m[v]) {
            const int b = r.bin(l[v]);
            if (r.cut_k) atomicAdd(&count[b], 1u);
            if (r.cut_p) atomicAdd(&mass[b], m[v]);
        }
    }
}

// Entries of the cut bins into a list of `room`; SURE: returns the mass of the
// ids above them.
template <bool SURE>
__device__ __forceinline__ u64 to_list(const Row& r, const Cuts& c, const v4f& l, int id, u64* list, int room,
                                       uint32_t* listed) {
    u64 sure = 0;
    int bin[4];
    bool any = false;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        bin[v] = r.bin(l[v]);
        any |= c.lists(bin[v]) || (SURE && bin[v] < c.sure);
    }
    if (!__any(any)) return 0;
    u64 m[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) m[v] = r.mass(l[v]);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        if (bin[v] < c.sure) {
            sure += m[v];
        } else if (m[v] && c.lists(bin[v])) {
            const uint32_t at = atomicAdd(listed, 1u);
            if (at < (uint32_t)room) list[at] = entry_of(l[v], id + v);
        }
    }
    return sure;
}

// The last kept id and its logit; id past the row and -inf: all are kept.
struct Bound {
    float value;
    int id;
    __device__ __forceinline__ explicit Bound(const SmpArgs& a) : value(-INFINITY), id(a.V) {}
    __device__ __forceinline__ explicit Bound(u64 entry) : value(entry_value(entry)), id(entry_id(entry)) {}
    __device__ __forceinline__ bool keeps(float l, int i) const { return l > value || (l == value && i <= id); }
};

// Masses of the kept of four ids, and their sum.
__device__ __forceinline__ u64 kept_masses(const Row& r, const v4f& l, int id, const Bound& bound, u64 (&m)[4]) {
    bool in[4], any = false;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        in[v] = bound.keeps(l[v], id + v);
        any |= in[v];
        m[v] = 0;
    }
    if (!__any(any)) return 0;
    u64 sum = 0;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        m[v] = r.mass(l[v]);
        m[v] = in[v] ? m[v] : 0;
        sum += m[v];
    }
    return sum;
}

// The wave's lane whose ids hold the target finishes the row.
__device__ __forceinline__ void pick(const SmpArgs& a, const Row& r, int row, const v4f& l, int id, const Bound& bound,
                                     u64 z, u64 target) {
    u64 m[4];
    const u64 sum = kept_masses(r, l, id, bound, m);
    u64 at = moe::wave_upto(sum) - sum;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        if (m[v] && at <= target && at + m[v] > target) finish(a, row, id + v, m[v], z);
        at += m[v];
    }
}

// -------------------------------------------------- rows in one workgroup

template <int LD>
__global__ void __launch_bounds__(ROW_NT) k_row(SmpArgs a) {
    constexpr int NT = ROW_NT;
    __shared__ v4f logits[ROW_MAX / 4];
    __shared__ u64 bin_mass[BINS];        // then the listed masses
    __shared__ uint32_t bin_count[BINS];  // then the search's bins and its last few
    __shared__ u64 list[ROW_LIST];
    __shared__ u64 scratch[2 * NT / 64], s_z[2], group_mass[ROW_MAX / 256];
    __shared__ Cuts cuts;
    __shared__ uint32_t s_key, s_listed;
    __shared__ int s_at;
    static_assert(ROW_LIST <= BINS && (256 + 128) * 8 <= BINS * 4, "the list's arrays fit where the bins were");
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    Block<NT> block(scratch);
    const Settings set(a, row);
    float top = -INFINITY, low = INFINITY;
    for (int i = tid; i < BINS; i += NT) bin_mass[i] = 0, bin_count[i] = 0;
    for (int i = tid; i < ROW_MAX / 256; i += NT) group_mass[i] = 0;
    if (tid == 0) s_listed = 0;
    // f(id of the first, four logits) for each group of 256 ids of this wave
    const auto groups = [&](const auto& f) {
#pragma unroll 1
        for (int i = tid; 4 * i - 4 * lane < a.V; i += NT) f(4 * i, logits[i]);
    };
    v4f held_[ROW_MAX / 4 / NT];
#pragma unroll
    for (int i = 0; i < ROW_MAX / 4 / NT; ++i)
        if (4 * (i * NT + tid - lane) < a.V) held_[i] = load_four<LD>(a, row, 4 * (i * NT + tid));
#pragma unroll
    for (int i = 0; i < ROW_MAX / 4 / NT; ++i)
        if (4 * (i * NT + tid - lane) < a.V) {
            logits[i * NT + tid] = held_[i];
            ends(held_[i], top, low);
        }
    block.ends(top, low);
    if (top == -INFINITY) {
        if (tid == 0) finish(a, row, -1, 0, 0);
        return;
    }
    const Row r(a, set, top, low);
    if (r.greedy) {
        uint32_t first = ~0u;
        groups([&](int id, const v4f& l) {
#pragma unroll
            for (int v = 3; v >= 0; --v)
                if (l[v] == top && (uint32_t)(id + v) < first) first = id + v;
        });
        first = block.reduce(first, UMin());
        if (tid == 0) finish(a, row, (int)first, 1, 1);
        return;
    }
    Bound bound(a);
    if (r.cut_k || r.cut_p) {
        groups([&](int, const v4f& l) { to_bins(r, l, bin_count, bin_mass); });
        __syncthreads();
        find_cuts<NT>(r, bin_count, bin_mass, &cuts, s_z, block);
        const Cuts c = cuts;
        if (c.any()) {
            groups([&](int id, const v4f& l) {
                to_list<false>(r, c, l, id, list, ROW_LIST, &s_listed);
            });
            __syncthreads();
            const int n = (int)s_listed;
            u64* hist = reinterpret_cast<u64*>(bin_count);
            if (n > ROW_LIST) {
                select_row<LD, NT>(a, r, row, hist, scratch, s_z, &s_key, &s_at);
                return;
            }
            for (int i = tid; i < n; i += NT) bin_mass[i] = r.mass(entry_value(list[i]));
            __syncthreads();
            bound = Bound(resolve<NT>(r, c, n, list, bin_mass, hist, hist + 256, block, s_z, &s_at));
        }
    }
    groups([&](int id, const v4f& l) {
        u64 m[4];
        const u64 all = moe::wave_all_sum(kept_masses(r, l, id, bound, m));
        if (lane == 0) group_mass[id / 256] = all;
    });
    __syncthreads();
    static_assert(ROW_MAX / 256 <= 64, "a lane a group");
    const u64 mine = lane < ROW_MAX / 256 ? group_mass[lane] : 0;
    const u64 upto = moe::wave_upto(mine), z = __shfl(upto, 63, moe::WAVE), target = r.target(z);
    const unsigned long long hit = __ballot(mine && upto > target);
    const int g = hit ? __ffsll(hit) - 1 : 0;
    const u64 before = __shfl(upto - mine, g, moe::WAVE);
    if (wid == 0) pick(a, r, row, logits[g * 64 + lane], g * 256 + 4 * lane, bound, z, target - before);
}

// -------------------------------------------------------------- longer rows

// This wave's segments.
__device__ __forceinline__ int first_seg(const SmpArgs& a) {
    return ((int)blockIdx.x * (CHUNK_NT / 64) + (int)(threadIdx.x >> 6)) * a.share;
}
__device__ __forceinline__ int end_seg(const SmpArgs& a) {
    const int e = first_seg(a) + a.share;
    return e < a.segs ? e : a.segs;
}

template <int LD>
__global__ void __launch_bounds__(CHUNK_NT) k_top(SmpArgs a, void* ws) {
    const int row = blockIdx.y, lane = threadIdx.x & 63;
    const RowWs w(ws, row, a.segs);
    for (int i = blockIdx.x * CHUNK_NT + threadIdx.x; i < BINS; i += gridDim.x * CHUNK_NT) w.bin_mass[i] = 0, w.bin_count[i] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) w.head->listed = 0;
    float top = -INFINITY, low = INFINITY;
    each_group(first_seg(a), 1, end_seg(a), FromRow<LD>{a, row}, [&](int seg, int, const v4f& l, int g) {
        ends(l, top, low);
        if (g + 1 < GROUPS) return;
        top = moe::wave_all_max(top);
        low = -moe::wave_all_max(-low);
        if (lane == 0) w.seg_max[seg] = top, w.seg_min[seg] = low;
        top = -INFINITY, low = INFINITY;
    });
}

template <int LD>
__global__ void __launch_bounds__(CHUNK_NT) k_bins(SmpArgs a, void* ws) {
    constexpr int NT = CHUNK_NT;
    __shared__ u64 bin_mass[BINS];
    __shared__ uint32_t bin_count[BINS];
    __shared__ u64 scratch[2 * NT / 64];
    const int row = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
    const RowWs w(ws, row, a.segs);
    Block<NT> block(scratch);
    const Settings set(a, row);
    const FromRow<LD> load{a, row};
    for (int i = tid; i < BINS; i += NT) bin_mass[i] = 0, bin_count[i] = 0;
    float top = -INFINITY, low = INFINITY;
    for (int i = tid; i < a.segs; i += NT) top = fmaxf(top, w.seg_max[i]), low = fminf(low, w.seg_min[i]);
    block.ends(top, low);
    if (blockIdx.x == 0 && tid == 0) w.head->top = top, w.head->low = low;
    if (top == -INFINITY) return;
    const Row r(a, set, top, low);
    if (r.greedy) return;
    if (!r.cut_k && !r.cut_p) {
        u64 sum = 0;
        each_group(first_seg(a), 1, end_seg(a), load, [&](int seg, int, const v4f& l, int g) {
#pragma unroll
            for (int v = 0; v < 4; ++v) sum += r.mass(l[v]);
            if (g + 1 < GROUPS) return;
            sum = moe::wave_all_sum(sum);
            if (lane == 0) w.seg_mass[seg] = sum;
            sum = 0;
        });
        return;
    }
    each_group(first_seg(a), 1, end_seg(a), load, [&](int, int, const v4f& l, int) { to_bins(r, l, bin_count, bin_mass); });
    __syncthreads();
    for (int i = tid; i < BINS; i += NT) {
        if (r.cut_k && bin_count[i]) atomicAdd(&w.bin_count[i], bin_count[i]);
        if (r.cut_p && bin_mass[i]) atomicAdd(&w.bin_mass[i], bin_mass[i]);
    }
}

template <int LD>
__global__ void __launch_bounds__(CHUNK_NT) k_list(SmpArgs a, void* ws) {
    constexpr int NT = CHUNK_NT;
    __shared__ u64 list[LIST];
    __shared__ u64 scratch[2 * NT / 64], s_z[2];
    __shared__ Cuts cuts;
    __shared__ uint32_t s_listed, s_first;
    const int row = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
    const RowWs w(ws, row, a.segs);
    Block<NT> block(scratch);
    const Settings set(a, row);
    const float top = w.head->top, low = w.head->low;
    if (tid == 0) s_listed = 0;
    if (top == -INFINITY) return;
    const Row r(a, set, top, low);
    if (r.greedy || (!r.cut_k && !r.cut_p)) return;
    find_cuts<NT>(r, w.bin_count, w.bin_mass, &cuts, s_z, block);
    const Cuts c = cuts;
    if (blockIdx.x == 0 && tid == 0) w.head->cuts = c;
    u64 sure = 0;
    each_group(first_seg(a), 1, end_seg(a), FromRow<LD>{a, row},
               [&](int seg, int id, const v4f& l, int g) {
                   sure += to_list<true>(r, c, l, id, list, LIST, &s_listed);
                   if (g + 1 < GROUPS) return;
                   sure = moe::wave_all_sum(sure);
                   if (lane == 0) w.seg_mass[seg] = sure;
                   sure = 0;
               });
    __syncthreads();
    const uint32_t n = s_listed;
    if (n == 0) return;
    if (tid == 0) s_first = atomicAdd(&w.head->listed, n);  // a place for all of the workgroup's
    __syncthreads();
    if (n > LIST) return;  // too many: the count says so
    const uint32_t first = s_first;
    for (uint32_t i = tid; i < n; i += NT)
        if (first + i < LIST) w.list[first + i] = list[i];
}

template <int LD>
__global__ void __launch_bounds__(DRAW_NT) k_draw(SmpArgs a, void* ws) {
    constexpr int NT = DRAW_NT, MINE = MAX_SEGS / NT;  // segments a thread looks after
    __shared__ u64 list[LIST], list_mass[LIST], hist[256], few[128];
    __shared__ u64 seg_mass[MAX_SEGS];
    __shared__ u64 scratch[2 * NT / 64], s_z[2], group_mass[GROUPS], s_target;
    __shared__ uint32_t s_key;
    __shared__ int s_at;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const RowWs w(ws, row, a.segs);
    Block<NT> block(scratch);
    const Settings set(a, row);
    const Head head = *w.head;
    const int s0 = tid * MINE;
    u64 mass[MINE];
#pragma unroll
    for (int i = 0; i < MINE; ++i) mass[i] = s0 + i < a.segs ? w.seg_mass[s0 + i] : 0;
    const u64 entry = w.list[tid];  // the list's first, before its length is known
    if (head.top == -INFINITY) {
        if (tid == 0) finish(a, row, -1, 0, 0);
        return;
    }
    const Row r(a, set, head.top, head.low);
    if (r.greedy) {
        // the first segment that holds the largest, and the first id there
        uint32_t at = ~0u;
#pragma unroll
        for (int i = MINE - 1; i >= 0; --i)
            if (s0 + i < a.segs && w.seg_max[s0 + i] == head.top) at = s0 + i;
        at = block.reduce(at, UMin());
        const int id = (int)at * SEG + 4 * tid;
        uint32_t first = ~0u;
        if (tid < SEG / 4) {
            const v4f l = load_four<LD>(a, row, id);
#pragma unroll
            for (int v = 3; v >= 0; --v)
                if (l[v] == head.top) first = id + v;
        }
        first = block.reduce(first, UMin());
        if (tid == 0) finish(a, row, (int)first, 1, 1);
        return;
    }
    Bound bound(a);
    if ((r.cut_k || r.cut_p) && head.cuts.any()) {
        const int n = (int)head.listed;
        if (n > LIST) {
            select_row<LD, NT>(a, r, row, hist, scratch, s_z, &s_key, &s_at);
            return;
        }
#pragma unroll
        for (int i = 0; i < MINE; ++i) seg_mass[s0 + i] = mass[i];
        for (int i = tid; i < n; i += NT) {
            const u64 e = i < NT ? entry : w.list[i];
            list[i] = e;
            list_mass[i] = r.mass(entry_value(e));
        }
        __syncthreads();
        const u64 last = resolve<NT>(r, head.cuts, n, list, list_mass, hist, few, block, s_z, &s_at);
        bound = Bound(last);
        for (int i = tid; i < n; i += NT)
            if (list[i] >= last) atomicAdd(&seg_mass[entry_id(list[i]) / SEG], list_mass[i]);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MINE; ++i) mass[i] = seg_mass[s0 + i];
    }
    u64 sum = 0, z;
#pragma unroll
    for (int i = 0; i < MINE; ++i) sum += mass[i];
    u64 at = block.scan(sum, z) - sum;
    const u64 target = r.target(z);
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
        if (mass[i] && at <= target && at + mass[i] > target) s_at = s0 + i, s_target = target - at;
        at += mass[i];
    }
    __syncthreads();
    // the segment's groups, a wave each
    static_assert(GROUPS <= NT / 64, "a wave a group");
    const int id = s_at * SEG + 4 * tid;
    const u64 rest = s_target;
    v4f l;
    u64 all = 0;
    if (wid < GROUPS) {
        l = load_four<LD>(a, row, id);
        u64 m[4];
        all = moe::wave_all_sum(kept_masses(r, l, id, bound, m));
        if (lane == 0) group_mass[wid] = all;
    }
    __syncthreads();
    if (wid >= GROUPS) return;
    u64 before = 0;
    for (int g = 0; g < wid; ++g) before += group_mass[g];
    if (before <= rest && before + all > rest) pick(a, r, row, l, id, bound, z, rest - before);
}

inline int segs_of(int V) { return (V + SEG - 1) / SEG; }

template <int LD>
int run(SmpArgs a, void* ws, hipStream_t st) {
    a.segs = segs_of(a.V);
    if (a.V <= ROW_MAX) {
        hipLaunchKernelGGL(k_row<LD>, dim3(a.T), dim3(ROW_NT), 0, st, a);
        return moe_check_launch("moe_sample");
    }
    // one segment a wave, so that the CUs end together; from 16 workgroups a CU
    // on a wave takes several, so that a row's bins are gathered fewer times
    // (128 x 100003: several from 4, 8 and 16 a CU on 78, 69 and 68 us; 64 x
    // 131072: 47 to 48 us)
    const int64_t all = (int64_t)a.T * a.segs;
    const int64_t share = (all + 16384 - 1) / 16384;
    a.share = share < a.segs ? (int)share : a.segs;
    constexpr int NW = CHUNK_NT / 64;
    const dim3 grid((a.segs + NW * a.share - 1) / (NW * a.share), a.T), block(CHUNK_NT);
    hipLaunchKernelGGL(k_top<LD>, grid, block, 0, st, a, ws);
    if (int rc = moe_check_launch("moe_sample/top")) return rc;
    hipLaunchKernelGGL(k_bins<LD>, grid, block, 0, st, a, ws);
    if (int rc = moe_check_launch("moe_sample/bins")) return rc;
    if (a.top_k || a.top_p) {
        hipLaunchKernelGGL(k_list<LD>, grid, block, 0, st, a, ws);
        if (int rc = moe_check_launch("moe_sample/list")) return rc;
    }
    hipLaunchKernelGGL(k_draw<LD>, dim3(a.T), dim3(DRAW_NT), 0, st, a, ws);
    return moe_check_launch("moe_sample/draw");
}

}  // namespace

extern "C" {

size_t moe_sample_workspace_bytes(int T, int V) {
    if (T < 0 || T > MOE_SAMPLE_MAX_T || V < 1 || V > MOE_SAMPLE_MAX_V) return 0;
    if (T == 0 || V <= ROW_MAX) return 16;
    return (size_t)T * RowWs::bytes(segs_of(V));
}

int moe_sample(const void* logits, int l_dtype, int64_t ldl, int T, int V, const float* temperature,
               const float* min_p, const int32_t* top_k, const float* top_p, const float* u, int32_t* ids, float* prob,
               void* ws, size_t ws_bytes, hipStream_t stream) {
    MOE_REQUIRE(T >= 0 && V >= 1, MOE_E_ARG, "moe_sample: T=%d V=%d", T, V);
    MOE_REQUIRE(T == 0 || (logits && u && ids && ws), MOE_E_ARG, "moe_sample: logits, u, ids and ws must be non-NULL");
    MOE_REQUIRE(l_dtype == MOE_X_F32 || l_dtype == MOE_X_BF16, MOE_E_DTYPE, "moe_sample: logit format %d", l_dtype);
    MOE_REQUIRE(T <= MOE_SAMPLE_MAX_T && V <= MOE_SAMPLE_MAX_V, MOE_E_SHAPE, "moe_sample: T=%d V=%d beyond the limits",
                T, V);
    MOE_REQUIRE(ldl >= V && ldl <= MOE_SAMPLE_MAX_LD, MOE_E_ARG, "moe_sample: row stride %lld for V=%d",
                (long long)ldl, V);
    const int el = l_dtype == MOE_X_F32 ? 4 : 2;
    MOE_REQUIRE(reinterpret_cast<uintptr_t>(logits) % el == 0 && moe_aligned16(ws), MOE_E_ALIGN,
                "moe_sample: logits must be aligned to their elements, ws to 16 bytes");
    MOE_REQUIRE(ws_bytes >= moe_sample_workspace_bytes(T, V), MOE_E_ARG, "moe_sample: workspace of %zu bytes, %zu needed",
                ws_bytes, moe_sample_workspace_bytes(T, V));
    if (T == 0) return moe_ok();
    SmpArgs a{logits, ldl, T, V, 51, 0, 0, temperature, min_p, top_k, top_p, u, ids, prob};
    while (((int64_t)1 << (62 - a.S)) < V) --a.S;
    return l_dtype == MOE_X_F32 ? run<MOE_X_F32>(a, ws, stream) : run<MOE_X_BF16>(a, ws, stream);
}

}  // extern "C"
