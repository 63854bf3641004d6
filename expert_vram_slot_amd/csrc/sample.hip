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
//   rows of up to ROW_MAX ids   one workgroup a row, logits in registers
//   longer rows                 k_top (largest and smallest candidate of each
//                               chunk) -> k_bins (counts and masses per bin)
//                               -> k_list (ids of the cut bins, mass of each
//                               chunk above them) -> k_draw (one workgroup a
//                               row: the cuts, the draw's chunk, the draw)
// A row whose cut bins hold more than LIST ids (many equal logits, or one far
// outlier under a high temperature) takes a radix selection instead, eight
// bits of the logit's key a pass over the whole row: slower, the same result.
#include <math.h>

#include <type_traits>

#include "common.hpp"
#include "exp64.hpp"
#include "wave.hpp"

namespace {

using u64 = unsigned long long;
using v4u = uint32_t __attribute__((ext_vector_type(4)));
using v2u = uint32_t __attribute__((ext_vector_type(2)));

constexpr int BINS = 1024;
constexpr int LIST = 2048;
constexpr int PER = 16;               // ids a thread holds
constexpr int GROUPS = PER / 4;       // in groups of four
constexpr int ROW_MAX = 1024 * PER;   // ids of a row one workgroup holds
constexpr int MAX_CHUNKS = MOE_SAMPLE_MAX_V / (256 * PER);

// Rising with the value; -inf and NaN give 0 (not a candidate).  -0 counts as +0.
__device__ __forceinline__ uint32_t key_of(float l) {
    if (!(l > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(l + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

struct SmpArgs {
    const void* logits;
    int64_t ldl;
    int T, V, S, chunks;
    const float* temperature;
    const float* min_p;
    const int32_t* top_k;
    const float* top_p;
    const float* u;
    int32_t* ids;
    float* prob;
    int vec;  // rows start on four logits
};

// Where the cuts fall.  Ids of bins below `sure` are kept whatever happens
// inside the cut bins: bins p0 .. p1 (top-p; the last one is open as long as
// the mass that top-k leaves is) and bin `bk` (top-k).
struct Cuts {
    int sure, p0, p1, bk;
    u64 rank, mass_bk;  // ids of bin bk that top-k keeps; mass above bin bk (no such bin: the row's)
    __device__ __forceinline__ bool lists(int b) const { return (b >= p0 && b <= p1) || b == bk; }
    __device__ __forceinline__ bool any() const { return sure < BINS; }
};

// Per row of the workspace (longer rows).
struct Head {
    Cuts cuts;
    uint32_t kmax, kmin;  // keys of the row's largest and smallest candidate; kmax 0: none
    uint32_t listed, pad;
};

struct RowWs {
    Head* head;
    u64* bin_mass;       // [BINS]
    u64* list;           // [LIST] key << 32 | ~id
    u64* chunk_mass;     // [chunks] mass of the chunk's ids above the cut bins
    uint32_t* bin_count;  // [BINS]
    uint32_t* chunk_max;  // [chunks] keys
    uint32_t* chunk_min;  // [chunks]

    static __host__ __device__ size_t bytes(int chunks) {
        return sizeof(Head) + (size_t)BINS * 12 + (size_t)LIST * 8 + (size_t)((chunks + 1) & ~1) * 16;
    }
    __host__ __device__ RowWs(void* ws, int64_t row, int chunks) {
        const int c = (chunks + 1) & ~1;
        char* p = reinterpret_cast<char*>(ws) + row * bytes(chunks);
        head = reinterpret_cast<Head*>(p);
        bin_mass = reinterpret_cast<u64*>(p + sizeof(Head));
        list = bin_mass + BINS;
        chunk_mass = list + LIST;
        bin_count = reinterpret_cast<uint32_t*>(chunk_mass + c);
        chunk_max = bin_count + BINS;
        chunk_min = chunk_max + c;
    }
};
static_assert(sizeof(Head) % 16 == 0, "rows of the workspace start on 16 bytes");

template <int LD>
__device__ __forceinline__ uint32_t load_key(const SmpArgs& a, int row, int i) {
    const int64_t at = (int64_t)row * a.ldl + i;
    if constexpr (LD == MOE_X_F32) return key_of(reinterpret_cast<const float*>(a.logits)[at]);
    else return key_of(moe::bf16_to_f32(reinterpret_cast<const uint16_t*>(a.logits)[at]));
}

// Keys of ids i .. i + 3 (0 past the row).
template <int LD>
__device__ __forceinline__ v4u load_keys(const SmpArgs& a, int row, int i) {
    v4u k = {0, 0, 0, 0};
    if (a.vec && i + 3 < a.V) {
        const int64_t at = (int64_t)row * a.ldl + i;
        if constexpr (LD == MOE_X_F32) {
            const v4u v = *reinterpret_cast<const v4u*>(reinterpret_cast<const float*>(a.logits) + at);
#pragma unroll
            for (int j = 0; j < 4; ++j) k[j] = key_of(__uint_as_float(v[j]));
        } else {
            const v2u v = *reinterpret_cast<const v2u*>(reinterpret_cast<const uint16_t*>(a.logits) + at);
#pragma unroll
            for (int j = 0; j < 4; ++j) k[j] = key_of(j & 1 ? moe::bf16_hi(v[j >> 1]) : moe::bf16_lo(v[j >> 1]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < a.V) k[j] = load_key<LD>(a, row, i + j);
    }
    return k;
}

// A row's settings, and the mass and the bin of a key under them.
struct Row {
    double top, rtemp, min_p, one;
    float topf, width;  // width: bins per unit of the logit
    float p;
    uint32_t kmax;
    int k;
    bool greedy, cut_k, cut_p;

    __device__ __forceinline__ Row(const SmpArgs& a, int row, uint32_t kmax_, uint32_t kmin) {
        kmax = kmax_;
        const float temp = a.temperature ? a.temperature[row] : 1.0f;
        greedy = !(temp > 0.0f);
        topf = value_of(kmax);
        top = topf;
        rtemp = 1.0 / (double)temp;
        min_p = a.min_p ? (double)a.min_p[row] : 0.0;
        min_p = min_p > 0.0 ? fmin(min_p, 1.0) : 0.0;
        one = ldexp(1.0, a.S);
        k = a.top_k ? a.top_k[row] : 0;
        p = a.top_p ? a.top_p[row] : 1.0f;
        cut_k = k > 0 && k < a.V;
        cut_p = p < 1.0f;
        // masses are 0 from (S + 1) ln 2 temperatures below the top on
        const float span = fminf(topf - value_of(kmin), temp * ((float)(a.S + 1) * 0.6932f));
        width = span > 0.0f ? (float)BINS / span : 0.0f;
    }
    // of a candidate; 0 also for one that min-p drops
    __device__ __forceinline__ u64 mass(uint32_t key) const {
#pragma clang fp contract(off)
        double w = moe::exp64(((double)value_of(key) - top) * rtemp);
        w = key == kmax ? 1.0 : w;
        // added to 2^52 the product, at most 2^51, is rounded into the low bits
        const u64 m = __builtin_bit_cast(u64, fma(w, one, 0x1p52)) & ((1ull << 52) - 1);
        return w >= min_p ? m : 0;
    }
    // never falls as the key falls: each step rounds monotonically
    __device__ __forceinline__ int bin(uint32_t key) const {
        if (key == kmax) return 0;
        const float b = (topf - value_of(key)) * width;
        return b < (float)(BINS - 1) ? (int)b : BINS - 1;
    }
    // the mass a prefix must reach, of a mass z that is left
    __device__ __forceinline__ u64 want(u64 z) const {
        const double w = ceil((double)(p > 0.0f ? p : 0.0f) * (double)z);
        return w < 1.0 ? 1 : (u64)w < z ? (u64)w : z;
    }
};

// ------------------------------------------------------------- block helpers

// Over the block, for every thread.  scratch: NT / 64 entries, free again once
// the block has met another barrier.
template <int NT, typename T, typename Op>
__device__ __forceinline__ T block_reduce(T v, u64* scratch_, Op op) {
    T* scratch = reinterpret_cast<T*>(scratch_);
    v = moe::wave_all(v, op);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) v = op(v, scratch[w]);
    return v;
}

// Inclusive sum over the block's threads, in thread order; *total the sum of all.
template <int NT>
__device__ __forceinline__ u64 block_scan(u64 v, u64* scratch, u64* total) {
    const int wid = threadIdx.x >> 6;
    v = moe::wave_upto(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 63) scratch[wid] = v;
    __syncthreads();
    u64 all = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        if (w == wid) v += all;
        all += scratch[w];
    }
    *total = all;
    return v;
}

struct UMax { __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; } };
struct UMin { __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a < b ? a : b; } };
struct Add {
    __device__ u64 operator()(u64 a, u64 b) const { return a + b; }
};
struct U64Max { __device__ u64 operator()(u64 a, u64 b) const { return a > b ? a : b; } };
struct U64Min { __device__ u64 operator()(u64 a, u64 b) const { return a < b ? a : b; } };

__device__ __forceinline__ void finish(const SmpArgs& a, int row, int id, u64 w, u64 z) {
    a.ids[row] = id;
    if (a.prob) a.prob[row] = z ? (float)((double)w / (double)z) : 0.0f;
}

__device__ __forceinline__ u64 draw_at(const SmpArgs& a, int row, u64 z) {
    double u = a.u[row];
    u = u > 0.0 ? u < 1.0 ? u : 1.0 : 0.0;
    const u64 t = (u64)(u * (double)z);
    return t < z ? t : z - 1;
}

// ------------------------------------------------------ cuts: bins, then ids

// From the row's counts and masses per bin (counts only where top-k cuts,
// masses only where top-p does).  s_cuts and scratch in LDS.
template <int NT>
__device__ __forceinline__ void find_cuts(const Row& r, const uint32_t* count, const u64* mass, Cuts* s_cuts,
                                          u64* s_z, u64* scratch) {
    constexpr int NB = BINS / NT;
    const int b0 = threadIdx.x * NB;
    if (threadIdx.x == 0) {
        s_cuts->sure = BINS, s_cuts->p0 = BINS, s_cuts->p1 = -1, s_cuts->bk = -1;
        s_cuts->rank = 0, s_cuts->mass_bk = 0;
    }
    u64 m[NB], before = 0, total = 0;
    if (r.cut_p) {
        u64 sum = 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) sum += m[i] = mass[b0 + i];
        before = block_scan<NT>(sum, scratch, &total) - sum;
    }
    if (threadIdx.x == 0) s_z[0] = s_z[1] = total;  // the mass that top-k leaves lies between the two
    __syncthreads();
    if (r.cut_k) {
        u64 c[NB], sum = 0, all;
#pragma unroll
        for (int i = 0; i < NB; ++i) sum += c[i] = count[b0 + i];
        u64 at = block_scan<NT>(sum, scratch, &all) - sum, mb = before;
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
            if (mb < lo && mb + m[i] >= lo) s_cuts->p0 = s_cuts->sure = b0 + i;
            if (mb < hi && mb + m[i] >= hi) s_cuts->p1 = b0 + i;
            mb += m[i];
        }
        __syncthreads();
    }
}

// The entry of list[0 .. n) that ends the shortest prefix (falling order, all
// entries different) whose weight reaches `want` (at least 1, at most all of
// it); entries of weight 0 are not there.  weight(i): entry i's, of any thread.
// The span of the entries is cut into 256 by its leading bits, again and again,
// until a wave can hold what is left: a lane an entry, each summing the weights
// of the entries at least as large.
template <int NT, typename W>
__device__ __forceinline__ u64 select_list(const u64* list, int n, const W& weight, u64 want, u64* hist, u64* few,
                                           u64* scratch, u64* s_out, int* s_n) {
    u64 lo = ~0ull, hi = 0;
    for (int i = threadIdx.x; i < n; i += NT)
        if (weight(i)) lo = list[i] < lo ? list[i] : lo, hi = list[i] > hi ? list[i] : hi;
    if (n > 64) {
        lo = block_reduce<NT>(lo, scratch, U64Min());
        hi = block_reduce<NT>(hi, scratch, U64Max());
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
            lo = block_reduce<NT>(l, scratch, U64Min());
            hi = block_reduce<NT>(h, scratch, U64Max());
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
    } else {
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += NT) few[i] = list[i], few[64 + i] = weight(i);
        __syncthreads();
    }
    if (threadIdx.x < 64) {
        const u64 v = (int)threadIdx.x < n ? few[threadIdx.x] : 0, w = (int)threadIdx.x < n ? few[64 + threadIdx.x] : 0;
        u64 cum = 0;
        for (int i = 0; i < n; ++i) cum += few[i] >= v ? few[64 + i] : 0;
        if (w && cum >= want && cum - w < want) s_out[0] = v;
    }
    __syncthreads();
    const u64 out = s_out[0];
    __syncthreads();
    return out;
}

// The last kept entry of a row whose cut bins' ids are list[0 .. n), with their
// masses beside them; sure_mass: of the bins above.
template <int NT>
__device__ __forceinline__ u64 resolve(const Row& r, const Cuts& c, u64 sure_mass, int n, const u64* list,
                                       const u64* mass, u64* hist, u64* few, u64* scratch, u64* s_out, int* s_n) {
    u64 bound = 0, z = c.mass_bk;  // the mass that top-k leaves
    const auto in_bk = [&](int i) { return r.bin((uint32_t)(list[i] >> 32)) == c.bk; };
    if (c.bk >= 0) {
        bound = select_list<NT>(list, n, [&](int i) { return (u64)(in_bk(i) ? 1 : 0); }, c.rank, hist, few, scratch,
                                s_out, s_n);
        if (!r.cut_p) return bound;
        u64 part = 0;
        for (int i = threadIdx.x; i < n; i += NT)
            if (list[i] >= bound && in_bk(i)) part += mass[i];
        z += block_reduce<NT>(part, scratch, Add());
    }
    const u64 want = r.want(z);
    return select_list<NT>(list, n, [&](int i) { return list[i] >= bound ? mass[i] : 0; },
                           want > sure_mass ? want - sure_mass : 1, hist, few, scratch, s_out, s_n);
}

// ------------------------------------------------ the whole row, bit by bit

// Radix selection over the row in memory: for rows whose cut bins hold more
// ids than a list.  hist: 256 u64.
template <int LD, int NT>
__device__ __attribute__((noinline)) void select_row(const SmpArgs& a, const Row& r, int row, u64* hist, u64* scratch,
                                                     u64* s_left, uint32_t* s_key, int* s_at) {
    const int tid = threadIdx.x, V = a.V;
    uint32_t tkey = 0;
    int last = V;  // kept: key > tkey, or key == tkey and id <= last
    const auto kept = [&](uint32_t kk, int i) { return kk > tkey || (kk == tkey && i <= last); };
    const auto total_of = [&](auto weight) {
        u64 v = 0;
        for (int i = tid; i < V; i += NT) {
            const uint32_t kk = load_key<LD>(a, row, i);
            if (kk && kept(kk, i)) v += weight(kk);
        }
        return block_reduce<NT>(v, scratch, Add());
    };
    // the shortest prefix whose weight reaches `want` (at least 1, at most all of it)
    const auto select = [&](auto weight, u64 want) {
        uint32_t prefix = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += NT) hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < V; i += NT) {
                const uint32_t kk = load_key<LD>(a, row, i);
                if (kk == 0 || !kept(kk, i)) continue;
                if (shift < 24 && (kk >> (shift + 8)) != (prefix >> (shift + 8))) continue;
                const u64 w = weight(kk);
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
        const u64 each = weight(prefix);
        u64 need = each ? (want + each - 1) / each : 0;
        int found = V;
        for (int i0 = 0; i0 < V; i0 += NT) {
            const int i = i0 + tid;
            const uint32_t kk = i < V ? load_key<LD>(a, row, i) : 0;
            const bool is = kk == prefix && kept(kk, i);
            u64 total;
            const u64 at = block_scan<NT>(is ? 1 : 0, scratch, &total);
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
    const auto mass = [&](uint32_t kk) { return r.mass(kk); };
    const auto count = [&](uint32_t kk) { return (u64)(r.mass(kk) ? 1 : 0); };
    if (r.cut_k && total_of(count) > (u64)r.k) select(count, (u64)r.k);
    u64 z = total_of(mass);
    if (r.cut_p) {
        select(mass, r.want(z));
        z = total_of(mass);
    }
    u64 target = draw_at(a, row, z);
    for (int i0 = 0; i0 < V; i0 += NT) {
        const int i = i0 + tid;
        const uint32_t kk = i < V ? load_key<LD>(a, row, i) : 0;
        const u64 w = kk && kept(kk, i) ? r.mass(kk) : 0;
        u64 total;
        const u64 cum = block_scan<NT>(w, scratch, &total);
        if (w && cum > target && cum - w <= target) finish(a, row, i, w, z);
        if (total > target) break;
        target -= total;
    }
}

// ------------------------------------------------------------ the draw

// Thread's keys of group j are those of ids i0 + (j * NT + thread) * 4 .. + 3;
// a segment is a wave's part of a group: 256 ids in a row.  Finishes the row
// with the id where the running mass of the kept ids (entries from `bound` on)
// passes `target`.  WHOLE: these ids are the row; their mass is z, and the
// target is drawn from it.  seg: GROUPS * NT / 64 entries.
template <int NT, bool WHOLE>
__device__ __forceinline__ void draw(const SmpArgs& a, const Row& r, int row, int i0, const v4u (&key)[GROUPS],
                                     u64 bound, u64 z, u64 target, u64* seg) {
    constexpr int NW = NT / 64;
    const int wid = threadIdx.x >> 6;
    const auto mass = [&](int j, int v) {
        const uint32_t kk = key[j][v];
        const u64 at = ((u64)kk << 32) | (uint32_t)~(i0 + (j * NT + (int)threadIdx.x) * 4 + v);
        return kk && at >= bound ? r.mass(kk) : 0;
    };
    u64 sum[GROUPS];
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
        sum[j] = 0;
#pragma unroll
        for (int v = 0; v < 4; ++v) sum[j] += mass(j, v);
        const u64 all = moe::wave_all_sum(sum[j]);
        if ((threadIdx.x & 63) == 0) seg[j * NW + wid] = all;
    }
    __syncthreads();
    // segments are at most 64: a lane each
    const int lane = threadIdx.x & 63;
    const u64 mine = lane < GROUPS * NW ? seg[lane] : 0;
    const u64 upto = moe::wave_upto(mine);
    if constexpr (WHOLE) {
        z = __shfl(upto, 63, moe::WAVE);
        target = draw_at(a, row, z);
    }
    const unsigned long long hit = __ballot(mine && upto > target);
    const int s = hit ? __ffsll(hit) - 1 : 0;
    const u64 before = __shfl(upto - mine, s, moe::WAVE);
    if (s % NW != wid) return;
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
        if (j != s / NW) continue;
        u64 at = before + moe::wave_upto(sum[j]) - sum[j];
        if (at > target || at + sum[j] <= target) continue;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const u64 m = mass(j, v);
            if (m && at <= target && at + m > target)
                finish(a, row, i0 + (j * NT + (int)threadIdx.x) * 4 + v, m, z);
            at += m;
        }
    }
}

// A thread's share of a chunk of NT * PER ids from i0 on.
template <int LD, int NT>
__device__ __forceinline__ void load_ids(const SmpArgs& a, int row, int i0, v4u (&key)[GROUPS]) {
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) key[j] = load_keys<LD>(a, row, i0 + (j * NT + (int)threadIdx.x) * 4);
}

__device__ __forceinline__ void ends(const v4u (&key)[GROUPS], uint32_t& kmax, uint32_t& kmin) {
    kmax = 0, kmin = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < GROUPS; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            kmax = key[j][v] > kmax ? key[j][v] : kmax;
            kmin = key[j][v] && key[j][v] < kmin ? key[j][v] : kmin;
        }
}

// The lowest of a thread's ids that holds kmax (~0: none).
template <int NT>
__device__ __forceinline__ uint32_t first_top(const v4u (&key)[GROUPS], int i0, uint32_t kmax) {
    uint32_t id = ~0u;
#pragma unroll
    for (int j = GROUPS - 1; j >= 0; --j)
#pragma unroll
        for (int v = 3; v >= 0; --v)
            if (key[j][v] == kmax) id = i0 + (j * NT + (int)threadIdx.x) * 4 + v;
    return id;
}

// Counts and masses of a thread's ids into the bins.
__device__ __forceinline__ void fill_bins(const Row& r, const v4u (&key)[GROUPS], uint32_t* count, u64* mass) {
#pragma unroll
    for (int j = 0; j < GROUPS; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const uint32_t kk = key[j][v];
            const u64 m = kk ? r.mass(kk) : 0;
            if (m) {
                const int b = r.bin(kk);
                if (r.cut_k) atomicAdd(&count[b], 1u);
                if (r.cut_p) atomicAdd(&mass[b], m);
            }
        }
}

// Lists a thread's ids of the cut bins, and returns the mass of those above.
template <int NT>
__device__ __forceinline__ u64 fill_list(const Row& r, const Cuts& c, const v4u (&key)[GROUPS], int i0, u64* list,
                                         uint32_t* listed) {
    u64 sure = 0;
#pragma unroll
    for (int j = 0; j < GROUPS; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const uint32_t kk = key[j][v];
            const int b = kk ? r.bin(kk) : BINS;
            if (b >= c.sure && !c.lists(b)) continue;
            const u64 m = kk ? r.mass(kk) : 0;
            if (b < c.sure) {
                sure += m;
            } else if (m) {
                const uint32_t at = atomicAdd(listed, 1u);
                if (at < LIST) list[at] = ((u64)kk << 32) | (uint32_t)~(i0 + (j * NT + (int)threadIdx.x) * 4 + v);
            }
        }
    return sure;
}

// -------------------------------------------------- rows in one workgroup

template <int LD, int NT>
__global__ void __launch_bounds__(NT) k_row(SmpArgs a) {
    __shared__ u64 bin_mass[BINS];
    __shared__ uint32_t bin_count[BINS];
    __shared__ u64 list[LIST], list_mass[LIST], hist[256], few[128];
    __shared__ u64 scratch[NT / 64], s_z[2], seg[GROUPS * NT / 64];
    __shared__ Cuts cuts;
    __shared__ uint32_t s_key, s_listed;
    __shared__ int s_at;
    const int row = blockIdx.x, tid = threadIdx.x;
    v4u key[GROUPS];
    load_ids<LD, NT>(a, row, 0, key);
    for (int i = tid; i < BINS; i += NT) bin_mass[i] = 0, bin_count[i] = 0;
    if (tid == 0) s_listed = 0;
    uint32_t kmax, kmin;
    ends(key, kmax, kmin);
    kmax = block_reduce<NT>(kmax, scratch, UMax());
    if (kmax == 0) {
        if (tid == 0) finish(a, row, -1, 0, 0);
        return;
    }
    kmin = block_reduce<NT>(kmin, scratch, UMin());
    const Row r(a, row, kmax, kmin);
    if (r.greedy) {
        const uint32_t id = block_reduce<NT>(first_top<NT>(key, 0, kmax), scratch, UMin());
        if (tid == 0) finish(a, row, (int)id, 1, 1);
        return;
    }
    u64 bound = 0;
    if (r.cut_k || r.cut_p) {
        fill_bins(r, key, bin_count, bin_mass);
        __syncthreads();
        find_cuts<NT>(r, bin_count, bin_mass, &cuts, s_z, scratch);
        Cuts c = cuts;
        if (c.any()) {
            if (c.bk < 0) c.mass_bk = s_z[1];
            const u64 sure = block_reduce<NT>(fill_list<NT>(r, c, key, 0, list, &s_listed), scratch, Add());
            const uint32_t n = s_listed;
            if (n > LIST) {
                select_row<LD, NT>(a, r, row, hist, scratch, s_z, &s_key, &s_at);
                return;
            }
            for (int i = tid; i < (int)n; i += NT) list_mass[i] = r.mass((uint32_t)(list[i] >> 32));
            __syncthreads();
            bound = resolve<NT>(r, c, sure, (int)n, list, list_mass, hist, few, scratch, s_z, &s_at);
        }
    }
    draw<NT, true>(a, r, row, 0, key, bound, 0, 0, seg);
}

// -------------------------------------------------------------- longer rows

template <int LD, int NT>
__global__ void __launch_bounds__(NT) k_top(SmpArgs a, void* ws) {
    __shared__ u64 scratch[NT / 64];
    const int row = blockIdx.y, chunk = blockIdx.x;
    const RowWs w(ws, row, a.chunks);
    v4u key[GROUPS];
    load_ids<LD, NT>(a, row, chunk * NT * PER, key);
    for (int i = chunk * NT + threadIdx.x; i < BINS; i += a.chunks * NT) w.bin_mass[i] = 0, w.bin_count[i] = 0;
    if (chunk == 0 && threadIdx.x == 0) w.head->listed = 0;
    uint32_t kmax, kmin;
    ends(key, kmax, kmin);
    kmax = block_reduce<NT>(kmax, scratch, UMax());
    kmin = block_reduce<NT>(kmin, scratch, UMin());
    if (threadIdx.x == 0) w.chunk_max[chunk] = kmax, w.chunk_min[chunk] = kmin;
}

template <int LD, int NT>
__global__ void __launch_bounds__(NT) k_bins(SmpArgs a, void* ws) {
    static_assert(MAX_CHUNKS <= 256, "one chunk a thread");
    __shared__ u64 bin_mass[BINS];
    __shared__ uint32_t bin_count[BINS];
    __shared__ u64 scratch[NT / 64];
    const int row = blockIdx.y, chunk = blockIdx.x, tid = threadIdx.x;
    const RowWs w(ws, row, a.chunks);
    v4u key[GROUPS];
    load_ids<LD, NT>(a, row, chunk * NT * PER, key);
    for (int i = tid; i < BINS; i += NT) bin_mass[i] = 0, bin_count[i] = 0;
    const bool in = tid < a.chunks;
    const uint32_t kmax = block_reduce<NT>(in ? w.chunk_max[tid] : 0u, scratch, UMax());
    const uint32_t kmin = block_reduce<NT>(in ? w.chunk_min[tid] : 0xFFFFFFFFu, scratch, UMin());
    if (chunk == 0 && tid == 0) w.head->kmax = kmax, w.head->kmin = kmin;
    if (kmax == 0) return;
    const Row r(a, row, kmax, kmin);
    if (r.greedy) return;
    if (!r.cut_k && !r.cut_p) {
        u64 sum = 0;
#pragma unroll
        for (int j = 0; j < GROUPS; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) sum += key[j][v] ? r.mass(key[j][v]) : 0;
        sum = block_reduce<NT>(sum, scratch, Add());
        if (tid == 0) w.chunk_mass[chunk] = sum;
        return;
    }
    fill_bins(r, key, bin_count, bin_mass);
    __syncthreads();
    for (int i = tid; i < BINS; i += NT) {
        if (r.cut_k && bin_count[i]) atomicAdd(&w.bin_count[i], bin_count[i]);
        if (r.cut_p && bin_mass[i]) atomicAdd(&w.bin_mass[i], bin_mass[i]);
    }
}

template <int LD, int NT>
__global__ void __launch_bounds__(NT) k_list(SmpArgs a, void* ws) {
    __shared__ u64 scratch[NT / 64], s_z[2];
    __shared__ Cuts cuts;
    const int row = blockIdx.y, chunk = blockIdx.x;
    const RowWs w(ws, row, a.chunks);
    if (w.head->kmax == 0) return;
    const Row r(a, row, w.head->kmax, w.head->kmin);
    if (r.greedy || (!r.cut_k && !r.cut_p)) return;
    v4u key[GROUPS];
    load_ids<LD, NT>(a, row, chunk * NT * PER, key);
    find_cuts<NT>(r, w.bin_count, w.bin_mass, &cuts, s_z, scratch);
    Cuts c = cuts;
    if (c.bk < 0) c.mass_bk = s_z[1];
    if (chunk == 0 && threadIdx.x == 0) w.head->cuts = c;
    const u64 sure = block_reduce<NT>(fill_list<NT>(r, c, key, chunk * NT * PER, w.list, &w.head->listed), scratch, Add());
    if (threadIdx.x == 0) w.chunk_mass[chunk] = sure;
}

template <int LD, int NT>
__global__ void __launch_bounds__(NT) k_draw(SmpArgs a, void* ws) {
    constexpr int CHUNK = NT * PER;
    __shared__ u64 list[LIST], list_mass[LIST], hist[256], few[128];
    __shared__ u64 chunk_mass[MAX_CHUNKS];
    __shared__ u64 scratch[NT / 64], s_z[2], seg[GROUPS * NT / 64], s_target;
    __shared__ uint32_t s_key;
    __shared__ int s_at;
    const int row = blockIdx.x, tid = threadIdx.x;
    const RowWs w(ws, row, a.chunks);
    const uint32_t kmax = w.head->kmax;
    if (kmax == 0) {
        if (tid == 0) finish(a, row, -1, 0, 0);
        return;
    }
    const Row r(a, row, kmax, w.head->kmin);
    v4u key[GROUPS];
    if (r.greedy) {
        // the first chunk that holds the largest, and the first id there
        const uint32_t at = block_reduce<NT>(tid < a.chunks && w.chunk_max[tid] == kmax ? (uint32_t)tid : ~0u, scratch, UMin());
        load_ids<LD, NT>(a, row, (int)at * CHUNK, key);
        const uint32_t id = block_reduce<NT>(first_top<NT>(key, (int)at * CHUNK, kmax), scratch, UMin());
        if (tid == 0) finish(a, row, (int)id, 1, 1);
        return;
    }
    u64 mass = tid < a.chunks ? w.chunk_mass[tid] : 0;
    u64 bound = 0;
    if (r.cut_k || r.cut_p) {
        const Cuts c = w.head->cuts;
        if (c.any()) {
            const uint32_t n = w.head->listed;
            if (n > LIST) {
                select_row<LD, NT>(a, r, row, hist, scratch, s_z, &s_key, &s_at);
                return;
            }
            if (tid < MAX_CHUNKS) chunk_mass[tid] = mass;
            for (int i = tid; i < (int)n; i += NT) {
                const u64 e = w.list[i];
                list[i] = e;
                list_mass[i] = r.mass((uint32_t)(e >> 32));
            }
            const u64 sure = block_reduce<NT>(mass, scratch, Add());
            bound = resolve<NT>(r, c, sure, (int)n, list, list_mass, hist, few, scratch, s_z, &s_at);
            for (int i = tid; i < (int)n; i += NT)
                if (list[i] >= bound) atomicAdd(&chunk_mass[(uint32_t)~(uint32_t)list[i] / CHUNK], list_mass[i]);
            __syncthreads();
            if (tid < MAX_CHUNKS) mass = chunk_mass[tid];
        }
    }
    u64 z;
    const u64 upto = block_scan<NT>(mass, scratch, &z);
    const u64 target = draw_at(a, row, z);
    if (mass && upto > target && upto - mass <= target) s_at = tid, s_target = target - (upto - mass);
    __syncthreads();
    const int i0 = s_at * CHUNK;
    const u64 rest = s_target;
    load_ids<LD, NT>(a, row, i0, key);
    draw<NT, false>(a, r, row, i0, key, bound, z, rest, seg);
}

// Threads of a chunk's workgroup: few rows go to many small workgroups, many
// rows to large ones, which read a row's bins and ends once for four times the
// ids.
inline int chunk_threads(int T, int V) {
    return (int64_t)T * ((V + 256 * PER - 1) / (256 * PER)) > 1024 ? 1024 : 256;
}

inline int chunks_of(int T, int V) {
    const int ids = chunk_threads(T, V) * PER;
    return (V + ids - 1) / ids;
}

template <int LD, int NT>
int run_long(SmpArgs a, void* ws, hipStream_t st) {
    const dim3 grid(a.chunks, a.T), block(NT);
    hipLaunchKernelGGL((k_top<LD, NT>), grid, block, 0, st, a, ws);
    if (int rc = moe_check_launch("moe_sample/top")) return rc;
    hipLaunchKernelGGL((k_bins<LD, NT>), grid, block, 0, st, a, ws);
    if (int rc = moe_check_launch("moe_sample/bins")) return rc;
    if (a.top_k || a.top_p) {
        hipLaunchKernelGGL((k_list<LD, NT>), grid, block, 0, st, a, ws);
        if (int rc = moe_check_launch("moe_sample/list")) return rc;
    }
    hipLaunchKernelGGL((k_draw<LD, NT>), dim3(a.T), block, 0, st, a, ws);
    return moe_check_launch("moe_sample/draw");
}

template <int LD>
int run(SmpArgs a, void* ws, hipStream_t st) {
    if (a.V <= ROW_MAX) {
        const auto go = [&](auto nt) {
            constexpr int NT = decltype(nt)::value;
            hipLaunchKernelGGL((k_row<LD, NT>), dim3(a.T), dim3(NT), 0, st, a);
        };
        if (a.V <= 256 * PER) go(std::integral_constant<int, 256>{});
        else if (a.V <= 512 * PER) go(std::integral_constant<int, 512>{});
        else go(std::integral_constant<int, 1024>{});
        return moe_check_launch("moe_sample");
    }
    a.chunks = chunks_of(a.T, a.V);
    return chunk_threads(a.T, a.V) == 256 ? run_long<LD, 256>(a, ws, st) : run_long<LD, 1024>(a, ws, st);
}

}  // namespace

extern "C" {

size_t moe_sample_workspace_bytes(int T, int V) {
    if (T < 0 || T > MOE_SAMPLE_MAX_T || V < 1 || V > MOE_SAMPLE_MAX_V) return 0;
    if (T == 0 || V <= ROW_MAX) return 16;
    return (size_t)T * RowWs::bytes(chunks_of(T, V));
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
    SmpArgs a{logits, ldl, T, V, 51, 0, temperature, min_p, top_k, top_p, u, ids, prob, 0};
    while (((int64_t)1 << (62 - a.S)) < V) --a.S;
    a.vec = reinterpret_cast<uintptr_t>(logits) % (4 * el) == 0 && (T == 1 || ldl % 4 == 0);
    return l_dtype == MOE_X_F32 ? run<MOE_X_F32>(a, ws, stream) : run<MOE_X_BF16>(a, ws, stream);
}

}  // extern "C"
