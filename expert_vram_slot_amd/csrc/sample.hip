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
// 2^-S with S = 62 - ceil(log2 V), so a row's mass stays below 2^63.  Sums of
// whole numbers do not depend on their order: the result is one of the inputs
// alone, with integer atomics wherever they are handy.
//
// What is kept is always a prefix, so one pair (key, id) says it, and no row
// is ever sorted.  A row is cut into BINS of equal width in the logit (over
// the span where masses are not 0); counts and masses per bin tell in which
// bin a cut falls, and only the ids of those bins (a few hundred, whatever the
// row) are listed, sorted and summed to find where.
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

#include "common.hpp"
#include "exp64.hpp"

namespace {

using u64 = unsigned long long;
using v4u = uint32_t __attribute__((ext_vector_type(4)));
using v2u = uint32_t __attribute__((ext_vector_type(2)));

constexpr int BINS = 1024;
constexpr int LIST = 2048;
constexpr int CHUNK = 4096;          // ids of a workgroup of k_top .. k_list
constexpr int CHUNK_THREADS = 256;
constexpr int ROW_THREADS = 1024;
constexpr int ROW_MAX = 16384;       // ids a workgroup's registers hold
constexpr int MAX_CHUNKS = MOE_SAMPLE_MAX_V / CHUNK;

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

// Per row of the workspace (longer rows).
struct RowWs {
    u64* bin_mass;       // [BINS]
    u64* list;           // [LIST] key << 32 | ~id
    u64* chunk_mass;     // [chunks] mass of the chunk's ids above the cut bins
    uint32_t* bin_count;  // [BINS]
    uint32_t* chunk_max;  // [chunks] keys
    uint32_t* chunk_min;  // [chunks]
    uint32_t* listed;    // [1]

    static __host__ __device__ size_t bytes(int chunks) {
        return (size_t)BINS * 12 + (size_t)LIST * 8 + (size_t)((chunks + 1) & ~1) * 16 + 16;
    }
    __host__ __device__ RowWs(void* ws, int64_t row, int chunks) {
        const int c = (chunks + 1) & ~1;
        char* p = reinterpret_cast<char*>(ws) + row * bytes(chunks);
        bin_mass = reinterpret_cast<u64*>(p);
        list = bin_mass + BINS;
        chunk_mass = list + LIST;
        bin_count = reinterpret_cast<uint32_t*>(chunk_mass + c);
        chunk_max = bin_count + BINS;
        chunk_min = chunk_max + c;
        listed = chunk_min + c;
    }
};

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
        if (!(min_p > 0.0)) min_p = 0.0;
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
        if (key == kmax) return (u64)one;
        const double w = moe::exp64(((double)value_of(key) - top) * rtemp);
        return w >= min_p ? (u64)rint(w * one) : 0;
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

template <int NT, typename T, typename Op>
__device__ __forceinline__ T block_reduce(T v, u64* scratch_, Op op) {
    T* scratch = reinterpret_cast<T*>(scratch_);
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) v = op(v, __shfl_xor(v, s, moe::WAVE));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) v = op(v, scratch[w]);
    return v;
}

__device__ __forceinline__ u64 wave_scan(u64 v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const u64 o = __shfl_up(v, s, moe::WAVE);
        if (lane >= s) v += o;
    }
    return v;
}

// Inclusive sum over the block's threads, in thread order; *total the sum of all.
template <int NT>
__device__ __forceinline__ u64 block_scan(u64 v, u64* scratch, u64* total) {
    const int wid = threadIdx.x >> 6;
    v = wave_scan(v);
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
struct Add { __device__ u64 operator()(u64 a, u64 b) const { return a + b; } };

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

// Where the cuts fall.  Ids of bins below `sure` are kept whatever happens
// inside the cut bins: bins p0 .. p1 (top-p; the last one is open as long as
// the mass that top-k leaves is) and bin `bk` (top-k).
struct Cuts {
    int sure, p0, p1, bk;
    u64 rank, mass_bk;  // ids of bin bk that top-k keeps; mass above bin bk
    __device__ __forceinline__ bool lists(int b) const { return (b >= p0 && b <= p1) || b == bk; }
    __device__ __forceinline__ bool any() const { return sure < BINS; }
};

// From the row's counts and masses per bin (counts only where top-k cuts,
// masses only where top-p does).  s_cuts and scratch in LDS.
template <int NT>
__device__ __forceinline__ void find_cuts(const Row& r, const uint32_t* count, const u64* mass, Cuts* s_cuts,
                                          u64* s_z, u64* scratch) {
    constexpr int PER = BINS / NT;
    const int b0 = threadIdx.x * PER;
    if (threadIdx.x == 0) {
        s_cuts->sure = BINS, s_cuts->p0 = BINS, s_cuts->p1 = -1, s_cuts->bk = -1;
        s_cuts->rank = 0, s_cuts->mass_bk = 0;
    }
    u64 m[PER], before = 0, total = 0;
    if (r.cut_p) {
        u64 sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += m[i] = mass[b0 + i];
        before = block_scan<NT>(sum, scratch, &total) - sum;
    }
    if (threadIdx.x == 0) s_z[0] = s_z[1] = total;  // the mass that top-k leaves lies between the two
    __syncthreads();
    if (r.cut_k) {
        u64 c[PER], sum = 0, all;
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += c[i] = count[b0 + i];
        u64 at = block_scan<NT>(sum, scratch, &all) - sum, mb = before;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
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
        for (int i = 0; i < PER; ++i) {
            if (mb < lo && mb + m[i] >= lo) s_cuts->p0 = s_cuts->sure = b0 + i;
            if (mb < hi && mb + m[i] >= hi) s_cuts->p1 = b0 + i;
            mb += m[i];
        }
        __syncthreads();
    }
}

// Sorts list[0 .. n) falling (n at most LIST) and finds the last kept entry.
// Returns its position; cum[i] is the mass of entries 0 .. i.
template <int NT>
__device__ __forceinline__ int resolve(const Row& r, const Cuts& c, u64 sure_mass, int n, u64* list, u64* cum,
                                       u64* scratch, int* s_at) {
    int size = 2;
    while (size < n) size <<= 1;
    for (int i = n + threadIdx.x; i < size; i += NT) list[i] = 0;
    __syncthreads();
    for (int w = 2; w <= size; w <<= 1)
        for (int s = w >> 1; s >= 1; s >>= 1) {
            for (int h = threadIdx.x; h < size >> 1; h += NT) {
                const int i = 2 * h - (h & (s - 1)), j = i + s;
                const u64 x = list[i], y = list[j];
                if ((x < y) == ((i & w) == 0)) list[i] = y, list[j] = x;
            }
            __syncthreads();
        }
    u64 base = 0;
    for (int i0 = 0; i0 < n; i0 += NT) {
        const int i = i0 + threadIdx.x;
        u64 total;
        const u64 v = block_scan<NT>(i < n ? r.mass((uint32_t)(list[i] >> 32)) : 0, scratch, &total);
        if (i < n) cum[i] = base + v;
        base += total;
    }
    if (threadIdx.x == 0) *s_at = n - 1;
    __syncthreads();
    u64 z = 0;  // the mass that top-k leaves
    int last = n - 1;
    if (c.bk >= 0) {
        // entries of bins above bk come first
        for (int i = threadIdx.x; i < n; i += NT) {
            const bool in = r.bin((uint32_t)(list[i] >> 32)) >= c.bk;
            if (in && (i == 0 || r.bin((uint32_t)(list[i - 1] >> 32)) < c.bk)) *s_at = i + (int)c.rank - 1;
        }
        __syncthreads();
        last = *s_at < n ? *s_at : n - 1;
        const int first = last - (int)c.rank + 1;
        z = c.mass_bk + cum[last] - (first > 0 ? cum[first - 1] : 0);
    }
    if (r.cut_p) {
        if (c.bk < 0) z = c.mass_bk;
        const u64 want = r.want(z);
        __syncthreads();
        for (int i = threadIdx.x; i <= last; i += NT) {
            const u64 prev = sure_mass + (i > 0 ? cum[i - 1] : 0);
            if (sure_mass + cum[i] >= want && prev < want) *s_at = i;
        }
        __syncthreads();
        last = *s_at;
    }
    return last;
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
// a segment is a wave's part of a group: 256 ids in a row.  Writes the result
// of the id where the running mass passes `target`; z < 0: z is the mass of
// these ids and target is drawn from it.  seg: J * NT / 64 u64.
template <int NT, int J, bool WHOLE>
__device__ __forceinline__ void draw(const SmpArgs& a, const Row& r, int row, int i0, const v4u (&key)[J], u64 bound,
                                     u64 z, u64 target, u64* seg) {
    constexpr int NW = NT / 64;
    const int wid = threadIdx.x >> 6;
    u64 m[J][4], sum[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        sum[j] = 0;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const uint32_t kk = key[j][v];
            const u64 at = ((u64)kk << 32) | (uint32_t)~(i0 + (j * NT + (int)threadIdx.x) * 4 + v);
            m[j][v] = kk && at >= bound ? r.mass(kk) : 0;
            sum[j] += m[j][v];
        }
        const u64 all = moe::wave_sum(sum[j]);
        if ((threadIdx.x & 63) == 0) seg[j * NW + wid] = all;
    }
    __syncthreads();
    if constexpr (WHOLE) {
        z = 0;
        for (int s = 0; s < J * NW; ++s) z += seg[s];
        target = draw_at(a, row, z);
    }
    u64 before = 0;
    int s = 0;
    while (s < J * NW - 1 && before + seg[s] <= target) before += seg[s++];
    if (s % NW != wid) return;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if (j != s / NW) continue;
        u64 at = before + wave_scan(sum[j]) - sum[j];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            if (m[j][v] && at <= target && at + m[j][v] > target)
                finish(a, row, i0 + (j * NT + (int)threadIdx.x) * 4 + v, m[j][v], z);
            at += m[j][v];
        }
    }
}

// -------------------------------------------------- rows in one workgroup

template <int LD>
__global__ void __launch_bounds__(ROW_THREADS) k_row(SmpArgs a) {
    constexpr int NT = ROW_THREADS, J = ROW_MAX / (4 * NT);
    __shared__ u64 bin_mass[BINS];
    __shared__ uint32_t bin_count[BINS];
    __shared__ u64 list[LIST], cum[LIST];
    __shared__ u64 scratch[NT / 64], s_z[2], seg[J * NT / 64];
    __shared__ Cuts cuts;
    __shared__ uint32_t s_key, s_n;
    __shared__ int s_at;
    const int row = blockIdx.x, tid = threadIdx.x;
    v4u key[J];
    uint32_t kmax = 0, kmin = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        key[j] = load_keys<LD>(a, row, (j * NT + tid) * 4);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            kmax = key[j][v] > kmax ? key[j][v] : kmax;
            kmin = key[j][v] && key[j][v] < kmin ? key[j][v] : kmin;
        }
    }
    for (int i = tid; i < BINS; i += NT) bin_mass[i] = 0, bin_count[i] = 0;
    if (tid == 0) s_n = 0, s_at = a.V;
    kmax = block_reduce<NT>(kmax, scratch, UMax());
    if (kmax == 0) {
        if (tid == 0) finish(a, row, -1, 0, 0);
        return;
    }
    kmin = block_reduce<NT>(kmin, scratch, UMin());
    const Row r(a, row, kmax, kmin);
    if (r.greedy) {
        int at = a.V;
#pragma unroll
        for (int j = J - 1; j >= 0; --j)
#pragma unroll
            for (int v = 3; v >= 0; --v)
                if (key[j][v] == kmax) at = (j * NT + tid) * 4 + v;
        if (at < a.V) atomicMin(&s_at, at);
        __syncthreads();
        if (tid == 0) finish(a, row, s_at, 1, 1);
        return;
    }
    u64 bound = 0;
    if (r.cut_k || r.cut_p) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const uint32_t kk = key[j][v];
                const u64 w = kk ? r.mass(kk) : 0;
                if (w) {
                    const int b = r.bin(kk);
                    if (r.cut_k) atomicAdd(&bin_count[b], 1u);
                    if (r.cut_p) atomicAdd(&bin_mass[b], w);
                }
            }
        __syncthreads();
        find_cuts<NT>(r, bin_count, bin_mass, &cuts, s_z, scratch);
        const Cuts c = cuts;
        if (c.any()) {
            u64 sure = 0;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const uint32_t kk = key[j][v];
                    const int b = kk ? r.bin(kk) : BINS;
                    if (b < c.sure && r.cut_p) sure += r.mass(kk);
                    if (kk && c.lists(b) && r.mass(kk)) {
                        const uint32_t at = atomicAdd(&s_n, 1u);
                        if (at < LIST) list[at] = ((u64)kk << 32) | (uint32_t)~((j * NT + tid) * 4 + v);
                    }
                }
            sure = block_reduce<NT>(sure, scratch, Add());
            Cuts cc = c;
            if (c.bk < 0) cc.mass_bk = s_z[1];
            if (s_n > LIST) {
                select_row<LD, NT>(a, r, row, list, scratch, s_z, &s_key, &s_at);
                return;
            }
            const int last = resolve<NT>(r, cc, sure, s_n, list, cum, scratch, &s_at);
            bound = list[last];
        }
    }
    draw<NT, J, true>(a, r, row, 0, key, bound, 0, 0, seg);
}

// -------------------------------------------------------------- longer rows

template <int LD>
__device__ __forceinline__ void load_chunk(const SmpArgs& a, int row, int chunk, v4u (&key)[CHUNK / 4 / CHUNK_THREADS]) {
#pragma unroll
    for (int j = 0; j < CHUNK / 4 / CHUNK_THREADS; ++j)
        key[j] = load_keys<LD>(a, row, chunk * CHUNK + (j * CHUNK_THREADS + (int)threadIdx.x) * 4);
}

template <int LD>
__global__ void __launch_bounds__(CHUNK_THREADS) k_top(SmpArgs a, void* ws) {
    constexpr int NT = CHUNK_THREADS, J = CHUNK / 4 / NT;
    __shared__ u64 scratch[NT / 64];
    const int row = blockIdx.y, chunk = blockIdx.x;
    const RowWs w(ws, row, a.chunks);
    v4u key[J];
    load_chunk<LD>(a, row, chunk, key);
    for (int i = chunk * NT + threadIdx.x; i < BINS; i += a.chunks * NT) w.bin_mass[i] = 0, w.bin_count[i] = 0;
    if (chunk == 0 && threadIdx.x == 0) *w.listed = 0;
    uint32_t kmax = 0, kmin = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            kmax = key[j][v] > kmax ? key[j][v] : kmax;
            kmin = key[j][v] && key[j][v] < kmin ? key[j][v] : kmin;
        }
    kmax = block_reduce<NT>(kmax, scratch, UMax());
    kmin = block_reduce<NT>(kmin, scratch, UMin());
    if (threadIdx.x == 0) w.chunk_max[chunk] = kmax, w.chunk_min[chunk] = kmin;
}

// The row's largest and smallest candidate (kmax 0: none).
__device__ __forceinline__ void row_ends(const SmpArgs& a, const RowWs& w, u64* scratch, uint32_t& kmax,
                                         uint32_t& kmin) {
    static_assert(MAX_CHUNKS <= CHUNK_THREADS, "one chunk a thread");
    const bool in = (int)threadIdx.x < a.chunks;
    kmax = block_reduce<CHUNK_THREADS>(in ? w.chunk_max[threadIdx.x] : 0u, scratch, UMax());
    kmin = block_reduce<CHUNK_THREADS>(in ? w.chunk_min[threadIdx.x] : 0xFFFFFFFFu, scratch, UMin());
}

template <int LD>
__global__ void __launch_bounds__(CHUNK_THREADS) k_bins(SmpArgs a, void* ws) {
    constexpr int NT = CHUNK_THREADS, J = CHUNK / 4 / NT;
    __shared__ u64 bin_mass[BINS];
    __shared__ uint32_t bin_count[BINS];
    __shared__ u64 scratch[NT / 64];
    const int row = blockIdx.y, chunk = blockIdx.x;
    const RowWs w(ws, row, a.chunks);
    v4u key[J];
    load_chunk<LD>(a, row, chunk, key);
    uint32_t kmax, kmin;
    row_ends(a, w, scratch, kmax, kmin);
    if (kmax == 0) return;
    const Row r(a, row, kmax, kmin);
    if (r.greedy) return;
    if (!r.cut_k && !r.cut_p) {
        u64 sum = 0;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) sum += key[j][v] ? r.mass(key[j][v]) : 0;
        sum = block_reduce<NT>(sum, scratch, Add());
        if (threadIdx.x == 0) w.chunk_mass[chunk] = sum;
        return;
    }
    for (int i = threadIdx.x; i < BINS; i += NT) bin_mass[i] = 0, bin_count[i] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const uint32_t kk = key[j][v];
            const u64 m = kk ? r.mass(kk) : 0;
            if (m) {
                const int b = r.bin(kk);
                if (r.cut_k) atomicAdd(&bin_count[b], 1u);
                if (r.cut_p) atomicAdd(&bin_mass[b], m);
            }
        }
    __syncthreads();
    for (int i = threadIdx.x; i < BINS; i += NT) {
        if (r.cut_k && bin_count[i]) atomicAdd(&w.bin_count[i], bin_count[i]);
        if (r.cut_p && bin_mass[i]) atomicAdd(&w.bin_mass[i], bin_mass[i]);
    }
}

template <int LD>
__global__ void __launch_bounds__(CHUNK_THREADS) k_list(SmpArgs a, void* ws) {
    constexpr int NT = CHUNK_THREADS, J = CHUNK / 4 / NT;
    __shared__ u64 scratch[NT / 64], s_z[2];
    __shared__ Cuts cuts;
    const int row = blockIdx.y, chunk = blockIdx.x;
    const RowWs w(ws, row, a.chunks);
    v4u key[J];
    load_chunk<LD>(a, row, chunk, key);
    uint32_t kmax, kmin;
    row_ends(a, w, scratch, kmax, kmin);
    if (kmax == 0) return;
    const Row r(a, row, kmax, kmin);
    if (r.greedy || (!r.cut_k && !r.cut_p)) return;
    find_cuts<NT>(r, w.bin_count, w.bin_mass, &cuts, s_z, scratch);
    const Cuts c = cuts;
    u64 sure = 0;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const uint32_t kk = key[j][v];
            const int b = kk ? r.bin(kk) : BINS;
            if (b < c.sure) sure += r.mass(kk);
            if (kk && c.lists(b) && r.mass(kk)) {
                const uint32_t at = atomicAdd(w.listed, 1u);
                if (at < LIST) w.list[at] = ((u64)kk << 32) | (uint32_t)~(chunk * CHUNK + (j * NT + (int)threadIdx.x) * 4 + v);
            }
        }
    sure = block_reduce<NT>(sure, scratch, Add());
    if (threadIdx.x == 0) w.chunk_mass[chunk] = sure;
}

template <int LD>
__global__ void __launch_bounds__(CHUNK_THREADS) k_draw(SmpArgs a, void* ws) {
    constexpr int NT = CHUNK_THREADS, J = CHUNK / 4 / NT;
    __shared__ u64 list[LIST], cum[LIST];
    __shared__ u64 chunk_mass[MAX_CHUNKS];
    __shared__ u64 scratch[NT / 64], s_z[2], seg[J * NT / 64];
    __shared__ Cuts cuts;
    __shared__ uint32_t s_key;
    __shared__ int s_at;
    const int row = blockIdx.x, tid = threadIdx.x;
    const RowWs w(ws, row, a.chunks);
    uint32_t kmax, kmin;
    row_ends(a, w, scratch, kmax, kmin);
    if (kmax == 0) {
        if (tid == 0) finish(a, row, -1, 0, 0);
        return;
    }
    const Row r(a, row, kmax, kmin);
    if (r.greedy) {
        // the first chunk that holds the largest, and the first id there
        const uint32_t at = block_reduce<NT>(tid < a.chunks && w.chunk_max[tid] == kmax ? (uint32_t)tid : ~0u, scratch, UMin());
        v4u key[J];
        load_chunk<LD>(a, row, (int)at, key);
        uint32_t id = ~0u;
#pragma unroll
        for (int j = J - 1; j >= 0; --j)
#pragma unroll
            for (int v = 3; v >= 0; --v)
                if (key[j][v] == kmax) id = at * CHUNK + (j * NT + tid) * 4 + v;
        id = block_reduce<NT>(id, scratch, UMin());
        if (tid == 0) finish(a, row, (int)id, 1, 1);
        return;
    }
    u64 mass = tid < a.chunks ? w.chunk_mass[tid] : 0;
    chunk_mass[tid] = mass;
    u64 bound = 0;
    if (r.cut_k || r.cut_p) {
        find_cuts<NT>(r, w.bin_count, w.bin_mass, &cuts, s_z, scratch);
        Cuts c = cuts;
        if (c.any()) {
            const uint32_t n = *w.listed;
            if (n > LIST) {
                select_row<LD, NT>(a, r, row, list, scratch, s_z, &s_key, &s_at);
                return;
            }
            for (int i = tid; i < (int)n; i += NT) list[i] = w.list[i];
            const u64 sure = block_reduce<NT>(mass, scratch, Add());
            if (c.bk < 0) c.mass_bk = s_z[1];
            const int last = resolve<NT>(r, c, sure, (int)n, list, cum, scratch, &s_at);
            bound = list[last];
            for (int i = tid; i <= last; i += NT)
                atomicAdd(&chunk_mass[(uint32_t)~(uint32_t)list[i] / CHUNK], cum[i] - (i > 0 ? cum[i - 1] : 0));
            __syncthreads();
            mass = chunk_mass[tid];
        }
    }
    u64 z;
    const u64 upto = block_scan<NT>(mass, scratch, &z);
    const u64 target = draw_at(a, row, z);
    if (mass && upto > target && upto - mass <= target) s_at = tid, s_z[0] = target - (upto - mass);
    __syncthreads();
    v4u key[J];
    load_chunk<LD>(a, row, s_at, key);
    draw<NT, J, false>(a, r, row, s_at * CHUNK, key, bound, z, s_z[0], seg);
}

}  // namespace

extern "C" {

size_t moe_sample_workspace_bytes(int T, int V) {
    if (T < 0 || T > MOE_SAMPLE_MAX_T || V < 1 || V > MOE_SAMPLE_MAX_V) return 0;
    if (T == 0 || V <= ROW_MAX) return 16;
    return (size_t)T * RowWs::bytes((V + CHUNK - 1) / CHUNK);
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
    SmpArgs a{logits, ldl, T, V, 62, (V + CHUNK - 1) / CHUNK, temperature, min_p, top_k, top_p, u, ids, prob, 0};
    while ((1 << (62 - a.S)) < V) --a.S;
    a.vec = reinterpret_cast<uintptr_t>(logits) % (4 * el) == 0 && (T == 1 || ldl % 4 == 0);
    const bool f32 = l_dtype == MOE_X_F32;
    if (V <= ROW_MAX) {
        hipLaunchKernelGGL(f32 ? k_row<MOE_X_F32> : k_row<MOE_X_BF16>, dim3(T), dim3(ROW_THREADS), 0, stream, a);
        return moe_check_launch("moe_sample");
    }
    const dim3 grid(a.chunks, T), block(CHUNK_THREADS);
    hipLaunchKernelGGL(f32 ? k_top<MOE_X_F32> : k_top<MOE_X_BF16>, grid, block, 0, stream, a, ws);
    if (int rc = moe_check_launch("moe_sample/top")) return rc;
    hipLaunchKernelGGL(f32 ? k_bins<MOE_X_F32> : k_bins<MOE_X_BF16>, grid, block, 0, stream, a, ws);
    if (int rc = moe_check_launch("moe_sample/bins")) return rc;
    if (top_k || top_p) {
        hipLaunchKernelGGL(f32 ? k_list<MOE_X_F32> : k_list<MOE_X_BF16>, grid, block, 0, stream, a, ws);
        if (int rc = moe_check_launch("moe_sample/list")) return rc;
    }
    hipLaunchKernelGGL(f32 ? k_draw<MOE_X_F32> : k_draw<MOE_X_BF16>, dim3(T), block, 0, stream, a, ws);
    return moe_check_launch("moe_sample/draw");
}

}  // extern "C"
