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
// One workgroup takes one row.  Thresholds come from a radix selection over
// order-preserving keys of the logits, eight bits a pass, by count (top-k) and
// by mass (top-p).
#include <math.h>

#include "common.hpp"

namespace {

using u64 = unsigned long long;

constexpr int SMP_THREADS = 1024;
constexpr int SMP_WAVES = SMP_THREADS / 64;

// Rising with the value; -inf and NaN give 0 (not a candidate).  -0 counts as +0.
__device__ __forceinline__ uint32_t key_of(float l) {
    if (!(l > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(l + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

template <int LD>
__device__ __forceinline__ float load_l(const void* p, int64_t i) {
    if constexpr (LD == MOE_X_F32) return reinterpret_cast<const float*>(p)[i];
    else return moe::bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}

// A row's settings and the mass of a logit under them.
struct Row {
    double top, rtemp, min_p, one;
    uint32_t kmax;
    // mass of a candidate; 0 also for one that min-p drops
    __device__ __forceinline__ u64 mass(uint32_t key) const {
        if (key == kmax) return (u64)one;
        const double w = exp(((double)value_of(key) - top) * rtemp);
        return w >= min_p ? (u64)rint(w * one) : 0;
    }
    __device__ __forceinline__ bool candidate(uint32_t key) const {
        if (key == 0 || key == kmax) return key != 0;
        return min_p <= 0.0 || exp(((double)value_of(key) - top) * rtemp) >= min_p;
    }
};

template <typename T, typename Op>
__device__ __forceinline__ T block_reduce(T v, T* scratch, Op op) {
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) v = op(v, __shfl_xor(v, s, moe::WAVE));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
    __syncthreads();
    v = scratch[0];
    for (int w = 1; w < SMP_WAVES; ++w) v = op(v, scratch[w]);
    return v;
}

// Inclusive sum over the block's threads, in thread order; *total the sum of all.
__device__ __forceinline__ u64 block_scan(u64 v, u64* scratch, u64* total) {
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const u64 o = __shfl_up(v, s, moe::WAVE);
        if (lane >= s) v += o;
    }
    __syncthreads();
    if (lane == 63) scratch[wid] = v;
    __syncthreads();
    u64 all = 0;
    for (int w = 0; w < SMP_WAVES; ++w) {
        if (w == wid) v += all;
        all += scratch[w];
    }
    *total = all;
    return v;
}

template <int LD>
__global__ void __launch_bounds__(SMP_THREADS) k_sample(const void* __restrict__ logits, int64_t ldl, int V, int S,
                                                        const float* __restrict__ temperature,
                                                        const float* __restrict__ min_p,
                                                        const int32_t* __restrict__ top_k,
                                                        const float* __restrict__ top_p, const float* __restrict__ u,
                                                        int32_t* __restrict__ ids, float* __restrict__ prob) {
    __shared__ u64 scratch[SMP_WAVES];
    __shared__ u64 hist[256];
    __shared__ uint32_t s_key;
    __shared__ u64 s_left;
    __shared__ int s_at;
    const int row = blockIdx.x, tid = threadIdx.x;
    const int64_t base = (int64_t)row * ldl;
    const auto key = [&](int i) { return key_of(load_l<LD>(logits, base + i)); };
    const auto umax = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    const auto imin = [](int a, int b) { return a < b ? a : b; };
    const auto add = [](u64 a, u64 b) { return a + b; };

    uint32_t kmax = 0;
    for (int i = tid; i < V; i += SMP_THREADS) kmax = umax(kmax, key(i));
    kmax = block_reduce(kmax, reinterpret_cast<uint32_t*>(scratch), umax);
    if (kmax == 0) {
        if (tid == 0) {
            ids[row] = -1;
            if (prob) prob[row] = 0.0f;
        }
        return;
    }
    const float temp = temperature ? temperature[row] : 1.0f;
    if (!(temp > 0.0f)) {  // greedy
        int at = V;
        for (int i = tid; i < V; i += SMP_THREADS)
            if (key(i) == kmax) at = imin(at, i);
        at = block_reduce(at, reinterpret_cast<int*>(scratch), imin);
        if (tid == 0) {
            ids[row] = at;
            if (prob) prob[row] = 1.0f;
        }
        return;
    }
    Row r;
    r.kmax = kmax;
    r.top = value_of(kmax);
    r.rtemp = 1.0 / (double)temp;
    r.min_p = min_p ? (double)min_p[row] : 0.0;
    if (!(r.min_p > 0.0)) r.min_p = 0.0;
    r.one = ldexp(1.0, S);

    // kept: key > tkey, or key == tkey and id <= tid_
    uint32_t tkey = 0;
    int tidx = V;
    const auto kept = [&](uint32_t kk, int i) { return kk > tkey || (kk == tkey && i <= tidx); };

    // the prefix whose weight (count or mass) first reaches `want` (>= 1 and at most all of it)
    const auto select = [&](auto weight, u64 want) {
        uint32_t prefix = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += SMP_THREADS) hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < V; i += SMP_THREADS) {
                const uint32_t kk = key(i);
                if (kk == 0 || !kept(kk, i)) continue;
                if (shift < 24 && (kk >> (shift + 8)) != (prefix >> (shift + 8))) continue;
                const u64 w = weight(kk);
                if (w) atomicAdd(&hist[(kk >> shift) & 255], w);
            }
            __syncthreads();
            if (tid == 0) {
                int d = 255;
                while (d > 0 && hist[d] < want) want -= hist[d--];
                s_key = prefix | ((uint32_t)d << shift);
                s_left = want;
            }
            __syncthreads();
            prefix = s_key;
            want = s_left;
            __syncthreads();
        }
        // how many of the equal ones: all weigh the same
        const u64 each = weight(prefix);
        u64 need = each ? (want + each - 1) / each : 0;
        int last = V;
        for (int i0 = 0; i0 < V; i0 += SMP_THREADS) {
            const int i = i0 + tid;
            const uint32_t kk = i < V ? key(i) : 0;
            const bool is = kk == prefix && kept(kk, i);
            u64 total;
            const u64 at = block_scan(is ? 1 : 0, scratch, &total);
            if (tid == 0) s_at = V;
            __syncthreads();
            if (is && at == need) s_at = i;
            __syncthreads();
            if (s_at < V) {
                last = s_at;
                break;
            }
            need -= total;
        }
        tkey = prefix;
        tidx = last;
        __syncthreads();
    };

    const auto count = [&](uint32_t kk) { return (u64)(r.candidate(kk) ? 1 : 0); };
    const auto mass = [&](uint32_t kk) { return r.mass(kk); };
    const auto total_of = [&](auto weight) {
        u64 v = 0;
        for (int i = tid; i < V; i += SMP_THREADS) {
            const uint32_t kk = key(i);
            if (kk && kept(kk, i)) v += weight(kk);
        }
        return block_reduce(v, scratch, add);
    };

    const int k = top_k ? top_k[row] : 0;
    if (k > 0 && k < V && total_of(count) > (u64)k) select(count, (u64)k);
    u64 Z = total_of(mass);
    const float p = top_p ? top_p[row] : 1.0f;
    if (p < 1.0f) {
        const double want = ceil((double)(p > 0.0f ? p : 0.0f) * (double)Z);
        select(mass, want < 1.0 ? 1 : (u64)want < Z ? (u64)want : Z);
        Z = total_of(mass);
    }
    double uu = u[row];
    if (!(uu > 0.0)) uu = 0.0;
    if (uu > 1.0) uu = 1.0;
    u64 target = (u64)(uu * (double)Z);
    if (target >= Z) target = Z - 1;
    for (int i0 = 0; i0 < V; i0 += SMP_THREADS) {
        const int i = i0 + tid;
        const uint32_t kk = i < V ? key(i) : 0;
        const u64 w = kk && kept(kk, i) ? r.mass(kk) : 0;
        u64 total;
        const u64 cum = block_scan(w, scratch, &total);
        if (w && cum > target && cum - w <= target) {
            ids[row] = i;
            if (prob) prob[row] = (float)((double)w / (double)Z);
        }
        if (total > target) break;
        target -= total;
    }
}

}  // namespace

extern "C" {

size_t moe_sample_workspace_bytes(int T, int V) {
    if (T < 0 || T > MOE_SAMPLE_MAX_T || V < 1 || V > MOE_SAMPLE_MAX_V) return 0;
    return 16;
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
    const uintptr_t lm = l_dtype == MOE_X_F32 ? 3 : 1;
    MOE_REQUIRE(!(reinterpret_cast<uintptr_t>(logits) & lm) && moe_aligned16(ws), MOE_E_ALIGN,
                "moe_sample: logits must be aligned to their elements, ws to 16 bytes");
    MOE_REQUIRE(ws_bytes >= moe_sample_workspace_bytes(T, V), MOE_E_ARG, "moe_sample: workspace of %zu bytes, %zu needed",
                ws_bytes, moe_sample_workspace_bytes(T, V));
    if (T == 0) return moe_ok();
    int S = 62;
    while ((1 << (62 - S)) < V) --S;
    auto kern = l_dtype == MOE_X_F32 ? k_sample<MOE_X_F32> : k_sample<MOE_X_BF16>;
    hipLaunchKernelGGL(kern, dim3(T), dim3(SMP_THREADS), 0, stream, logits, ldl, V, S, temperature, min_p, top_k, top_p,
                       u, ids, prob);
    return moe_check_launch("moe_sample");
}

}  // extern "C"
