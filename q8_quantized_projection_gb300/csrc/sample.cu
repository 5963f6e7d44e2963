// sample.cu -- sampling of one token a row from the head's logits.
//
// One CTA a row.  A token's weight is an integer: exp((x - M)/T) in units of
// 2^-shift, so sums are exact and independent of their order.  The filters cut
// the tokens in order of x (ties: lowest index first), so what they keep is
// "key above t, and of those equal to t the ones up to index `last`".  t is
// found by a binary search over the bits of an ordered key.
#include <math.h>

#include "common.cuh"
#include "launch.h"

namespace q8 {

namespace {

constexpr int kThreads = 1024, kWarpsN = kThreads / 32;
typedef unsigned long long u64;

// Order of the logits as unsigned integers: 0 for NaN and -inf (never drawn).
__device__ __forceinline__ uint32_t logit_key(float x) {
    if (!(x > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ u64 block_sum(u64 v, u64* s) {
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    u64 t = 0;
    for (int w = 0; w < kWarpsN; ++w) t += s[w];
    __syncthreads();
    return t;
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* s) {
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t t = 0;
    for (int w = 0; w < kWarpsN; ++w) t = max(t, s[w]);
    __syncthreads();
    return t;
}

// Index of the e-th (from 1) element of the row for which pred holds, by an
// ordered pass; the row has at least e of them.
template <typename P>
__device__ __forceinline__ int64_t nth_index(int64_t N, u64 e, P weight, u64* s, int64_t* s_at) {
    u64 before = 0;
    for (int64_t i0 = 0; i0 < N; i0 += kThreads) {
        const int64_t i = i0 + threadIdx.x;
        const u64 w = i < N ? weight(i) : 0;
        u64 x = w;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        for (int d = 1; d < 32; d <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) s[warp] = x;
        __syncthreads();
        u64 b = before, total = 0;
        for (int k = 0; k < kWarpsN; ++k) {
            if (k < warp) b += s[k];
            total += s[k];
        }
        // the one element whose inclusive sum first reaches e
        if (w && b + x >= e && b + x - w < e) *s_at = i;
        __syncthreads();
        before += total;
        if (before >= e) break;
    }
    const int64_t at = *s_at;
    __syncthreads();
    return at;
}

__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a, int shift, int* err) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ u64 s_sum[kWarpsN];
    __shared__ uint32_t s_max[kWarpsN];
    __shared__ int64_t s_at;
    const int64_t m = blockIdx.x, N = a.N;
    const float* x = a.x + m * a.ldx;
    const float T = a.temperature ? a.temperature[m] : 1.0f;
    const int32_t k = a.top_k ? a.top_k[m] : 0;
    const float p = a.top_p ? a.top_p[m] : 1.0f, mp = a.min_p ? a.min_p[m] : 0.0f;
    const auto give = [&](int64_t tok, float prob, int32_t kept) {
        if (threadIdx.x == 0) {
            a.tok[m] = int32_t(tok);
            if (a.prob) a.prob[m] = prob;
            if (a.kept) a.kept[m] = kept;
        }
    };
    if (!(T >= 0.0f) || isnan(p) || isnan(mp)) {
        if (threadIdx.x == 0) atomicExch(err, Q8_DEVERR_PARAM);
        return give(0, 0.0f, 0);
    }
    uint32_t top = 0;
    u64 n = 0;
    for (int64_t i = threadIdx.x; i < N; i += kThreads) {
        const uint32_t key = logit_key(x[i]);
        top = max(top, key);
        n += key != 0;
    }
    top = block_max(top, s_max);
    if (top == 0) return give(0, 0.0f, 0);
    n = block_sum(n, s_sum);
    if (threadIdx.x == 0) s_at = 0;
    __syncthreads();
    const bool greedy = T < 0x1p-60f;
    const int64_t first = nth_index(N, 1, [&](int64_t i) { return u64(logit_key(x[i]) == top); }, s_sum, &s_at);
    if (greedy) return give(first, 1.0f, 1);
    const float M = x[first];
    const u64 one = u64(1) << shift;
    const double c = 1.0 / double(T);
    const auto weight = [&](float v) -> u64 {
        if (v == M) return one;
        if (!(v > -INFINITY) || M == INFINITY) return 0;
        return u64(__double2ll_rn(exp((double(v) - double(M)) * c) * double(one)));
    };
    uint32_t t = 1;          // kept: key > t, or key == t and index <= last
    int64_t last = N;
    if (k > 0 && u64(k) < n) {
        t = 0;
        for (int b = 31; b >= 0; --b) {
            const uint32_t cand = t | (1u << b);
            u64 cnt = 0;
            for (int64_t i = threadIdx.x; i < N; i += kThreads) cnt += logit_key(x[i]) >= cand;
            if (block_sum(cnt, s_sum) >= u64(k)) t = cand;
        }
        u64 above = 0;
        for (int64_t i = threadIdx.x; i < N; i += kThreads) above += logit_key(x[i]) > t;
        above = block_sum(above, s_sum);
        last = nth_index(N, u64(k) - above, [&](int64_t i) { return u64(logit_key(x[i]) == t); }, s_sum, &s_at);
    }
    const auto in_cut = [&](uint32_t key, int64_t i) { return key > t || (key == t && i <= last); };
    if (p < 1.0f) {
        u64 S = 0;
        for (int64_t i = threadIdx.x; i < N; i += kThreads)
            if (in_cut(logit_key(x[i]), i)) S += weight(x[i]);
        S = block_sum(S, s_sum);
        const double P = double(p) * double(S);
        uint32_t t2 = 0;     // the largest key that reaches the mass
        for (int b = 31; b >= 0; --b) {
            const uint32_t cand = t2 | (1u << b);
            u64 mass = 0;
            for (int64_t i = threadIdx.x; i < N; i += kThreads) {
                const uint32_t key = logit_key(x[i]);
                if (key >= cand && in_cut(key, i)) mass += weight(x[i]);
            }
            if (cand <= top && double(block_sum(mass, s_sum)) >= P) t2 = cand;
        }
        u64 above = 0;
        for (int64_t i = threadIdx.x; i < N; i += kThreads)
            if (logit_key(x[i]) > t2) above += weight(x[i]);
        above = block_sum(above, s_sum);
        // ties at t2 weigh the same: the fewest that reach the mass, at least one
        u64 w2 = 0, lo = 1, hi = u64(N);
        for (int64_t i = threadIdx.x; i < N; i += kThreads)
            if (logit_key(x[i]) == t2) w2 = weight(x[i]);
        for (int d = 16; d; d >>= 1) w2 = max(w2, __shfl_xor_sync(0xffffffffu, w2, d));
        if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = w2;
        __syncthreads();
        for (int w = 0; w < kWarpsN; ++w) w2 = max(w2, s_sum[w]);
        __syncthreads();
        while (lo < hi) {
            const u64 e = (lo + hi) / 2;
            if (double(above + e * w2) >= P) hi = e; else lo = e + 1;
        }
        u64 ties = 0;
        for (int64_t i = threadIdx.x; i < N; i += kThreads) {
            const uint32_t key = logit_key(x[i]);
            ties += key == t2 && in_cut(key, i);
        }
        ties = block_sum(ties, s_sum);
        const int64_t end = nth_index(N, min(lo, ties), [&](int64_t i) { return u64(logit_key(x[i]) == t2); },
                                      s_sum, &s_at);
        t = t2;
        last = end;
    }
    if (mp > 1.0f) {
        t = top;
        last = first;
    }
    const double floor_w = double(mp) * double(one);
    u64 S = 0, cnt = 0;
    const auto kept_weight = [&](int64_t i) -> u64 {
        if (!in_cut(logit_key(x[i]), i)) return 0;
        const u64 w = weight(x[i]);
        return double(w) >= floor_w || i == first ? w : 0;
    };
    for (int64_t i = threadIdx.x; i < N; i += kThreads) {
        if (!in_cut(logit_key(x[i]), i)) continue;
        const u64 w = weight(x[i]);
        if (double(w) < floor_w && i != first) continue;
        S += w;
        ++cnt;
    }
    S = block_sum(S, s_sum);
    cnt = block_sum(cnt, s_sum);
    const float u = a.u[m];
    const double r = u > 0.0f ? floor(double(u) * double(S)) : 0.0;
    const u64 e = r >= double(S) ? S : min(u64(r) + 1, S);   // the first sum above u * S
    // every kept weight is above 0, also one below half a unit: u = 0 draws the first
    const auto kept_any = [&](int64_t i) -> u64 {
        return kept_weight(i) || (M < INFINITY && floor_w <= 0.0 && in_cut(logit_key(x[i]), i));
    };
    const int64_t at = u > 0.0f ? nth_index(N, e, kept_weight, s_sum, &s_at)
                                : nth_index(N, 1, kept_any, s_sum, &s_at);
    const double w = x[at] == M ? 1.0 : exp((double(x[at]) - double(M)) * c);
    give(at, float(w * double(one) / double(S)), int32_t(cnt));
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, const LaunchCtx& ctx) {
    int bits = 0;
    while ((int64_t(1) << bits) < a.N) ++bits;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attrs[1];
    cfg.gridDim = dim3(unsigned(a.rows));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = ctx.stream;
    cfg.numAttrs = pdl_attrs(ctx, attrs);
    cfg.attrs = attrs;
    return cudaLaunchKernelEx(&cfg, sample_kernel, a, 62 - bits, ctx.dev_err);
}

}  // namespace q8
