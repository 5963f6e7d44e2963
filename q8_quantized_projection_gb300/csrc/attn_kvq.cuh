// attn_kvq.cuh -- the attention kernels over quantised caches (kvq.cuh).
#pragma once

#include "attn.cuh"
#include "kvq.cuh"

namespace q8 {

// Value d of an entry from its codes and words.
template <int KIND>
__device__ __forceinline__ float kvq_value(const unsigned char* codes, const uint32_t* words, int d) {
    if constexpr (KIND == Q8_KVQ_I8) return __uint_as_float(words[d / 32]) * float(static_cast<signed char>(codes[d]));
    const float2 sm = kvq_scale_min(words[d / 32]);
    return fmaf(float(codes[d / 2] >> (d % 2 * 4) & 15), sm.x, sm.y);
}

// A warp's states entry by entry in binary32, lanes over the values.
template <class T>
__device__ __forceinline__ void kvq_plain_states(const Segment& s) {
    const AttnArgs& a = s.p.a;
    const int lane = threadIdx.x & 31, D = int(a.dim);
    constexpr int J = T::DMAX / 32;
    const int64_t row = kvq_row(T::KIND, D), words = D / 32;
    stage_q<T>(s);
    for (int g = 0; g < s.ng; ++g) {
        float* const scores = s.p.scores ? s.p.scores + (int64_t(s.row) * a.heads + s.g0 + g) * s.p.cap : nullptr;
        float top = -INFINITY, l = 0.0f, o[J] = {};
        for (int it = 0; it < s.its; ++it)
            for (int r = 0; r < T::KT; ++r) {
                const uint32_t v = s.v_begin + uint32_t(it) * T::TK + r;
                if (v >= s.v_end) break;
                const int64_t at = s.off + v + (v < s.vis.ns ? 0 : s.vis.gap);
                const unsigned char* kc = static_cast<const unsigned char*>(a.k) + at * row;
                const unsigned char* vc = static_cast<const unsigned char*>(a.v) + at * row;
                float x = 0.0f;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int d = lane + 32 * j;
                    if (d < D) x = fmaf(s.q[g * T::DMAX + d], kvq_value<T::KIND>(kc, a.k_words + at * words, d), x);
                }
#pragma unroll
                for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
                if (scores && lane == 0) scores[v] = x;
                const float n = fmaxf(top, x), f = n == top ? 1.0f : ex2(top - n), w = x == -INFINITY ? 0.0f : ex2(x - n);
                top = n;
                l = l * f + w;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int d = lane + 32 * j;
                    if (d < D) o[j] = o[j] * f + w * kvq_value<T::KIND>(vc, a.v_words + at * words, d);
                }
            }
        if (lane == 0) {
            s.m[g] = top;
            s.l[g] = l;
        }
#pragma unroll
        for (int j = 0; j < J; ++j) reinterpret_cast<float*>(s.ring)[g * T::DV + lane + 32 * j] = o[j];
    }
}

template <int KIND_, int NG_>
struct AttnKvqPlain {
    static constexpr int KIND = KIND_, NG = NG_, DMAX = 256, DV = DMAX, SPLIT = 1;
    static constexpr int CTAS = 2, RING = 16 * 1024, MAX_CTAS = kKvqMaxCtas;
    static constexpr bool HEAD_MAJOR = true;
    static constexpr int ROW = 0, KT = 16, TK = kAttnWarps * KT, EXTRA = 4, LEAST = 1;
    static __device__ __forceinline__ void states(const Segment& s) { kvq_plain_states<AttnKvqPlain>(s); }
};

template <int KIND>
cudaError_t launch_attn_kvq_kind(const AttnParams& p, const LaunchCtx& ctx) {
    if (kvq_block_heads(p.gsz) == 4) return launch_attn_kernel<AttnKvqPlain<KIND, 4>>(p, ctx);
    return launch_attn_kernel<AttnKvqPlain<KIND, 8>>(p, ctx);
}

}  // namespace q8
