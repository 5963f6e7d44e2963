// attn.cu -- attention of one token a sequence over its K/V cache.
//
// One CTA a row and K/V head; its warps take the visible entries in turn, the
// lanes of a warp the values of an entry, each with a running maximum and sum
// (softmax in one pass over K and V); the warps' states are joined at the end.
// Scores wait in the workspace until their row's sum is known, where the
// weights are accumulated.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "q8proj.h"

namespace q8 {

namespace {

constexpr int kWarps = 8;
constexpr size_t kHeader = 1024;

// The entries of a row that can be visible.
int64_t visible_cap(int64_t n_pos, int64_t window, int64_t sinks) {
    if (window < 0 || window >= n_pos || sinks >= n_pos - window) return n_pos;
    return sinks + window;
}

template <int KV>
__device__ __forceinline__ float kv_load(const void* p, int64_t i) {
    if constexpr (KV == Q8_KV_F32) return static_cast<const float*>(p)[i];
    if constexpr (KV == Q8_KV_F16) return __half2float(static_cast<const __half*>(p)[i]);
    if constexpr (KV == Q8_KV_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// The visible entries in order: entry v of nvis is cache row v + (v < ns ? 0 : gap).
struct Visible {
    int64_t nvis, ns, gap;
};

__device__ __forceinline__ Visible visible(int pos, int64_t n_pos, int64_t window, int64_t sinks,
                                           bool report, int* err) {
    if (pos < -1 || pos >= n_pos) {
        if (report) atomicExch(err, Q8_DEVERR_POSITION);
        return {0, 0, 0};
    }
    const int64_t n = int64_t(pos) + 1;
    if (window < 0 || window >= n) return {n, n, 0};
    const int64_t ns = sinks < n - window ? sinks : n - window;
    return {ns + window, ns, n - window - ns};
}

template <int KV>
__global__ void __launch_bounds__(32 * kWarps) attn_kernel(const AttnArgs a, int64_t cap, int* err) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ float s_o[kWarps][256], s_m[kWarps], s_l[kWarps];
    const int64_t m = blockIdx.y, h = blockIdx.x, D = a.dim, group = a.heads / a.kv_heads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Visible vis = visible(a.pos[m], a.n_pos, a.window, a.sinks, h == 0 && threadIdx.x == 0, err);
    for (int64_t g = h * group; g < (h + 1) * group; ++g) {
        const float* q = a.q + m * a.ldq + g * D;
        float* scores = a.acc ? static_cast<float*>(a.ws) + kHeader / 4 + (m * a.heads + g) * cap : nullptr;
        float qr[8], o[8];
        for (int j = 0; j < 8; ++j) {
            const int d = lane + 32 * j;
            qr[j] = d < D ? q[d] * a.scale : 0.0f;
            o[j] = 0.0f;
        }
        const auto score = [&](int64_t at) {
            float s = 0.0f;
            for (int j = 0; j < 8; ++j)
                if (lane + 32 * j < D) s = fmaf(qr[j], kv_load<KV>(a.k, at + lane + 32 * j), s);
            for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
            return s;
        };
        float top = -INFINITY, l = 0.0f;
        for (int64_t v = warp; v < vis.nvis; v += kWarps) {
            const int64_t at = ((m * a.n_pos + v + (v < vis.ns ? 0 : vis.gap)) * a.kv_heads + h) * D;
            const float s = score(at), nm = fmaxf(top, s), ref = nm == -INFINITY ? 0.0f : nm;
            if (scores && lane == 0) scores[v] = s;
            const float c = expf(top - ref), p = expf(s - ref);
            l = l * c + p;
            for (int j = 0; j < 8; ++j)
                if (lane + 32 * j < D) o[j] = o[j] * c + p * kv_load<KV>(a.v, at + lane + 32 * j);
            top = nm;
        }
        for (int j = 0; j < 8; ++j) s_o[warp][lane + 32 * j] = o[j];
        if (lane == 0) {
            s_m[warp] = top;
            s_l[warp] = l;
        }
        __syncthreads();
        float all = -INFINITY, sum = 0.0f;
        for (int w = 0; w < kWarps; ++w) all = fmaxf(all, s_m[w]);
        const float ref = all == -INFINITY ? 0.0f : all;
        for (int w = 0; w < kWarps; ++w) sum += s_l[w] * expf(s_m[w] - ref);
        for (int64_t d = threadIdx.x; d < D; d += 32 * kWarps) {
            float v = 0.0f;
            for (int w = 0; w < kWarps; ++w) v += s_o[w][d] * expf(s_m[w] - ref);
            a.out[m * a.ldo + g * D + d] = vis.nvis ? v / sum : 0.0f;
        }
        if (a.acc) {
            float* acc = a.acc + (m * a.kv_heads + h) * a.n_pos;
            for (int64_t v = warp; v < vis.nvis; v += kWarps) {
                const int64_t i = v + (v < vis.ns ? 0 : vis.gap);
                if (lane == 0) acc[i] += expf(scores[v] - ref) / sum;
            }
        }
        __syncthreads();
    }
}

}  // namespace

size_t attn_workspace_bytes(int64_t rows, int64_t heads, int64_t, int64_t, int64_t n_pos, int64_t window,
                            int64_t sinks, bool acc) {
    return kHeader + (acc ? size_t(rows * heads) * size_t(visible_cap(n_pos, window, sinks)) * 4 : 0);
}

cudaError_t launch_attn(const AttnArgs& a, const LaunchCtx& ctx) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attrs[1];
    const int64_t cap = visible_cap(a.n_pos, a.window, a.sinks);
    cfg.gridDim = dim3(unsigned(a.kv_heads), unsigned(a.rows));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = ctx.stream;
    cfg.numAttrs = pdl_attrs(ctx, attrs);
    cfg.attrs = attrs;
    if (a.kv_type == Q8_KV_F32) return cudaLaunchKernelEx(&cfg, attn_kernel<Q8_KV_F32>, a, cap, ctx.dev_err);
    if (a.kv_type == Q8_KV_F16) return cudaLaunchKernelEx(&cfg, attn_kernel<Q8_KV_F16>, a, cap, ctx.dev_err);
    return cudaLaunchKernelEx(&cfg, attn_kernel<Q8_KV_BF16>, a, cap, ctx.dev_err);
}

}  // namespace q8
