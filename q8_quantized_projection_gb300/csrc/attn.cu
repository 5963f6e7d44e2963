// attn.cu -- attn_decode's host side: the workspace, the choice of kernel, and
// the kernel that accumulates the weights once a row's sums are known.
#include "attn.cuh"

namespace q8 {

cudaError_t launch_attn_f32(const AttnParams& p, const LaunchCtx& ctx);
cudaError_t launch_attn_f16(const AttnParams& p, const LaunchCtx& ctx);
cudaError_t launch_attn_bf16(const AttnParams& p, const LaunchCtx& ctx);

namespace {

constexpr int kAccThreads = 256, kAccPer = 4;

// acc[m][h][i] += the sum over K/V head h's query heads of 2^(s - r) / sum.
// Scores and weights once each: 4 bytes a head and entry against the cache's
// hundreds.  One thread an entry, so nothing is added atomically.  Positions and
// the first old values are read before the wait: the attention kernel, whose
// scores it waits for, lets this one begin behind its own wait, so whatever wrote
// those is done.
__global__ void __launch_bounds__(kAccThreads) attn_acc_kernel(const AttnParams p) {
    const AttnArgs& a = p.a;
    const int64_t m = blockIdx.x / a.kv_heads, h = blockIdx.x % a.kv_heads, group = a.heads / a.kv_heads;
    const Visible vis = visible(__ldcg(a.pos + m), a.n_pos, a.window, a.sinks);
    float* acc = a.acc + int64_t(blockIdx.x) * a.n_pos;
    const int64_t step = int64_t(gridDim.y) * kAccThreads * kAccPer;
    int64_t v0 = int64_t(blockIdx.y) * kAccThreads * kAccPer + threadIdx.x;
    float old[kAccPer];
    const auto fetch = [&] {
#pragma unroll
        for (int j = 0; j < kAccPer; ++j) {
            const int64_t v = v0 + j * kAccThreads;
            if (v < vis.nvis) old[j] = __ldcg(acc + v + (v < vis.ns ? 0 : vis.gap));
        }
    };
    fetch();
    pdl_wait();
    pdl_launch_dependents();
    while (v0 < vis.nvis) {
        float w[kAccPer] = {};
#pragma unroll 4
        for (int64_t g = m * a.heads + h * group; g < m * a.heads + (h + 1) * group; ++g) {
            const float2 ml = p.ml[g];
            const float* s = p.scores + g * p.cap;
#pragma unroll
            for (int j = 0; j < kAccPer; ++j) {
                const int64_t v = v0 + j * kAccThreads;
                if (v < vis.nvis) w[j] += ex2(s[v] - ml.x) * ml.y;
            }
        }
#pragma unroll
        for (int j = 0; j < kAccPer; ++j) {
            const int64_t v = v0 + j * kAccThreads;
            if (v < vis.nvis) acc[v + (v < vis.ns ? 0 : vis.gap)] = old[j] + w[j];
        }
        v0 += step;
        fetch();
    }
}

// The entries of a row that can be visible.
int64_t visible_cap(int64_t n_pos, int64_t window, int64_t sinks) {
    if (window < 0 || window >= n_pos || sinks >= n_pos - window) return n_pos;
    return sinks + window;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Query heads a block: a K/V head's group in equal blocks of at most 8.
int block_heads(int64_t group) {
    const int64_t nb = (group + 7) / 8;
    return int((group + nb - 1) / nb);
}

size_t part_bytes(int gsz, int64_t dim) {
    const int ng = gsz <= 2 ? gsz : gsz <= 4 ? 4 : 8;
    return round256(size_t(2) * kAttnMaxCtas * attn_slot(ng, dim) * 4);
}

}  // namespace

// [tickets][partial states][per query head: reference, 1 / sum][scores]
size_t attn_workspace_bytes(int64_t rows, int64_t heads, int64_t kv_heads, int64_t dim, int64_t n_pos,
                            int64_t window, int64_t sinks, bool acc) {
    size_t n = kCounterBytes + part_bytes(block_heads(heads / kv_heads), dim);
    if (acc)
        n += round256(size_t(rows * heads) * 8) +
             round256(size_t(rows * heads) * size_t(visible_cap(n_pos, window, sinks)) * 4);
    return n;
}

cudaError_t launch_attn(const AttnArgs& a, const LaunchCtx& ctx) {
    AttnParams p{};
    p.a = a;
    const int64_t group = a.heads / a.kv_heads;
    p.gsz = block_heads(group);
    p.nb = int((group + p.gsz - 1) / p.gsz);
    p.cap = visible_cap(a.n_pos, a.window, a.sinks);
    // all tiles of all units number below 2^31: a stage of all warps holds 8
    // entries at least, and a unit counts at most 16 tiles more
    p.tile_its = 1;
    while (a.rows * a.kv_heads * p.nb * (p.cap / (8 * p.tile_its) + 17) > INT32_MAX) p.tile_its *= 2;
    p.qscale = float(double(a.scale) * 1.4426950408889634);
    p.err = ctx.dev_err;
    unsigned char* ws = static_cast<unsigned char*>(a.ws) + kCounterBytes;
    p.part = reinterpret_cast<float*>(ws);
    if (a.acc) {
        ws += part_bytes(p.gsz, a.dim);
        p.ml = reinterpret_cast<float2*>(ws);
        p.scores = reinterpret_cast<float*>(ws + round256(size_t(a.rows * a.heads) * 8));
    }
    const cudaError_t e = a.kv_type == Q8_KV_F32   ? launch_attn_f32(p, ctx)
                          : a.kv_type == Q8_KV_F16 ? launch_attn_f16(p, ctx)
                                                   : launch_attn_bf16(p, ctx);
    if (e != cudaSuccess || !a.acc || p.cap == 0) return e;
    const int64_t units = a.rows * a.kv_heads, chunk = kAccThreads * kAccPer;
    int64_t gy = (p.cap + chunk - 1) / chunk;
    const int64_t most = (int64_t(16) * ctx.num_sms + units - 1) / units;   // 16 CTAs an SM in all
    gy = gy < most ? gy : most;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attrs[1];
    cfg.gridDim = dim3(unsigned(units), unsigned(gy));
    cfg.blockDim = dim3(kAccThreads);
    cfg.stream = ctx.stream;
    cfg.numAttrs = pdl_attrs(ctx, attrs);
    cfg.attrs = attrs;
    return cudaLaunchKernelEx(&cfg, attn_acc_kernel, p);
}

}  // namespace q8
