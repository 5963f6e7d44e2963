// evict.cu -- eviction from the K/V caches by accumulated attention weight.
//
// evict_select_kernel, one CTA a row and K/V head: the smallest kept weight by
// a binary search over the 32 bits of an ordered key, then one ordered pass
// that lists the kept entries and moves acc.  evict_move_kernel: K and V move
// to the front, in place.  Entry j of the result comes from an entry idx[j]
// >= j, so a tile of rows may be written as soon as the tile has been read:
// what it overwrites is read by itself and earlier tiles only.
#include "common.cuh"
#include "launch.h"
#include "q8proj.h"

namespace q8 {

namespace {

constexpr int kSelThreads = 1024, kMoveThreads = 256;

// Order of the weights as unsigned integers: NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (isnan(w)) return 0u;
    const uint32_t b = __float_as_uint(w + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Exclusive prefix sum over the CTA's threads; total in *all.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* s_warp, uint32_t* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    uint32_t before = 0, total = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
        const uint32_t t = s_warp[w];
        if (w < warp) before += t;
        total += t;
    }
    __syncthreads();
    *all = total;
    return before + x - v;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a, int* err) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ uint32_t s_warp[kSelThreads / 32];
    const int64_t m = blockIdx.y, h = blockIdx.x, unit = m * a.kv_heads + h;
    const int pos = a.pos[m];
    const bool bad = pos < -1 || pos >= a.n_pos;
    if (bad && h == 0 && threadIdx.x == 0) atomicExch(err, Q8_DEVERR_POSITION);
    const int64_t n = bad ? 0 : int64_t(pos) + 1;
    const float* acc = a.acc + unit * a.n_pos;
    float* new_acc = a.new_acc + unit * a.n_pos;
    int32_t* kept = a.kept ? a.kept + unit * a.budget : nullptr;
    int32_t* idx = static_cast<int32_t*>(a.ws) + unit * a.budget;
    if (n <= a.budget) {
        for (int64_t i = threadIdx.x; i < a.n_pos; i += kSelThreads)
            if (new_acc != acc) new_acc[i] = acc[i];
        for (int64_t i = threadIdx.x; i < a.budget; i += kSelThreads)
            if (kept) kept[i] = i < n ? int32_t(i) : -1;
        return;
    }
    const int64_t lo = a.sinks, hi = n - a.recent;
    const uint32_t need = uint32_t(a.budget - a.sinks - a.recent);
    // the largest key that at least `need` entries reach (0xffffffff: need = 0)
    uint32_t t = 0, above = 0;
    if (need == 0) {
        t = 0xffffffffu;
    } else {
        for (int b = 31; b >= 0; --b) {
            const uint32_t cand = t | (1u << b);
            uint32_t c = 0, all;
            for (int64_t i = lo + threadIdx.x; i < hi; i += kSelThreads) c += weight_key(acc[i]) >= cand;
            block_scan(c, s_warp, &all);
            if (all >= need) t = cand;
        }
        uint32_t c = 0;
        for (int64_t i = lo + threadIdx.x; i < hi; i += kSelThreads) c += weight_key(acc[i]) > t;
        block_scan(c, s_warp, &above);
    }
    const uint32_t ties = need - above;   // entries equal to t that stay, the first ones
    uint32_t done = 0, ties_seen = 0;
    for (int64_t i0 = 0; i0 < n; i0 += kSelThreads) {
        const int64_t i = i0 + threadIdx.x;
        float w = 0.0f;
        bool keep = false, tie = false;
        if (i < n) {
            w = acc[i];
            keep = i < lo || i >= hi;
            if (!keep && need) {
                const uint32_t key = weight_key(w);
                keep = key > t;
                tie = key == t;
            }
        }
        uint32_t all;
        const uint32_t tb = block_scan(tie, s_warp, &all);
        keep = keep || (tie && ties_seen + tb < ties);
        ties_seen += all;
        const uint32_t kb = block_scan(keep, s_warp, &all);
        if (keep) {
            const uint32_t j = done + kb;
            idx[j] = int32_t(i);
            if (kept) kept[j] = int32_t(i);
            new_acc[j] = w;
        }
        done += all;
    }
    __syncthreads();
    for (int64_t i = a.budget + threadIdx.x; i < a.n_pos; i += kSelThreads) new_acc[i] = 0.0f;
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, int elt) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t m = blockIdx.y, h = blockIdx.x, unit = m * a.kv_heads + h;
    const int pos = a.pos[m];
    const bool over = pos < a.n_pos && int64_t(pos) + 1 > a.budget;
    if (!over) return;
    const int64_t chunks = a.dim * elt / 16, pitch = a.kv_heads * a.dim * elt;
    unsigned char* base = static_cast<unsigned char*>(blockIdx.z ? a.v : a.k) +
                          m * a.n_pos * pitch + h * a.dim * elt;
    const int32_t* idx = static_cast<const int32_t*>(a.ws) + unit * a.budget;
    for (int64_t c0 = 0; c0 < a.budget * chunks; c0 += kMoveThreads) {
        const int64_t c = c0 + threadIdx.x, j = c / chunks, col = (c % chunks) * 16;
        int4 x{};
        const bool in = j < a.budget;
        if (in) x = *reinterpret_cast<const int4*>(base + int64_t(idx[j]) * pitch + col);
        __syncthreads();
        if (in) *reinterpret_cast<int4*>(base + j * pitch + col) = x;
    }
}

// after the moves: the new positions (pos may be new_pos)
__global__ void evict_pos_kernel(const EvictArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int m = threadIdx.x;
    if (m >= a.rows) return;
    const int pos = a.pos[m];
    a.new_pos[m] = pos < a.n_pos && int64_t(pos) + 1 > a.budget ? int32_t(a.budget - 1) : pos;
}

}  // namespace

size_t evict_workspace_bytes(int64_t rows, int64_t kv_heads, int64_t budget) {
    return size_t(rows * kv_heads) * size_t(budget) * sizeof(int32_t);
}

cudaError_t launch_evict(const EvictArgs& a, const LaunchCtx& ctx) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attrs[1];
    cfg.stream = ctx.stream;
    cfg.numAttrs = pdl_attrs(ctx, attrs);
    cfg.attrs = attrs;
    cfg.gridDim = dim3(unsigned(a.kv_heads), unsigned(a.rows));
    cfg.blockDim = dim3(kSelThreads);
    cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, ctx.dev_err);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(unsigned(a.kv_heads), unsigned(a.rows), 2);
    cfg.blockDim = dim3(kMoveThreads);
    e = cudaLaunchKernelEx(&cfg, evict_move_kernel, a, a.kv_type == Q8_KV_F32 ? 4 : 2);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&cfg, evict_pos_kernel, a);
}

}  // namespace q8
