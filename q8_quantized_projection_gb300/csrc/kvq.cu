// kvq.cu -- tokens stored into quantised K/V caches, and entries read back as floats.
//
// A thread has eight values of one head of one token; four neighbours share a block and
// exchange its extremes by two shuffles.  A CTA takes up to 256 / (head_dim / 8) tokens of
// one head, whose codes and words are one run of the cache, or, where a row has fewer
// tokens, those of several heads.
#include "kvq.cuh"

#include <cuda_bf16.h>

namespace q8 {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kSegment = 65536;   // tokens a grid plane

template <typename F>
__device__ __forceinline__ void load8(const F* p, float (&x)[8]) {
    if constexpr (sizeof(F) == 4) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
        const int4 a = __ldcs(reinterpret_cast<const int4*>(p));
        const int w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f;
            if constexpr (std::is_same<F, __half>::value)
                f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            else
                f = make_float2(__int_as_float(w[i] << 16), __int_as_float(w[i] & int(0xffff0000)));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
}

template <typename F>
__device__ __forceinline__ void store8(F* p, const float (&x)[8]) {
    if constexpr (sizeof(F) == 4) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
        __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
    } else {
        int w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<F, __half>::value) {
                const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const int*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const int*>(&h);
            }
        }
        __stcs(reinterpret_cast<int4*>(p), make_int4(w[0], w[1], w[2], w[3]));
    }
}

// What a thread has: its eight values' place in the floats and in a cache.
struct Place {
    bool in;             // there is such a token, and its entry lies in the cache
    bool v;              // of V
    int64_t at;          // values from the floats' beginning
    int64_t entry;       // (row, head, entry) in one line
    int c;               // which eight of the head
};

__device__ __forceinline__ Place place(const KvqIoArgs& a, int slots, int tb, int* err) {
    const int c8 = int(a.dim) / 8, slot = threadIdx.x / c8, c = threadIdx.x - slot * c8;
    const int64_t m = blockIdx.z, t_first = int64_t(blockIdx.y) * kSegment;
    const int ub = slots / tb, units = int(a.kv_heads) * 2, ublocks = (units + ub - 1) / ub;
    const int uu = slot / tb, unit = int(blockIdx.x % ublocks) * ub + uu;
    const int64_t t = t_first + int64_t(blockIdx.x / ublocks) * tb + (slot - uu * tb);
    const int64_t t_end = a.T < t_first + kSegment ? a.T : t_first + kSegment;
    Place p;
    const int64_t len = a.lens ? a.lens[m] : a.T, pos = a.pos ? a.pos[m] : 0;
    p.in = slot < slots && uu < ub && unit < units && t < t_end && t < len;
    const int64_t i = pos + t;
    if (p.in && (i < 0 || i >= a.n_pos)) {
        p.in = false;
        if (c == 0) atomicExch(err, Q8_DEVERR_POSITION);
    }
    p.v = unit >= a.kv_heads;
    const int64_t h = p.v ? unit - a.kv_heads : unit;
    p.at = m * a.ld_row + t * a.ld_tok + h * a.dim + c * 8;
    p.entry = (m * a.kv_heads + h) * a.n_pos + i;
    p.c = c;
    return p;
}

template <typename F, int KIND>
__global__ void __launch_bounds__(kThreads) kvq_store_kernel(const KvqIoArgs a, int slots, int tb, int* err) {
    pdl_wait();
    pdl_launch_dependents();
    const Place p = place(a, slots, tb, err);
    float x[8] = {};
    if (p.in) load8(static_cast<const F*>(p.v ? a.v : a.k) + p.at, x);
    // (magnitudes as integers: infinities and NaN are the largest)
    uint32_t most = 0;
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        most = max(most, __float_as_uint(x[i]) & 0x7fffffffu);
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int k = 1; k < 4; k *= 2) {
        most = max(most, __shfl_xor_sync(0xffffffffu, most, k));
        if constexpr (KIND == Q8_KVQ_U4) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, k));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, k));
        }
    }
    if (!p.in) return;
    const int64_t row = p.entry * kvq_row(KIND, a.dim);
    uint32_t* word = static_cast<uint32_t*>(p.v ? a.v_words : a.k_words) + p.entry * (a.dim / 32) + p.c / 4;
    unsigned char* codes = static_cast<unsigned char*>(p.v ? a.v_codes : a.k_codes) + row;
    bool bad = most >= 0x7f800000u;                    // the block reads back as NaN
    if constexpr (KIND == Q8_KVQ_I8) {
        const float d = bad ? __int_as_float(0x7fc00000) : __fdiv_rn(__uint_as_float(most), 127.0f);
        uint32_t w[2] = {0u, 0u};
        if (!bad) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i / 4] |= uint32_t(quantize_code(x[i], d, 127.0f) & 255) << (8 * (i & 3));
        }
        *reinterpret_cast<uint2*>(codes + p.c * 8) = make_uint2(w[0], w[1]);
        if ((p.c & 3) == 0) *word = __float_as_uint(d);
    } else {
        const __half s = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f)), m = __float2half_rn(lo);
        const float sf = __half2float(s), mf = __half2float(m);
        bad = bad || isinf(sf) || isinf(mf);
        uint32_t w = 0;
        if (!bad && sf != 0.0f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = roundf(__fdiv_rn(__fsub_rn(x[i], mf), sf));
                w |= uint32_t(fminf(fmaxf(q, 0.0f), 15.0f)) << (4 * i);
            }
        }
        *reinterpret_cast<uint32_t*>(codes + p.c * 4) = w;
        if ((p.c & 3) == 0)
            *word = bad ? 0x7e007e00u : uint32_t(__half_as_ushort(s)) | uint32_t(__half_as_ushort(m)) << 16;
    }
}

template <typename F, int KIND>
__global__ void __launch_bounds__(kThreads) kvq_load_kernel(const KvqIoArgs a, int slots, int tb, int* err) {
    pdl_wait();
    pdl_launch_dependents();
    const Place p = place(a, slots, tb, err);
    if (!p.in) return;
    const int64_t row = p.entry * kvq_row(KIND, a.dim);
    const uint32_t word = static_cast<const uint32_t*>(p.v ? a.v_words : a.k_words)[p.entry * (a.dim / 32) + p.c / 4];
    const unsigned char* codes = static_cast<const unsigned char*>(p.v ? a.v_codes : a.k_codes) + row;
    float x[8];
    if constexpr (KIND == Q8_KVQ_I8) {
        const uint2 w = *reinterpret_cast<const uint2*>(codes + p.c * 8);
        const float d = __uint_as_float(word);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = byte_as_float(int(i < 4 ? w.x : w.y), i & 3) * d;
    } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + p.c * 4);
        const float2 sm = kvq_scale_min(word);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(float(w >> (4 * i) & 15u), sm.x, sm.y);   // (the product is exact)
    }
    store8(static_cast<F*>(p.v ? a.v : a.k) + p.at, x);
}

template <typename F, int KIND, bool STORE>
cudaError_t launch_io_kernel(const KvqIoArgs& a, const LaunchCtx& ctx) {
    const int slots = kThreads / int(a.dim / 8);
    const int tb = a.T < slots ? int(a.T) : slots, ub = slots / tb;
    const int64_t units = 2 * a.kv_heads, seg = a.T < kSegment ? a.T : kSegment;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attrs[1];
    cfg.gridDim = dim3(unsigned((units + ub - 1) / ub * ((seg + tb - 1) / tb)), unsigned((a.T + kSegment - 1) / kSegment),
                       unsigned(a.rows));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = ctx.stream;
    cfg.numAttrs = pdl_attrs(ctx, attrs);
    cfg.attrs = attrs;
    if constexpr (STORE) return cudaLaunchKernelEx(&cfg, kvq_store_kernel<F, KIND>, a, slots, tb, ctx.dev_err);
    return cudaLaunchKernelEx(&cfg, kvq_load_kernel<F, KIND>, a, slots, tb, ctx.dev_err);
}

template <bool STORE>
cudaError_t launch_io(const KvqIoArgs& a, const LaunchCtx& ctx) {
    if (a.kind == Q8_KVQ_I8) {
        if (a.type == Q8_KV_F32) return launch_io_kernel<float, Q8_KVQ_I8, STORE>(a, ctx);
        if (a.type == Q8_KV_F16) return launch_io_kernel<__half, Q8_KVQ_I8, STORE>(a, ctx);
        return launch_io_kernel<__nv_bfloat16, Q8_KVQ_I8, STORE>(a, ctx);
    }
    if (a.type == Q8_KV_F32) return launch_io_kernel<float, Q8_KVQ_U4, STORE>(a, ctx);
    if (a.type == Q8_KV_F16) return launch_io_kernel<__half, Q8_KVQ_U4, STORE>(a, ctx);
    return launch_io_kernel<__nv_bfloat16, Q8_KVQ_U4, STORE>(a, ctx);
}

}  // namespace

cudaError_t launch_kvq_store(const KvqIoArgs& a, const LaunchCtx& ctx) { return launch_io<true>(a, ctx); }
cudaError_t launch_kvq_load(const KvqIoArgs& a, const LaunchCtx& ctx) { return launch_io<false>(a, ctx); }

}  // namespace q8
