// kvq.cu -- tokens stored into quantised K/V caches, and entries read back as floats.
//
// A thread has some values of one head of one token: 16 of a store, where two neighbours
// share a block and exchange its extremes, and 16 bytes of them of a load.  A CTA takes as many tokens of
// one head as it has threads for, whose codes and words are one run of the cache, or, where
// a row has fewer tokens, those of several heads.
//
// What bounds them.  Long prompts: a store of 16-bit floats its instructions (0.8 issued a clock; some
// 18 a value, of which 9 are the code and, where a quotient near it is near a half, 13 more to
// decide it; 4 rows of 16384 tokens, 8 K/V heads of 128 values: bf16 80 us in 4 bits, 85 in
// 8, 4.4 and 4.9 TB/s; binary32 102 and 111, 6.1 and 6.2 TB/s); a load HBM (58 and 66 us into
// bf16, 98 and 106 into binary32, 6.1 to 6.5 TB/s).  Single tokens: the launch, 1.8 us each.
// A reciprocal in place of divisions, three-operand extremes and 16 values a thread made the
// first 102 us of 167, eight turns 96, halves decided for a few values at a time 89 (8 bits: 108
// to 96); turns that read ahead took a load from 155 to 131 us (2 rows of 65536, bf16), 32-bit
// places within a grid plane to 113.
#include "kvq.cuh"

#include <cuda_bf16.h>

#include <type_traits>

namespace q8 {

namespace {

// (Of 256, whose registers fit twice an SM and leave a quarter of them idle, the stores above took
// 89 and 96, 105 and 113 us; of 64 the same as here.)
constexpr int kThreads = 128;
constexpr int64_t kSegment = 65536;   // tokens a grid plane

// Values a thread: of a load, 16 bytes of floats (twice as many, and lanes that write every other
// 16 bytes, read back 2 x 65536 bf16 entries in 130 us, not 113).
constexpr int kStored = 16;
template <typename F>
constexpr int kLoaded = 16 / int(sizeof(F));

// kStored floats as they lie in memory.
template <typename F>
struct Floats {
    int4 w[sizeof(F)];
};

template <typename F>
__device__ __forceinline__ void expand(const Floats<F>& e, float (&x)[kStored]) {
#pragma unroll
    for (int i = 0; i < int(sizeof(F)); ++i) {
        const int w[4] = {e.w[i].x, e.w[i].y, e.w[i].z, e.w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(F) == 4) {
                x[4 * i + j] = __int_as_float(w[j]);
            } else if constexpr (std::is_same<F, __half>::value) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                x[8 * i + 2 * j] = f.x, x[8 * i + 2 * j + 1] = f.y;
            } else {
                x[8 * i + 2 * j] = __int_as_float(w[j] << 16);
                x[8 * i + 2 * j + 1] = __int_as_float(w[j] & int(0xffff0000));
            }
        }
    }
}

template <typename F, int V>
__device__ __forceinline__ void put(F* p, const float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 16 / int(sizeof(F))) {
        if constexpr (sizeof(F) == 4) {
            __stcs(reinterpret_cast<float4*>(p + i), make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
        } else {
            int w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (std::is_same<F, __half>::value) {
                    const __half2 h = __floats2half2_rn(x[i + 2 * j], x[i + 2 * j + 1]);
                    w[j] = *reinterpret_cast<const int*>(&h);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(x[i + 2 * j], x[i + 2 * j + 1]);
                    w[j] = *reinterpret_cast<const int*>(&h);
                }
            }
            __stcs(reinterpret_cast<int4*>(p + i), make_int4(w[0], w[1], w[2], w[3]));
        }
    }
}

// x[i] of a register array, by selection.
__device__ __forceinline__ float pick(const float (&x)[kStored], int i) {
    float y = x[0];
#pragma unroll
    for (int j = 1; j < kStored; ++j) y = i == j ? x[j] : y;
    return y;
}

// The smallest and the largest of a thread's values and its neighbour's (a block); NaN if one is.
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
    float r;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float2 block_range(const Floats<float>& e) {
    float x[kStored];
    expand(e, x);
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i + 1 < kStored; i += 2) {
        lo = min_nan(lo, x[i], x[i + 1]);
        hi = max_nan(hi, x[i], x[i + 1]);
    }
    lo = min_nan(lo, x[kStored - 1]);
    hi = max_nan(hi, x[kStored - 1]);
    return make_float2(min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, 1)), max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, 1)));
}

// 16-bit types in their own, two at a time; then the smallest and the largest's negative as one word.
template <typename F>
__device__ __forceinline__ float2 block_range(const Floats<F>& e) {
    using P = typename std::conditional<std::is_same<F, __half>::value, __half2, __nv_bfloat162>::type;
    const int w[8] = {e.w[0].x, e.w[0].y, e.w[0].z, e.w[0].w, e.w[1].x, e.w[1].y, e.w[1].z, e.w[1].w};
    P lo = *reinterpret_cast<const P*>(&w[0]), hi = lo;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        const P x = *reinterpret_cast<const P*>(&w[i]);
        lo = __hmin2_nan(lo, x);
        hi = __hmax2_nan(hi, x);
    }
    const uint32_t l = *reinterpret_cast<const uint32_t*>(&lo), h = *reinterpret_cast<const uint32_t*>(&hi) ^ 0x80008000u;
    const uint32_t first = __byte_perm(l, h, 0x5410), second = __byte_perm(l, h, 0x7632);
    P m = __hmin2_nan(*reinterpret_cast<const P*>(&first), *reinterpret_cast<const P*>(&second));
    const uint32_t other = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&m), 1);
    m = __hmin2_nan(m, *reinterpret_cast<const P*>(&other));
    return make_float2(float(m.x), -float(m.y));
}

// 2^23 plus byte j of w (a conversion instruction runs at a quarter of this one's rate).
__device__ __forceinline__ float byte_above_2_23(uint32_t w, int j) {
    return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540 + j));
}

constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: a sum with it is an integer in its low bits

// round_half_away(x / d) as the formats define it, the quotient rounded to binary32 first, of
// x >= 0 and 2^-100 < d < 2^126, from any r near enough that the answer is floor(r) or one
// more.  With h = floor(r) + 1/2, the rounded quotient reaches h where x / d >= h - u, u half
// a step of binary32 below h (h is even, so u itself rounds up): where x - h d, exact in one
// multiply-add (its operands cancel but for some bits), is at least -u d.
// `tiny` is d * 2^-24.
__device__ __forceinline__ float half_away(float x, float d, float tiny, float r) {
    const float n = __fsub_rn(__fadd_rd(r, 8388608.0f), 8388608.0f);
    const float rest = fmaf(-(n + 0.5f), d, x);
    // (the binade below h: floor(r)'s, and that of 1/4 below 1/2, whatever r is rounded to)
    const float binade = __uint_as_float(__float_as_uint(fmaxf(n, 0.25f)) & 0x7f800000u);
    return rest >= -(binade * tiny) ? n + 1.0f : n;
}

// 1 / x within 2^-23, of a normal x and result.
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Codes by way of 1 / d.  The product is within 127 * 1.5 * 2^-23 of the quotient (1 / d, and
// its own rounding) and that within 127 * 2^-24 of its rounding, 3.1e-5 in all: where it lies
// 2^-14 or more from every half, both round to the same integer.  Elsewhere (of 16-bit values
// many quotients are halves) half_away decides.
template <int G>
__device__ __forceinline__ void codes_i8(const float (&x)[kStored], float d, uint32_t (&w)[4]) {
    const float inv = reciprocal(d);
    float far[kStored / G] = {}, n[kStored];
#pragma unroll
    for (int i = 0; i < kStored; ++i) {
        const float r = __fmul_rn(x[i], inv);
        n[i] = __fadd_rn(r, kMagic);
        far[i / G] = fmaxf(far[i / G], fabsf(r - __fsub_rn(n[i], kMagic)));
    }
    if (!(d > 0x1p-100f && d < 0x1p126f)) {
#pragma unroll 1
        for (int i = 0; i < kStored; ++i) {
            const uint32_t code = uint32_t(quantize_code(pick(x, i), d, 127.0f) & 255) << (8 * (i & 3));
            w[i / 4] = i & 3 ? w[i / 4] | code : code;
        }
        return;
    }
    const float tiny = d * 0x1p-24f;
#pragma unroll
    for (int g = 0; g < kStored; g += G) {
        if (far[g / G] < 0.5f - 0x1p-14f) continue;
#pragma unroll
        for (int i = g; i < g + G; ++i)
            n[i] = __fadd_rn(copysignf(half_away(fabsf(x[i]), d, tiny, __fmul_rn(fabsf(x[i]), inv)), x[i]), kMagic);
    }
#pragma unroll
    for (int i = 0; i < kStored / 4; ++i)
        w[i] = __byte_perm(__byte_perm(__float_as_uint(n[4 * i]), __float_as_uint(n[4 * i + 1]), 0x0040),
                           __byte_perm(__float_as_uint(n[4 * i + 2]), __float_as_uint(n[4 * i + 3]), 0x0040), 0x5410);
}

// The same of (x - m) / s, which the rounding of m may push out of [0, 15] (lo, hi: the smallest
// and largest x).  Of at most 15.25, the product is within 3.7e-6 of the rounded quotient.
template <int G>
__device__ __forceinline__ uint2 codes_u4(const float (&x)[kStored], float s, float m, float lo, float hi) {
    const float inv = s == 0.0f ? 0.0f : reciprocal(s);
    float far[kStored / G] = {}, n[kStored];
#pragma unroll
    for (int i = 0; i < kStored; ++i) {
        const float r = __fmul_rn(__fsub_rn(x[i], m), inv);
        n[i] = __fsub_rn(__fadd_rn(r, kMagic), kMagic);
        far[i / G] = fmaxf(far[i / G], fabsf(r - n[i]));
    }
    // (neither where s is 0: those products are)
    const bool outside = (lo - m) * inv < -0.25f || (hi - m) * inv > 15.25f;
    const float tiny = s * 0x1p-24f;
#pragma unroll
    for (int g = 0; g < kStored; g += G) {
        if (far[g / G] < 0.5f - 0x1p-17f && !outside) continue;
#pragma unroll
        for (int i = g; i < g + G; ++i) {
            const float y = fminf(fmaxf(__fsub_rn(x[i], m), 0.0f), 15.0f * s);
            n[i] = half_away(y, s, tiny, __fmul_rn(y, inv));
        }
    }
    uint32_t b[kStored / 2];
#pragma unroll
    for (int i = 0; i < kStored / 2; ++i) b[i] = __float_as_uint(__fadd_rn(fmaf(n[2 * i + 1], 16.0f, n[2 * i]), kMagic));
    return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
}

// A thread's V values of a head; its tokens are `first`, counted from the grid plane's
// first one, and every tb-th behind.
struct Place {
    int first, end;      // the row's tokens end there
    int lo, hi;          // those whose entries lie in the cache
    int64_t at;          // the first token's floats
    int64_t entry;       // and entry, (row, head, entry) in one line
    bool v;              // of V
    int c;               // which V of the head
};

template <int V>
__device__ __forceinline__ Place place(const KvqIoArgs& a, int slots, int tb, int every) {
    const int cv = int(a.dim) / V, slot = threadIdx.x / cv, c = threadIdx.x - slot * cv;
    const int64_t m = blockIdx.z, plane = int64_t(blockIdx.y) * kSegment;
    const int ub = slots / tb, units = int(a.kv_heads) * 2, ublocks = (units + ub - 1) / ub;
    const int uu = slot / tb, block = int(blockIdx.x) / ublocks, unit = (int(blockIdx.x) - block * ublocks) * ub + uu;
    Place p;
    p.first = block * every + (slot - uu * tb);
    const int64_t len = a.lens ? a.lens[m] : a.T, pos = a.pos ? a.pos[m] : 0;
    const auto within = [&](int64_t t) { return int(t < plane ? 0 : t > plane + kSegment ? kSegment : t - plane); };
    p.end = slot < slots && uu < ub && unit < units ? within(len < a.T ? len : a.T) : 0;
    p.lo = within(-pos);
    p.hi = within(a.n_pos - pos);
    p.v = unit >= a.kv_heads;
    const int64_t h = p.v ? unit - a.kv_heads : unit;
    p.at = m * a.ld_row + (plane + p.first) * a.ld_tok + h * a.dim + c * V;
    p.entry = (m * a.kv_heads + h) * a.n_pos + pos + plane + p.first;
    p.c = c;
    return p;
}

// Whether token t is the row's, and its entry in the cache.
__device__ __forceinline__ bool inside(const Place& p, int t, int* err) {
    if (t >= p.end) return false;
    if (t >= p.lo && t < p.hi) return true;
    if (p.c == 0) atomicExch(err, Q8_DEVERR_POSITION);
    return false;
}

// R tokens at a time and thread, tb apart, whose reads go out together, `turns` times; a
// turn's reads go out before the one before is worked on.
template <typename F, int KIND, int R>
__global__ void __launch_bounds__(kThreads) kvq_store_kernel(const KvqIoArgs a, int slots, int tb, int turns, int* err) {
    pdl_wait();
    pdl_launch_dependents();
    const Place p = place<kStored>(a, slots, tb, tb * R * turns);
    Floats<F> next[R] = {}, now[R];
    bool in_next[R], in[R];
    const F* from = static_cast<const F*>(p.v ? a.v : a.k) + p.at;
    const int64_t step = tb * a.ld_tok;
    const auto fetch = [&](int turn) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            in_next[r] = inside(p, p.first + (turn * R + r) * tb, err);
            if (in_next[r]) {
#pragma unroll
                for (int i = 0; i < int(sizeof(F)); ++i) next[r].w[i] = __ldcs(reinterpret_cast<const int4*>(from) + i);
            }
            from += step;
        }
    };
    fetch(0);
    const int words_row = int(a.dim) / 32, codes_row = int(kvq_row(KIND, a.dim));
    uint32_t* const words = static_cast<uint32_t*>(p.v ? a.v_words : a.k_words) + p.entry * words_row + p.c / 2;
    unsigned char* const codes = static_cast<unsigned char*>(p.v ? a.v_codes : a.k_codes) + p.entry * codes_row +
                                 p.c * (KIND == Q8_KVQ_I8 ? kStored : kStored / 2);
#pragma unroll 1
    for (int turn = 0; turn < turns; ++turn) {
#pragma unroll
        for (int r = 0; r < R; ++r) now[r] = next[r], in[r] = in_next[r];
        if (turn + 1 < turns) fetch(turn + 1);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 range = block_range(now[r]);
            if (!in[r]) continue;
            const float lo = range.x, hi = range.y;
            float x[kStored];
            expand(now[r], x);
            const int o = (turn * R + r) * tb;
            uint32_t* const word = words + o * words_row;
            unsigned char* const to = codes + o * codes_row;
            if constexpr (KIND == Q8_KVQ_I8) {
                const float most = fmaxf(-lo, hi);
                // (infinities and NaN: the block reads back as NaN)
                const float d = lo - lo == 0.0f && hi - hi == 0.0f ? __fdiv_rn(most, 127.0f) : __int_as_float(0x7fc00000);
                uint32_t w[4] = {0u, 0u, 0u, 0u};
                if (d > 0.0f) codes_i8<kStored / (sizeof(F) == 4 ? 2 : 4)>(x, d, w);
                *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
                if ((p.c & 1) == 0) *word = __float_as_uint(d);
            } else {
                const __half s = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f)), m = __float2half_rn(lo);
                const float sf = __half2float(s), mf = __half2float(m);
                const bool fine = sf - sf == 0.0f && mf - mf == 0.0f;      // (s is NaN or infinite where lo or hi is)
                *reinterpret_cast<uint2*>(to) = fine ? codes_u4<8>(x, sf, mf, lo, hi) : make_uint2(0u, 0u);
                if ((p.c & 1) == 0)
                    *word = fine ? uint32_t(__half_as_ushort(s)) | uint32_t(__half_as_ushort(m)) << 16 : 0x7e007e00u;
            }
        }
    }
}

template <typename F, int KIND, int R>
__global__ void __launch_bounds__(kThreads) kvq_load_kernel(const KvqIoArgs a, int slots, int tb, int turns, int* err) {
    constexpr int V = kLoaded<F>, BYTES = KIND == Q8_KVQ_I8 ? V : V / 2, W = (BYTES + 3) / 4;   // values, bytes and words of codes
    pdl_wait();
    pdl_launch_dependents();
    const Place p = place<V>(a, slots, tb, tb * R * turns);
    const int words_row = int(a.dim) / 32, codes_row = int(kvq_row(KIND, a.dim));
    const uint32_t* const words = static_cast<const uint32_t*>(p.v ? a.v_words : a.k_words) + p.entry * words_row + p.c / (32 / V);
    const unsigned char* const codes =
        static_cast<const unsigned char*>(p.v ? a.v_codes : a.k_codes) + p.entry * codes_row + p.c * BYTES;
    F* to = static_cast<F*>(p.v ? a.v : a.k) + p.at;
    const int64_t step = tb * a.ld_tok;
    struct Held {
        bool in;
        uint32_t word, w[W];
    } next[R], now[R];
    const auto fetch = [&](int turn) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int o = (turn * R + r) * tb;
            next[r].in = inside(p, p.first + o, err);
            if (!next[r].in) continue;
            next[r].word = words[o * words_row];
            const unsigned char* from = codes + o * codes_row;
            if constexpr (BYTES == 8) {
                const uint2 x = *reinterpret_cast<const uint2*>(from);
                next[r].w[0] = x.x, next[r].w[W - 1] = x.y;
            } else if constexpr (BYTES == 4) {
                next[r].w[0] = *reinterpret_cast<const uint32_t*>(from);
            } else {
                next[r].w[0] = *reinterpret_cast<const uint16_t*>(from);
            }
        }
    };
    fetch(0);
#pragma unroll 1
    for (int turn = 0; turn < turns; ++turn) {
#pragma unroll
        for (int r = 0; r < R; ++r) now[r] = next[r];
        if (turn + 1 < turns) fetch(turn + 1);
#pragma unroll
        for (int r = 0; r < R; ++r, to += step) {
            if (!now[r].in) continue;
            float x[V];
            const float2 sm = KIND == Q8_KVQ_U4 ? kvq_scale_min(now[r].word) : make_float2(__uint_as_float(now[r].word), 0.0f);
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const uint32_t w = now[r].w[k];
                if constexpr (KIND == Q8_KVQ_I8) {
                    const uint32_t u = w ^ 0x80808080u;                           // (plus 128)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[4 * k + i] = (byte_above_2_23(u, i) - 8388736.0f) * sm.x;
                } else {
                    const uint32_t u[2] = {w & 0x0f0f0f0fu, w >> 4 & 0x0f0f0f0fu};
#pragma unroll
                    for (int i = 0; i < (V < 8 ? V : 8); ++i)                     // (the product is exact)
                        x[8 * k + i] = fmaf(byte_above_2_23(u[i & 1], i >> 1) - 8388608.0f, sm.x, sm.y);
                }
            }
            put(to, x);
        }
    }
}

template <typename F, int KIND, bool STORE, int R>
cudaError_t launch_io_kernel(const KvqIoArgs& a, int turns, const LaunchCtx& ctx) {
    const int slots = kThreads / int(a.dim / (STORE ? kStored : kLoaded<F>));
    const int tb = a.T < slots ? int(a.T) : slots, ub = slots / tb;
    const int64_t units = 2 * a.kv_heads, seg = a.T < kSegment ? a.T : kSegment, step = int64_t(tb) * R * turns;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attrs[1];
    cfg.gridDim = dim3(unsigned((units + ub - 1) / ub * ((seg + step - 1) / step)),
                       unsigned((a.T + kSegment - 1) / kSegment), unsigned(a.rows));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = ctx.stream;
    cfg.numAttrs = pdl_attrs(ctx, attrs);
    cfg.attrs = attrs;
    if constexpr (STORE) return cudaLaunchKernelEx(&cfg, kvq_store_kernel<F, KIND, R>, a, slots, tb, turns, ctx.dev_err);
    else return cudaLaunchKernelEx(&cfg, kvq_load_kernel<F, KIND, R>, a, slots, tb, turns, ctx.dev_err);
}

template <typename F, int KIND, bool STORE>
cudaError_t launch_io_tokens(const KvqIoArgs& a, const LaunchCtx& ctx) {
    // Several tokens a thread, and turns of them, as soon as there are threads for it (us, by turns of
    // none, 1 and 4: 1 row of 512 tokens of 8 heads of 128 values, bf16 in 4 bits, stored 2.6, 2.6, 4.5,
    // read back 3.5, 2.2, 3.2; of 2048: 6.0, 5.4, 5.6 and 6.8, 4.7, 3.8; 8 rows of 2048: 38, 32, 24 and
    // 45, 21, 14).  Two turns of a load just below (one, two and four, 4 bits into bf16: 3 rows of 1001 tokens
    // of 5 heads of 96, 2371 threads an SM, 4.6, 3.2, 4.0, that row of 2048, 3449 threads, 4.6, 3.5, 3.8;
    // above, 3 x 1001 into f32, 4742 threads, 4.5, 5.7, 4.3, from 8 bits 4.8, 4.1, 4.1), eight of a store
    // from some more on (4 rows of 8192: 43.6 and 42.3).
    constexpr int V = STORE ? kStored : kLoaded<F>, R = STORE ? 2 : 4;
    const int64_t threads = a.rows * a.T * a.kv_heads * (2 * a.dim / V), sms = ctx.num_sms;
    const int64_t tb = kThreads / (a.dim / V);
    if (STORE && a.T >= 8 * R * tb && threads >= 25600 * sms) return launch_io_kernel<F, KIND, STORE, R>(a, 8, ctx);
    if (a.T >= 4 * R * tb && threads >= (STORE ? 2048 : 4096) * sms) return launch_io_kernel<F, KIND, STORE, R>(a, 4, ctx);
    if (!STORE && a.T >= 2 * R * tb && threads >= 2048 * sms) return launch_io_kernel<F, KIND, STORE, R>(a, 2, ctx);
    if (a.T >= R * tb && threads >= (STORE ? 320 : 640) * sms) return launch_io_kernel<F, KIND, STORE, R>(a, 1, ctx);
    return launch_io_kernel<F, KIND, STORE, 1>(a, 1, ctx);
}

template <bool STORE>
cudaError_t launch_io(const KvqIoArgs& a, const LaunchCtx& ctx) {
    if (a.kind == Q8_KVQ_I8) {
        if (a.type == Q8_KV_F32) return launch_io_tokens<float, Q8_KVQ_I8, STORE>(a, ctx);
        if (a.type == Q8_KV_F16) return launch_io_tokens<__half, Q8_KVQ_I8, STORE>(a, ctx);
        return launch_io_tokens<__nv_bfloat16, Q8_KVQ_I8, STORE>(a, ctx);
    }
    if (a.type == Q8_KV_F32) return launch_io_tokens<float, Q8_KVQ_U4, STORE>(a, ctx);
    if (a.type == Q8_KV_F16) return launch_io_tokens<__half, Q8_KVQ_U4, STORE>(a, ctx);
    return launch_io_tokens<__nv_bfloat16, Q8_KVQ_U4, STORE>(a, ctx);
}

}  // namespace

cudaError_t launch_kvq_store(const KvqIoArgs& a, const LaunchCtx& ctx) { return launch_io<true>(a, ctx); }
cudaError_t launch_kvq_load(const KvqIoArgs& a, const LaunchCtx& ctx) { return launch_io<false>(a, ctx); }

}  // namespace q8
