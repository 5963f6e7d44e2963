// attn_mma.cuh -- the attention kernels over 16-bit caches: the products on the
// matrix instructions (mma.m16n8k16; m16n8k8 for f16's second product).
//
// With the entries of a stage as the n of the first product and the k of the
// second, a block of at most 8 query heads fills half of m = 16.  The other half
// takes what the operand's rounding lost: rows 0-7 hold q (then p) rounded, rows
// 8-15 the rest of it rounded, so one instruction gives both parts' products (f16:
// 22 bits; bf16: 16, and a second instruction adds 8 more).  K and V enter as they
// are.  The accumulator layout of the scores is the operand layout of the weights,
// and all that a lane holds belongs to one query head: no exchange between lanes
// but two shuffles where a reference moves.
//
// Precision.  Over f16 caches q is brought to [2^13, 2^14) by a power of two a
// head.  Weights span more than f16 holds, and where the largest stand on entries
// of no value (as a row's first tokens often are) the output is made of the small
// ones alone; so p enters the second product in two parts of tf32, 11 bits each
// and binary32's exponents, and V converted to it, exactly: m16n8k8, twice as many
// instructions (32 rows of 4096 entries, 8 K/V heads of 64, 128 and 256 values (16
// rows): 59.9, 98.7 and 109 us; with p in two parts of f16, which lost bits below
// 2^-16 of the largest weight, 58.7, 97.4 and 108).  The instruction truncates its
// sums; chains are kept short (every other step of a score; 64 entries of o) and
// joined by rounded binary32 additions: measured 2e-7 where one chain of 512 steps
// is 1e-5 off.  A part times infinity is NaN, so a warp whose state is not finite
// computes its entries again, one by one, by the formula (a call, for which the
// kernels keep a frame of 304 bytes; nothing is spilled).
//
// What bounds it: HBM.  A stage of 16 entries of 128 values is 64 instructions
// (bf16; 48 of f16) of 2 clocks an SM, 8 clocks an entry against 23 for its bytes
// (6.6 TB/s); on the lanes' FMA path eight query heads take 40.  Heads of 256
// values: 16 rows of 4096 entries, 8 K/V heads of 8 query heads, bf16 113 us, f16
// 109 (4.8 and 4.9 TB/s; on the lanes 146 and 151).
#pragma once

#include <cfloat>

#include "attn.cuh"

namespace q8 {

template <int KV>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (KV == Q8_KV_F16)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// m16n8k8: a 10-bit mantissa and binary32's exponents (what f16 holds, exactly).
__device__ __forceinline__ void mma8(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x rounded to that format; x becomes what the rounding lost.
__device__ __forceinline__ uint32_t round_tf32(float& x) {
    uint32_t w;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(w) : "f"(x));
    x -= __uint_as_float(w);
    return w;
}

template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr));
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr));
}

// a and b rounded to the cache's type, as one word (a in the low half); a and b
// become what the rounding lost.
template <int KV>
__device__ __forceinline__ uint32_t round_pair(float& a, float& b) {
    uint32_t w;
    if constexpr (KV == Q8_KV_F16) {
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        a -= f.x, b -= f.y;
    } else {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
        a -= __int_as_float(int(w << 16));
        b -= __int_as_float(int(w & 0xffff0000u));
    }
    return w;
}

template <int KV>
__device__ __forceinline__ float from16(const unsigned char* p) {
    if constexpr (KV == Q8_KV_F16) return __half2float(*reinterpret_cast<const __half*>(p));
    return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
}

// A warp's states entry by entry in binary32, lanes over the values.
template <class T>
__device__ __noinline__ void plain_states(const Segment& s) {
    const AttnArgs& a = s.p.a;
    const int lane = threadIdx.x & 31, D = int(a.dim);
    constexpr int J = T::DMAX / 32, JV = T::DV / 32;
    const int v0 = s.half * T::DV;                      // this warp's values of V
    for (int g = 0; g < s.ng; ++g) {
        float* const scores = s.p.scores && s.half == 0 ? s.p.scores + (int64_t(s.row) * a.heads + s.g0 + g) * s.p.cap : nullptr;
        float top = -INFINITY, l = 0.0f, o[JV] = {};
        for (int it = 0; it < s.its; ++it)
            for (int r = 0; r < T::KT; ++r) {
                const uint32_t v = s.v_begin + uint32_t(it) * T::TK + r;
                if (v >= s.v_end) break;
                const int64_t at = s.off + int64_t(v + (v < s.vis.ns ? 0 : s.vis.gap)) * s.pitch;
                float x = 0.0f;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int d = lane + 32 * j;
                    if (d < D)
                        x = fmaf(s.q[g * T::DMAX + d], from16<T::KV>(static_cast<const unsigned char*>(a.k) + at + 2 * d), x);
                }
#pragma unroll
                for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
                if (scores && lane == 0) scores[v] = x;
                const float n = fmaxf(top, x), f = n == top ? 1.0f : ex2(top - n), w = x == -INFINITY ? 0.0f : ex2(x - n);
                top = n;
                l = l * f + w;
#pragma unroll
                for (int j = 0; j < JV; ++j) {
                    const int d = v0 + lane + 32 * j;
                    if (d < D) o[j] = o[j] * f + w * from16<T::KV>(static_cast<const unsigned char*>(a.v) + at + 2 * d);
                }
            }
        if (lane == 0) {
            s.m[g] = top;
            s.l[g] = l;
        }
#pragma unroll
        for (int j = 0; j < JV; ++j) reinterpret_cast<float*>(s.ring)[g * T::DV + lane + 32 * j] = o[j];
    }
}

template <class T>
__device__ __forceinline__ void mma_states(const Segment& s) {
    constexpr int KV = T::KV, KS = T::KS, VS = T::VS, SUB = T::SUB;
    constexpr bool BF = KV == Q8_KV_BF16;
    const AttnParams& p = s.p;
    const AttnArgs& a = p.a;
    const int lane = threadIdx.x & 31, D = int(a.dim), its = s.its;
    const int g = lane >> 2, c2 = (lane & 3) * 2;       // this lane's query head, and its entries (or values) of 8
    const uint32_t ring_s = smem_u32(s.ring);
    // a lane copies the same 16-byte column of a row in RPI (VRPI); the row's swap of
    // chunks is its own (r0) and that of the row it begins at
    const int r0 = lane / T::CPR, c0 = lane % T::CPR, rv = lane / T::VCPR, cv = lane % T::VCPR;
    const bool copies = r0 < T::RPI && c0 * 8 < D, v_copies = rv < T::VRPI && s.half * T::DV + cv * 8 < D;
    const unsigned char* kp = static_cast<const unsigned char*>(a.k) + s.off + c0 * 16;
    const unsigned char* vp = static_cast<const unsigned char*>(a.v) + s.off + s.half * (2 * T::DV) + cv * 16;
    const uint32_t to = r0 * T::PITCH + T::swap(c0, r0) * 16, step = T::RPI * s.pitch;
    const uint32_t v_to = T::HALF + rv * T::VPITCH + T::swap(cv, rv) * 16, v_step = T::VRPI * s.pitch;

    int in_slot = 0, out_slot = 0;
    const auto load = [&](int it) {
        // (where K and V are alike, so are their lanes' columns: one pass for both)
        constexpr bool ALIKE = T::SPLIT == 1;
        if (it < its && (copies || (!ALIKE && v_copies))) {
            const uint32_t slot = ring_s + in_slot * T::STAGE, st = slot + to, sv = slot + v_to;
            const uint32_t vt = s.v_begin + uint32_t(it) * T::TK, vb = vt + r0, vbv = vt + rv;
            if (vt + T::KT <= s.v_end && (vt >= s.vis.ns || vt + T::KT <= s.vis.ns)) {
                // all of them, with none left out between
                const uint32_t gap = vt < s.vis.ns ? 0 : s.vis.gap;
                const uint64_t at = uint64_t(vb + gap) * s.pitch;
                const unsigned char *ka = kp + at, *va = vp + (ALIKE ? at : uint64_t(vbv + gap) * s.pitch);
                if (ALIKE || copies) {
#pragma unroll
                    for (int r = 0; r < T::KT; r += T::RPI, ka += step) {
                        const uint32_t dst = (st ^ T::turn(r)) + r * T::PITCH;
                        cp16(dst, ka, true);
                        if constexpr (ALIKE) {
                            cp16(dst + T::HALF, va, true);
                            va += step;
                        }
                    }
                }
                if (!ALIKE && v_copies) {
#pragma unroll
                    for (int r = 0; r < T::KT; r += T::VRPI, va += v_step)
                        cp16((sv ^ T::turn(r)) + r * T::VPITCH, va, true);
                }
            } else {
                const auto from = [&](uint32_t v, bool in) {
                    return in ? uint64_t(v + (v < s.vis.ns ? 0 : s.vis.gap)) * s.pitch : 0;
                };
                if (ALIKE || copies) {
#pragma unroll
                    for (int r = 0; r < T::KT; r += T::RPI) {
                        const uint32_t v = vb + r, dst = (st ^ T::turn(r)) + r * T::PITCH;
                        const bool in = v < s.v_end;
                        const uint64_t at = from(v, in);
                        cp16(dst, kp + at, in);
                        if constexpr (ALIKE) cp16(dst + T::HALF, vp + at, in);
                    }
                }
                if (!ALIKE && v_copies) {
#pragma unroll
                    for (int r = 0; r < T::KT; r += T::VRPI) {
                        const uint32_t v = vbv + r;
                        const bool in = v < s.v_end;
                        cp16((sv ^ T::turn(r)) + r * T::VPITCH, vp + from(v, in), in);
                    }
                }
            }
        }
        in_slot = in_slot + 1 == T::S ? 0 : in_slot + 1;
        cp_commit();
    };
#pragma unroll 1
    for (int i = 0; i < T::S - 1; ++i) load(i);

    stage_q<T>(s);
    float scale = 1.0f, back = 1.0f;
    const float* q = s.q + g * T::DMAX + c2;
    if constexpr (!BF) {
        float most = 0.0f;
#pragma unroll
        for (int k = 0; k < 2 * KS; ++k) most = fmaxf(most, fmaxf(fabsf(q[8 * k]), fabsf(q[8 * k + 1])));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        // powers of two: 2^(13 - the largest's exponent), and its inverse
        const int e = min(max(267 - (__float_as_int(most) >> 23), 1), 253);
        scale = __int_as_float(e << 23);
        back = __int_as_float((254 - e) << 23);
    }
    // (the second part is 2^-11 of the first at most: brought up by that, so that f16's
    // subnormals cost values down to 2^-28 of the largest none of their 22 bits)
    constexpr float LOW_SCALE = BF ? 1.0f : 2048.0f;
    // (the third part of 256 values lies in shared memory, each lane's its own)
    constexpr bool LOW = BF && T::SPLIT > 1;
    __shared__ uint2 s_low[LOW ? KS * 32 : 1];
    uint32_t qa[KS][4], ql[BF && !LOW ? KS : 1][2];
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x = q[16 * k + 8 * h] * scale, y = q[16 * k + 8 * h + 1] * scale;
            qa[k][2 * h] = round_pair<KV>(x, y);
            x *= LOW_SCALE, y *= LOW_SCALE;
            qa[k][2 * h + 1] = round_pair<KV>(x, y);
            if constexpr (LOW) {
                const uint32_t low = round_pair<KV>(x, y);
                if (threadIdx.x < 32) (h ? s_low[32 * k + lane].y : s_low[32 * k + lane].x) = low;
            } else if constexpr (BF) {
                ql[k][h] = round_pair<KV>(x, y);
            }
        }
    if constexpr (LOW) __syncthreads();
    float o[2 * VS][4] = {}, sum[2 * VS][2] = {};       // chains of o; their sums
    float ref = -INFINITY, l = 0.0f;
    float* const scores =
        p.scores && g < s.ng && s.half == 0 ? p.scores + (int64_t(s.row) * a.heads + s.g0 + g) * p.cap : nullptr;
    // where this lane's rows of the matrix loads begin: of K four of entries 0-7 and
    // 8-15 by values 0-7 and 8-15, of V transposed
    const int kr = (lane >> 4) * 8 + (lane & 7), vr = (lane >> 3 & 1) * 8 + (lane & 7);
    const uint32_t k_at = kr * T::PITCH + T::swap(lane >> 3 & 1, kr) * 16;
    const uint32_t v_at = T::HALF + vr * T::VPITCH + T::swap(lane >> 4, vr) * 16;
    const auto flush = [&] {
#pragma unroll
        for (int t = 0; t < 2 * VS; ++t) {
            sum[t][0] += o[t][0] + o[t][2];
            sum[t][1] += o[t][1] + o[t][3];
            o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.0f;
        }
    };

    for (int it = 0; it < its; ++it) {
        cp_wait<T::S - 2>();
        __syncwarp();
        load(it + T::S - 1);
        const uint32_t st = ring_s + out_slot * T::STAGE;
        out_slot = out_slot + 1 == T::S ? 0 : out_slot + 1;
        const uint32_t vb = s.v_begin + uint32_t(it) * T::TK;
        float x[SUB][4];                                // entries c2, c2 + 1, 8 + c2, 9 + c2 of each 16
        bool moves = false;
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            // scores of 16 entries, two chains each
            float c[2][2][4] = {};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t kb[4];
                ldmatrix4<false>(kb, T::column(st + k_at, 2 * k) + u * 16 * T::PITCH);
                mma16<KV>(c[0][k & 1], qa[k], kb[0], kb[1]);
                mma16<KV>(c[1][k & 1], qa[k], kb[2], kb[3]);
                if constexpr (BF) {
                    const uint2 lw = LOW ? s_low[32 * k + lane] : make_uint2(ql[LOW ? 0 : k][0], ql[LOW ? 0 : k][1]);
                    const uint32_t low[4] = {lw.x, 0u, lw.y, 0u};
                    mma16<KV>(c[0][k & 1], low, kb[0], kb[1]);
                    mma16<KV>(c[1][k & 1], low, kb[2], kb[3]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float(&d)[2][4] = c[j >> 1];
                float y = fmaf(d[0][2 + (j & 1)] + d[1][2 + (j & 1)], 1.0f / LOW_SCALE, d[0][j & 1] + d[1][j & 1]);
                if constexpr (!BF) y *= back;
                const uint32_t v = vb + 16 * u + (j >> 1) * 8 + c2 + (j & 1);
                if (scores && v < s.v_end) scores[v] = y;
                x[u][j] = v < s.v_end ? y : -INFINITY;
                moves = moves || x[u][j] > ref + 8.0f;
            }
        }
        if (__any_sync(0xffffffffu, moves)) {
            float top = ref;
#pragma unroll
            for (int u = 0; u < SUB; ++u) top = fmaxf(top, fmaxf(fmaxf(x[u][0], x[u][1]), fmaxf(x[u][2], x[u][3])));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float f = top == ref ? 1.0f : ex2(ref - top);
            ref = top;
            l *= f;
#pragma unroll
            for (int t = 0; t < 2 * VS; ++t) {
                sum[t][0] *= f, sum[t][1] *= f;
                o[t][0] *= f, o[t][1] *= f, o[t][2] *= f, o[t][3] *= f;
            }
        }
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[u][j] = x[u][j] == -INFINITY ? 0.0f : ex2(x[u][j] - ref);
                l += x[u][j];
            }
            uint32_t pa[4], pl[4] = {};      // f16: of entries 0-7 and 8-15
            if constexpr (BF) {
                pa[0] = round_pair<KV>(x[u][0], x[u][1]);
                pa[1] = round_pair<KV>(x[u][0], x[u][1]);
                pa[2] = round_pair<KV>(x[u][2], x[u][3]);
                pa[3] = round_pair<KV>(x[u][2], x[u][3]);
                pl[0] = round_pair<KV>(x[u][0], x[u][1]);
                pl[2] = round_pair<KV>(x[u][2], x[u][3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    pa[j] = round_tf32(x[u][j >> 1]);
                    pl[j] = round_tf32(x[u][2 + (j >> 1)]);
                }
            }
#pragma unroll
            for (int t = 0; t < VS; ++t) {
                uint32_t v[4];
                ldmatrix4<true>(v, T::column(st + v_at, 2 * t) + u * 16 * T::VPITCH);
                if constexpr (BF) {
                    mma16<KV>(o[2 * t], pa, v[0], v[1]);
                    mma16<KV>(o[2 * t + 1], pa, v[2], v[3]);
                    mma16<KV>(o[2 * t], pl, v[0], v[1]);
                    mma16<KV>(o[2 * t + 1], pl, v[2], v[3]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {        // (a lane's two entries as k and k + 4)
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[j]));
                        mma8(o[2 * t + (j >> 1)], j & 1 ? pl : pa, __float_as_uint(f.x), __float_as_uint(f.y));
                    }
                }
            }
        }
        if (it % (4 / SUB) == 4 / SUB - 1) flush();
    }
    flush();
    cp_wait<0>();
    __syncwarp();

    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    float zero = l * 0.0f;
#pragma unroll
    for (int t = 0; t < 2 * VS; ++t) zero += sum[t][0] * 0.0f + sum[t][1] * 0.0f;
    if (__any_sync(0xffffffffu, !(zero == 0.0f))) {      // something infinite or NaN among what was seen
        plain_states<T>(s);
        return;
    }
    if ((lane & 3) == 0) {
        s.m[g] = ref;
        s.l[g] = l;
    }
    float* so = reinterpret_cast<float*>(s.ring) + g * T::DV + c2;
#pragma unroll
    for (int t = 0; t < 2 * VS; ++t) *reinterpret_cast<float2*>(so + 8 * t) = make_float2(sum[t][0], sum[t][1]);
}

// KS: steps of 16 values a head.  SPLIT 2: two warps take the same entries, all of
// K and half of V's values each (the states of 256 values would not fit a warp's
// registers); K comes from L2 the second time.
template <int KV_, int KS_, int SPLIT_ = 1>
struct AttnMma {
    static constexpr int KV = KV_, KS = KS_, SPLIT = SPLIT_, VS = KS / SPLIT, NG = 8;
    static constexpr int ELT = 2, DMAX = 16 * KS, DV = 16 * VS;
    static constexpr int PITCH = 2 * DMAX, CPR = 2 * KS, VPITCH = 2 * DV, VCPR = 2 * VS;
    static constexpr int SUB = KS == 4 ? 2 : 1;               // products of 16 entries a stage
    static constexpr int KT = 16 * SUB, HALF = KT * PITCH, STAGE = HALF + KT * VPITCH;
    static constexpr int S0 = kAttnRing / STAGE;
    static constexpr int S = S0 > 6 ? 6 : S0;
    static constexpr int TK = kAttnWarps / SPLIT * KT;
    static constexpr int EXTRA = (128 * 1024 + TK * 2 * PITCH - 1) / (TK * 2 * PITCH);
    static constexpr int LEAST = 1;
    static constexpr int CTAS = 2, RING = kAttnRing, MAX_CTAS = kAttnMaxCtas;
    static constexpr bool HEAD_MAJOR = false;
    static_assert(S >= 2 && NG * DMAX * 4 <= kAttnRing && DV % 32 == 0, "attention tile");

    static constexpr int RPI = CPR == 8 ? 4 : CPR == 32 ? 1 : 2;       // rows a warp copies at a time
    static constexpr int VRPI = VCPR == 8 ? 4 : 2;

    // Chunk c of entry r lies at swap(c, r), so that the eight rows of a matrix load
    // are on banks of their own (rows of 12 chunks begin on every other half).
    static __device__ __forceinline__ int swap(int c, int r) { return CPR % 8 ? c ^ (r >> 1 & 3) : c ^ (r & 7); }
    // What row r (a multiple of RPI) adds to the swap of a place in row r0 < RPI; a
    // stage begins on a multiple of 128 bytes, and of a row where that is 256.
    static constexpr uint32_t turn(int r) { return uint32_t(CPR % 8 ? r >> 1 & 3 : r & 7) * 16; }
    // The place of chunk c more (even) than that at `at`.
    static __device__ __forceinline__ uint32_t column(uint32_t at, int c) {
        return CPR % 8 ? (at ^ uint32_t(c & 2) * 16) + uint32_t(c & ~3) * 16 : at ^ uint32_t(c) * 16;
    }
    static __device__ __forceinline__ void states(const Segment& s) { mma_states<AttnMma>(s); }
};

template <int KV>
cudaError_t launch_attn_16(const AttnParams& p, const LaunchCtx& ctx) {
    if (p.gsz <= kAttnLanesHeads) return launch_attn_type<KV>(p, ctx);
    if (p.a.dim <= 64) return launch_attn_kernel<AttnMma<KV, 4>>(p, ctx);
    if (p.a.dim <= 96) return launch_attn_kernel<AttnMma<KV, 6>>(p, ctx);
    if (p.a.dim <= 128) return launch_attn_kernel<AttnMma<KV, 8>>(p, ctx);
    return launch_attn_kernel<AttnMma<KV, 16, 2>>(p, ctx);
}

}  // namespace q8
