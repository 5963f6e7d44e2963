// attn_kvq.cuh -- the attention kernels over quantised caches (kvq.cuh), on the matrix
// instructions (mma.m16n8k16).
//
// Mathematics.  With codes u of blocks b, a score is sum_b s_b sum_d q_d u_d + m_b sum_d q_d,
// so codes enter the first product as they are, a block's sum takes its scale in binary32
// and the sums of q a block are made once.  The output is sum_i p_i s_ib u_id + p_i m_ib: the
// weights take the block's scale, p_i s_ib, and codes enter the second product as they are.
// Nothing is dequantised.  Softmax, split and join are attn.cuh's.
//
// Codes as operands.  Below the smallest normal (and up to twice that) a 16-bit float is an
// integer times the smallest subnormal: four bits are exact f16 or bf16 after a shift that two
// or four of them share and an AND, with no conversion and no offset, and the instruction
// takes subnormals.  It aligns their products as if they were normal, so what lies low loses
// bits: of K, in f16, bits 3 to 6 and 7 to 10 (units of 2^-21 and 2^-17; from bits 0 and 4 on,
// weights were 8e-7 off, not 2e-7), of V, in bf16, bits 0 to 3 and 4 to 7 (2^-133 and 2^-129).
// A signed byte takes an exclusive or (code + 128, subnormal) and one multiply-add, exact,
// that makes it normal and takes the 128 away.
//
// Precision.  q enters as two parts of f16, the second brought up by 2^11, of values brought
// to [2^13, 2^14) by a power of two a head: 22 bits of values down to 2^-28 (Q8_KVQ_U4: 2^-24)
// of the largest.  p s enters as its three bf16 parts, exactly (Q8_KVQ_U4: times 2^103, which
// codes' units take away).  The instruction truncates its sums: chains are a block of a score
// and one stage of the output, joined by rounded binary32 additions, and four-bit codes,
// which have no sign, enter the output's with both signs (see `turned`).
//
// What bounds it.  Four bits: instructions.  16 entries of 128 values are 360 of them a warp
// (four query heads: 24 products, 90 to unpack codes, 100 to scale and part the weights, 40 to
// scale the scores), a product holds a scheduler's issue for some 5 clocks beside its 8 of the
// tensor pipe, and together they take some 600 clocks where the bytes at HBM's rate take 430:
// 0.58 issued a clock with two to four warps a scheduler alike.  Eight bits: HBM, with eight
// query heads the instructions again.  Beside its bytes, a call that fills the GPU has some us
// that do not grow with the entries (a line through 16 rows of 2048 to 49152: 4 bits 13 us with
// four query heads, 17 with eight, 8 bits 10 and 15): the launch, positions, q as operands, the
// first stages, the join of parts.  tcgen05 would take the products out of the way, but not
// what is around them.  V's scales, one a block of values and not of entries, make the second
// product's other operand another one for every 32 values: its smallest tile (64 or 128
// values) would read all of V's 16-bit operand from shared memory for every block of it, 128
// KB for 128 entries of 128 values, more clocks than their bytes take.  The first product,
// whose scales are factors of its results, was not tried there: it wants K's codes unpacked in
// shared memory, 8 stores of 16 bytes a lane for 16 entries of 128 values, as many as its
// matrix instructions are now with four heads.
//
// Measured (16 rows of 16384 entries, 8 K/V heads of 128 values; device time): 4 bits, four query
// heads 77 us, 4.4 TB/s (5.6 TB/s between 16384 and 32768 entries), eight 108 us; 8 bits 107 us,
// 5.7 TB/s (6.5), and 123 us; 64 rows of 4100 to 8192 4-bit entries 110 us; one row of 130001
// with the weights accumulated 52 us; one row of 613 9.6 us, of one entry 5.0 us.
//
// Layout.  Entries are the m of the first product, and its n = 8 columns the parts of q: four
// query heads' first and second parts side by side, or eight heads' first parts and a second
// product of their second ones.  So a lane ends with entries g and g + 8 of 16 for one head
// (or two), g = lane / 4, without an exchange.  The weights' parts go through movmatrix (8 x 8
// transposed across the warp), entries becoming the k of the second product, whose m are
// values and whose n are heads (four: first and second part side by side again).
#pragma once

#include "attn_mma.cuh"
#include "kvq.cuh"

namespace q8 {

// 8 x 8 16-bit values across the warp, transposed.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// The upper halves of a (low) and b.
__device__ __forceinline__ uint32_t upper_halves(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float upper(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }

// Bytes 0 and 2 of w, signed, times 2^-10 (f16) or 2^-6 (bf16): as subnormals, plus 128,
// then normal less 128 of these units.
template <int KV>
__device__ __forceinline__ uint32_t signed_bytes(uint32_t w) {
    const uint32_t u = (w & 0x00ff00ffu) ^ 0x00800080u;
    uint32_t r;
    if constexpr (KV == Q8_KV_F16)      // 2^14 u - 2^-3
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(u), "r"(0x74007400u), "r"(0xb000b000u));
    else                                // 2^127 u - 2
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(u), "r"(0x7f007f00u), "r"(0xc000c000u));
    return r;
}

// Some bytes from global to shared memory, or as many zeros.
template <int BYTES>
__device__ __forceinline__ void cp_some(uint32_t dst, const void* src, bool read) {
    if constexpr (BYTES == 16) {
        cp16(dst, src, read);
    } else {
        const int n = read ? BYTES : 0;
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
    }
}

template <class T>
__device__ __forceinline__ void kvq_states(const Segment& s) {
    constexpr int NB = T::NB, NH = T::NH, SUB = T::SUB, CH = T::CH, KIND = T::KIND;
    constexpr bool U4 = KIND == Q8_KVQ_U4;
    const AttnParams& p = s.p;
    const AttnArgs& a = p.a;
    const int lane = threadIdx.x & 31, its = s.its;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring_s = smem_u32(s.ring);

    // a lane copies the same 16-byte column of a row in RPI; words are one run
    constexpr int RPI = 32 / CH;
    const int r0 = lane / CH, c0 = lane % CH;
    const bool copies = r0 < RPI;
    const unsigned char* const kp = static_cast<const unsigned char*>(a.k) + s.off * T::ROW + c0 * 16;
    const unsigned char* const vp = static_cast<const unsigned char*>(a.v) + s.off * T::ROW + c0 * 16;
    const unsigned char* const kw = reinterpret_cast<const unsigned char*>(a.k_words) + s.off * T::WB;
    const unsigned char* const vw = reinterpret_cast<const unsigned char*>(a.v_words) + s.off * T::WB;
    const uint32_t to = r0 * T::PITCH + c0 * 16;

    int in_slot = 0, out_slot = 0;
    const auto load = [&](int it) {
        if (it < its) {
            const uint32_t st = ring_s + in_slot * T::STAGE, vt = s.v_begin + uint32_t(it) * T::TK;
            constexpr int W = T::KT * T::WN;             // pieces of words
            if (vt + T::KT <= s.v_end && (vt >= s.vis.ns || vt + T::KT <= s.vis.ns)) {
                // all of them, with none left out between
                const int64_t at = vt + (vt < s.vis.ns ? 0 : s.vis.gap);
                const unsigned char *ka = kp + (at + r0) * T::ROW, *va = vp + (at + r0) * T::ROW;
#pragma unroll
                for (int r = 0; r < T::KT; r += RPI)
                    if (copies && (T::KT % RPI == 0 || r0 + r < T::KT)) {
                        cp16(st + to + r * T::PITCH, ka + r * T::ROW, true);
                        cp16(st + T::CODES + to + r * T::PITCH, va + r * T::ROW, true);
                    }
                const unsigned char *ks = kw + at * T::WB, *vs = vw + at * T::WB;
#pragma unroll
                for (int j = 0; j < W; j += 32)
                    if (W % 32 == 0 || j + lane < W) {
                        const int x = (j + lane) * T::WC;
                        cp_some<T::WC>(st + 2 * T::CODES + x, ks + x, true);
                        cp_some<T::WC>(st + 2 * T::CODES + T::WORDS + x, vs + x, true);
                    }
            } else {
#pragma unroll
                for (int r = 0; r < T::KT; r += RPI)
                    if (copies && (T::KT % RPI == 0 || r0 + r < T::KT)) {
                        const uint32_t v = vt + r0 + r;
                        const bool in = v < s.v_end;
                        const int64_t at = in ? int64_t(v + (v < s.vis.ns ? 0 : s.vis.gap)) * T::ROW : 0;
                        cp16(st + to + r * T::PITCH, kp + at, in);
                        cp16(st + T::CODES + to + r * T::PITCH, vp + at, in);
                    }
#pragma unroll
                for (int j = 0; j < W; j += 32)
                    if (W % 32 == 0 || j + lane < W) {
                        const int e = (j + lane) / T::WN, c = (j + lane - e * T::WN) * T::WC;
                        const uint32_t v = vt + e;
                        const bool in = v < s.v_end;
                        const int64_t at = in ? int64_t(v + (v < s.vis.ns ? 0 : s.vis.gap)) * T::WB + c : 0;
                        const int x = (j + lane) * T::WC;
                        cp_some<T::WC>(st + 2 * T::CODES + x, kw + at, in);
                        cp_some<T::WC>(st + 2 * T::CODES + T::WORDS + x, vw + at, in);
                    }
            }
        }
        in_slot = in_slot + 1 == T::S ? 0 : in_slot + 1;
        cp_commit();
    };
#pragma unroll 1
    for (int i = 0; i < T::S - 1; ++i) load(i);

    stage_q<T>(s);
    // q as B: lane (g, t) has column g, of it four values a step.  Four heads: column g is
    // part g % 2 of head g / 2; eight: head g, its parts in products of their own.
    const float* q = s.q + (NH == 1 ? g >> 1 : g) * T::DMAX;
    // the eight of a block that this lane holds, by step and register
    const auto value_at = [&](int k, int r, int half) {
        return U4 ? 8 * t + 2 * k + r + 4 * half : 16 * k + 4 * t + r + 2 * half;
    };
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 8 * NB; ++i) most = fmaxf(most, fabsf(q[32 * (i / 8) + 8 * t + i % 8]));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
    // powers of two: 2^(13 - the largest's exponent), and its inverse
    const int ex = min(max(267 - (__float_as_int(most) >> 23), 1), 253);
    const float scale = __int_as_float(ex << 23);
    uint32_t qb[NB][2][NH][2];
    float qsum[U4 ? NB : 1][NH], back[NH];           // of this lane's heads (see `head`)
    const auto head = [&](int hh) { return NH == 1 ? t : 2 * t + hh; };
    // Codes of four bits have no sign: half of a stage's entries enter the second product as
    // -p s (15 - u) + p (m + 15 s), or the truncated sums of all would lean one way
    const auto turned = [](int e) { return U4 && e == 1; };
    const auto owner = [&](int hh) { return NH == 1 ? 8 * t : 4 * (2 * t + hh); };   // a lane that holds its q
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = q[32 * b + value_at(k, r, 0)] * scale, y = q[32 * b + value_at(k, r, 1)] * scale;
                sum += x + y;
                if (U4 && r == 1) x *= 1.0f / 16.0f, y *= 1.0f / 16.0f;      // (its codes are 16 units)
                const uint32_t hi = round_pair<Q8_KV_F16>(x, y);
                x *= 2048.0f, y *= 2048.0f;
                const uint32_t lo = round_pair<Q8_KV_F16>(x, y);
                if constexpr (NH == 1) {
                    qb[b][k][0][r] = g & 1 ? lo : hi;
                } else {
                    qb[b][k][0][r] = hi;
                    qb[b][k][1][r] = lo;
                }
            }
        if constexpr (U4) {
            sum *= 0x1p-21f;
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
            for (int hh = 0; hh < NH; ++hh) qsum[b][hh] = __shfl_sync(0xffffffffu, sum, owner(hh));
        }
    }
    {
        const float inverse = __int_as_float((254 - ex) << 23);
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) back[hh] = __shfl_sync(0xffffffffu, inverse, owner(hh));
    }

    float o[2 * NB][2 * NH] = {};                    // 16 values each: rows g and g + 8, by head
    float mb[U4 ? NB : 1][NH] = {};                  // sums of p m over this lane's entries
    float ref[NH], l[NH];
#pragma unroll
    for (int hh = 0; hh < NH; ++hh) ref[hh] = -INFINITY, l[hh] = 0.0f;
    float* scores[NH];
#pragma unroll
    for (int hh = 0; hh < NH; ++hh)
        scores[hh] = p.scores && head(hh) < s.ng ? p.scores + (int64_t(s.row) * a.heads + s.g0 + head(hh)) * p.cap : nullptr;
    // where this lane's rows of the matrix loads begin: entries 0-7, 8-15 of a 16-byte
    // column, then of the next
    const uint32_t m_at = ((lane >> 3 & 1) * 8 + (lane & 7)) * T::PITCH + (lane >> 4) * 16;

    for (int it = 0; it < its; ++it) {
        cp_wait<T::S - 2>();
        __syncwarp();
        load(it + T::S - 1);
        const unsigned char* stage = s.ring + out_slot * T::STAGE;
        const uint32_t st = ring_s + out_slot * T::STAGE;
        out_slot = out_slot + 1 == T::S ? 0 : out_slot + 1;
        const uint32_t vb = s.v_begin + uint32_t(it) * T::TK;
        const auto words = [&](int plane, int entry, uint32_t (&w)[NB]) {
            const unsigned char* at = stage + 2 * T::CODES + plane * T::WORDS + entry * T::WB;
            if constexpr (T::WC == 16) {
#pragma unroll
                for (int i = 0; i < NB; i += 4) {
                    const uint4 x = *reinterpret_cast<const uint4*>(at + 4 * i);
                    w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
                }
            } else if constexpr (T::WC == 8) {
#pragma unroll
                for (int i = 0; i < NB; i += 2) {
                    const uint2 x = *reinterpret_cast<const uint2*>(at + 4 * i);
                    w[i] = x.x, w[i + 1] = x.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < NB; ++i) w[i] = *reinterpret_cast<const uint32_t*>(at + 4 * i);
            }
        };
        float x[SUB][NH][2];                         // entries g and g + 8 of each 16
        bool moves = false;
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            uint32_t w[2][NB];
            words(0, 16 * u + g, w[0]);
            words(0, 16 * u + g + 8, w[1]);
            float sc[NH][2] = {};
            const auto block = [&](int b, const float (&c)[NH][4]) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 sm = U4 ? kvq_scale_min(w[e][b]) : make_float2(__uint_as_float(w[e][b]), 0.0f);
#pragma unroll
                    for (int hh = 0; hh < NH; ++hh) {
                        const float hi = NH == 1 ? c[0][2 * e] : c[0][2 * e + hh];
                        const float lo = NH == 1 ? c[0][2 * e + 1] : c[NH - 1][2 * e + hh];
                        sc[hh][e] = fmaf(fmaf(lo, 1.0f / 2048.0f, hi), sm.x, sc[hh][e]);
                        if constexpr (U4) sc[hh][e] = fmaf(qsum[b][hh], sm.y, sc[hh][e]);
                    }
                }
            };
#pragma unroll
            for (int c = 0; c < CH; c += 2) {
                uint32_t r[4];
                ldmatrix4<false>(r, st + m_at + u * 16 * T::PITCH + (c + 1 < CH ? c * 16 : c * 16 - (lane >> 4) * 16));
                if constexpr (U4) {
#pragma unroll
                    for (int b = c; b < c + 2 && b < CH; ++b) {
                        float d[NH][4] = {};
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t w0 = k ? r[2 * (b - c)] >> 5 : r[2 * (b - c)] << 3;
                            const uint32_t w1 = k ? r[2 * (b - c) + 1] >> 5 : r[2 * (b - c) + 1] << 3;
                            const uint32_t f[4] = {w0 & 0x00780078u, w1 & 0x00780078u, w0 & 0x07800780u, w1 & 0x07800780u};
#pragma unroll
                            for (int n = 0; n < NH; ++n) mma16<Q8_KV_F16>(d[n], f, qb[b][k][n][0], qb[b][k][n][1]);
                        }
                        block(b, d);
                    }
                } else {
                    float d[NH][4] = {};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t w0 = r[2 * k], w1 = r[2 * k + 1];
                        const uint32_t f[4] = {signed_bytes<Q8_KV_F16>(w0), signed_bytes<Q8_KV_F16>(w1),
                                               signed_bytes<Q8_KV_F16>(w0 >> 8), signed_bytes<Q8_KV_F16>(w1 >> 8)};
#pragma unroll
                        for (int n = 0; n < NH; ++n) mma16<Q8_KV_F16>(d[n], f, qb[c / 2][k][n][0], qb[c / 2][k][n][1]);
                    }
                    block(c / 2, d);
                }
            }
#pragma unroll
            for (int hh = 0; hh < NH; ++hh)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float y = sc[hh][e] * (U4 ? 0x1p21f : 0x1p10f) * back[hh];
                    const uint32_t v = vb + 16 * u + 8 * e + g;
                    if (scores[hh] && v < s.v_end) scores[hh][v] = y;
                    x[u][hh][e] = v < s.v_end ? y : -INFINITY;
                    moves = moves || x[u][hh][e] > ref[hh] + 8.0f;
                }
        }
        if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
            for (int hh = 0; hh < NH; ++hh) {
                float top = ref[hh];
#pragma unroll
                for (int u = 0; u < SUB; ++u) top = fmaxf(top, fmaxf(x[u][hh][0], x[u][hh][1]));
#pragma unroll
                for (int mask = 4; mask < 32; mask *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, mask));
                const float f = top == ref[hh] ? 1.0f : ex2(ref[hh] - top);
                ref[hh] = top;
                l[hh] *= f;
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) o[i][hh] *= f, o[i][NH + hh] *= f;
                if constexpr (U4) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) mb[b][hh] *= f;
                }
            }
        }
        uint32_t w[SUB][2][NB];
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            words(1, 16 * u + g, w[u][0]);
            words(1, 16 * u + g + 8, w[u][1]);
        }
        float px[SUB][NH][2];
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int hh = 0; hh < NH; ++hh)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float y = x[u][hh][e] == -INFINITY ? 0.0f : ex2(x[u][hh][e] - ref[hh]);
                    l[hh] += y;
                    x[u][hh][e] = y;
                    px[u][hh][e] = U4 ? y * 0x1p103f : y;
                }
#pragma unroll
        for (int c = 0; c < CH; c += 2) {
            uint32_t r[SUB][4];
#pragma unroll
            for (int u = 0; u < SUB; ++u)
                ldmatrix4<true>(r[u], st + T::CODES + m_at + u * 16 * T::PITCH +
                                          (c + 1 < CH ? c * 16 : c * 16 - (lane >> 4) * 16));
#pragma unroll
            for (int b = U4 ? c : c / 2; b < (U4 ? c + 2 : c / 2 + 1) && b < NB; ++b) {
                // the weights' parts as B: columns as q's
                constexpr int PARTS = NH == 1 ? 2 : 3;
                uint32_t pb[SUB][PARTS][2];
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 sm = U4 ? kvq_scale_min(w[u][e][b]) : make_float2(__uint_as_float(w[u][e][b]), 0.0f);
                        float y[NH], mid[NH], lo[NH];
#pragma unroll
                        for (int hh = 0; hh < NH; ++hh) {
                            y[hh] = px[u][hh][e] * (turned(e) ? -sm.x : sm.x);
                            if constexpr (U4)
                                mb[b][hh] = fmaf(x[u][hh][e], turned(e) ? fmaf(15.0f, sm.x, sm.y) : sm.y, mb[b][hh]);
                            mid[hh] = y[hh] - upper(y[hh]);
                            lo[hh] = mid[hh] - upper(mid[hh]);
                        }
                        if constexpr (NH == 1) {
                            pb[u][0][e] = movmatrix(upper_halves(y[0], mid[0]));
                            pb[u][1][e] = movmatrix(__float_as_uint(lo[0]) >> 16);
                        } else {
                            pb[u][0][e] = movmatrix(upper_halves(y[0], y[NH - 1]));
                            pb[u][1][e] = movmatrix(upper_halves(mid[0], mid[NH - 1]));
                            pb[u][PARTS - 1][e] = movmatrix(upper_halves(lo[0], lo[NH - 1]));
                        }
                    }
#pragma unroll
                for (int k = 0; k < 2; ++k) {        // 16 values of the block
                    float d[4] = {};
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        uint32_t f[4];
                        if constexpr (U4) {                      // (entries 8-15: 15 less the code)
                            const uint32_t w0 = r[u][2 * (b - c)] >> (8 * k), w1 = r[u][2 * (b - c) + 1] >> (8 * k);
                            f[0] = w0 & 0x000f000fu, f[1] = w0 & 0x00f000f0u, f[2] = ~w1 & 0x000f000fu, f[3] = ~w1 & 0x00f000f0u;
                        } else {
                            const uint32_t w0 = r[u][2 * k], w1 = r[u][2 * k + 1];
                            f[0] = signed_bytes<Q8_KV_BF16>(w0), f[1] = signed_bytes<Q8_KV_BF16>(w0 >> 8);
                            f[2] = signed_bytes<Q8_KV_BF16>(w1), f[3] = signed_bytes<Q8_KV_BF16>(w1 >> 8);
                        }
#pragma unroll
                        for (int i = PARTS; i-- > 0;) mma16<Q8_KV_BF16>(d, f, pb[u][i][0], pb[u][i][1]);
                    }
                    float(&sum)[2 * NH] = o[2 * b + k];
                    if constexpr (NH == 1) {
                        sum[0] += d[0] + d[1];
                        sum[1] += d[2] + d[3];
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum[i] += d[i];
                    }
                }
            }
        }
    }
    cp_wait<0>();
    __syncwarp();

    constexpr float UNIT = U4 ? 0x1p30f : 0x1p6f;    // of the sums, in values of rows g
#pragma unroll
    for (int hh = 0; hh < NH; ++hh) {
#pragma unroll
        for (int mask = 4; mask < 32; mask *= 2) l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], mask);
        if (g == 0) {
            s.m[head(hh)] = ref[hh];
            s.l[head(hh)] = l[hh];
        }
        float* so = reinterpret_cast<float*>(s.ring) + head(hh) * T::DV;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float m = 0.0f;
            if constexpr (U4) {
                m = mb[b][hh];
#pragma unroll
                for (int mask = 4; mask < 32; mask *= 2) m += __shfl_xor_sync(0xffffffffu, m, mask);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float(&sum)[2 * NH] = o[2 * b + k];
                const int d = U4 ? 32 * b + 4 * g + 2 * k : 32 * b + 16 * k + 2 * g;
                *reinterpret_cast<float2*>(so + d) =
                    make_float2(fmaf(sum[hh], UNIT, m), fmaf(sum[NH + hh], U4 ? UNIT / 16.0f : UNIT, m));
            }
        }
    }
}

// NB: blocks a head.  NH: 1 for up to four query heads, 2 for up to eight.
template <int KIND_, int NB_, int NH_>
struct AttnKvq {
    static constexpr int KIND = KIND_, NB = NB_, NH = NH_, NG = 4 * NH, DMAX = 32 * NB, DV = DMAX, SPLIT = 1;
    static constexpr bool HEAD_MAJOR = true;
    static constexpr int ROW = KIND == Q8_KVQ_U4 ? 16 * NB : 32 * NB, CH = ROW / 16;
    static constexpr int PITCH = (CH | 1) * 16;                // an odd number of 16 bytes: no bank twice
    static constexpr int WB = 4 * NB, WC = NB % 4 == 0 ? 16 : NB % 2 == 0 ? 8 : 4, WN = WB / WC;
    static constexpr int SUB = CH <= 4 ? 2 : 1, KT = 16 * SUB;
    static constexpr int CODES = KT * PITCH, WORDS = KT * WB, STAGE = 2 * (CODES + WORDS);
    // CTAs an SM: what registers allow without spills of more than some words (of four heads of
    // 128 4-bit values 112 us with 128 registers, 112 with 168; of eight 126 with 168, 108 with 255)
    static constexpr int CTAS = NH == 1 ? (NB <= 2 && CH <= 4 ? 4 : CH <= 12 ? 3 : 2) : NB <= 2 ? 3 : 2, MAX_CTAS = kKvqMaxCtas;
    static constexpr int RING = (CTAS == 4 ? 12 : CTAS == 3 ? 16 : 24) * 1024;
    static constexpr int S0 = RING / STAGE, S = S0 > 6 ? 6 : S0;
    static constexpr int TK = kAttnWarps * KT;
    static constexpr int EXTRA = (128 * 1024 + kAttnWarps * STAGE - 1) / (kAttnWarps * STAGE);
    static constexpr int LEAST = 1;
    static_assert(S >= 2 && NG * DMAX * 4 <= RING && STAGE % 16 == 0 && CODES % 16 == 0, "attention tile");
    static __device__ __forceinline__ void states(const Segment& s) { kvq_states<AttnKvq>(s); }
};

template <int KIND, int NH>
cudaError_t launch_attn_kvq_heads(const AttnParams& p, const LaunchCtx& ctx) {
    switch (p.a.dim / 32) {
        case 1: return launch_attn_kernel<AttnKvq<KIND, 1, NH>>(p, ctx);
        case 2: return launch_attn_kernel<AttnKvq<KIND, 2, NH>>(p, ctx);
        case 3: return launch_attn_kernel<AttnKvq<KIND, 3, NH>>(p, ctx);
        case 4: return launch_attn_kernel<AttnKvq<KIND, 4, NH>>(p, ctx);
        case 5: return launch_attn_kernel<AttnKvq<KIND, 5, NH>>(p, ctx);
        case 6: return launch_attn_kernel<AttnKvq<KIND, 6, NH>>(p, ctx);
        case 7: return launch_attn_kernel<AttnKvq<KIND, 7, NH>>(p, ctx);
        default: return launch_attn_kernel<AttnKvq<KIND, 8, NH>>(p, ctx);
    }
}

}  // namespace q8
