// attn.cuh -- attention of one token a sequence over its K/V cache: the kernel
// template and its launch (one translation unit a cache type).
//
// Mathematics.  With s_i = scale q.k_i (in units of log 2), one pass over K and
// V keeps a reference r, l = sum 2^(s_i - r) and o = sum 2^(s_i - r) v_i; r
// moves (and l, o are rescaled) only when a score exceeds it by more than 2^3,
// which binary32 takes without loss.  States over parts of the entries join by
// the same rule, so the entries may be split anywhere.  Scores, weights and
// sums are binary32 throughout.
//
// What bounds it.  Each K and V value is read once and used in one multiply-add
// a query head: with 4 heads a K/V head that is 1 (f32) or 2 (16-bit) FMA a
// byte, below what the FMA pipes give at full HBM bandwidth.  So the kernel
// streams: every warp owns a ring of stages in shared memory that it fills
// with 16-byte cp.async and consumes alone -- no barrier between warps, about
// 128 KB in flight an SM.
//
// Layout.  LPK lanes share an entry, each with DPL of its values in registers
// (q and o of NG query heads: 64 + 64 registers at most); a warp takes 32/LPK
// entries at a time, U times a stage.  A stage's U x NG partial scores are
// summed over the LPK lanes by halving exchanges (each step leaves a lane half
// the values), so that each lane ends with few scores, exponentiates those
// only, and hands them back by shuffles.
//
// Split.  A unit is a row's K/V head (and block of at most 8 query heads); its
// visible entries are tiles of 4 warps x KT (several such where the tiles would
// not fit 32 bits), and it counts some tiles more for what it costs to begin
// and end (128 KB of loads where CTAs have long shares: of 64, 128, 192 and 256 KB
// the best on long and ragged batches).  The tiles of all units in one line are
// cut evenly over the CTAs, so ragged batches balance and one long sequence fills
// the GPU (few units, fewer CTAs: the join of many parts would be the time);
// lengths are read on the device, so one captured graph serves every step.  Two CTAs of four
// warps an SM (quantised caches: T::CTAS): one streams while the other ends a unit.
//
// Measured (32 query and 8 K/V heads of 128 values; device time): 64 rows of
// 4100 to 8192 bf16 entries 240 to 248 us (by the box), 6.5 to 6.7 TB/s; 16 rows
// of up to 2052 visible f32 entries 42 us, 5.5 TB/s; one row of 130001 bf16
// entries 90 us, 5.9 TB/s, and 103 us with the weights accumulated; one row of 613
// f32 entries 8.1 us, of one entry 4.3 us: there the launch, three dependent reads (positions, q
// and the entries, the partial states) and the ticket are the time.  A unit cut
// between CTAs leaves partial states in the workspace; the CTA that finishes it
// last (a ticket) joins them in CTA order, so results repeat bit for bit.
#pragma once

#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "q8proj.h"

namespace q8 {

constexpr int kAttnWarps = 4;                         // T::CTAS CTAs an SM
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kAttnRing = 24 * 1024;                  // bytes a warp
constexpr int kAttnMaxCtas = 512;
// 16-bit caches take the matrix instructions (attn_mma.cuh) from five query heads
// a block on.  (32 rows of 4096 bf16 entries, 8 K/V heads of 128 values: 4 query
// heads each 91 us on the lanes, 96 on the matrix instructions; 8 query heads 145
// and 100.)
constexpr int kAttnLanesHeads = 4;
static_assert(4 * kAttnMaxCtas <= kCounterBytes, "one ticket a CTA");
// Quantised caches: CTAs of a call at most, and the query heads a kernel is built for.
constexpr int kKvqMaxCtas = 640;
static_assert(4 * kKvqMaxCtas <= kCounterBytes, "one ticket a CTA");
constexpr int kvq_block_heads(int heads) { return heads <= 4 ? 4 : 8; }

// What bounds the number of tiles of a call: the entries of a stage of all warps at least, and
// the tiles that a unit counts for its begin and end at most (4-bit heads of 32 values).
constexpr int kAttnLeastStage = 8, kAttnMostExtra = 26;

// Floats of a partial state, whole 16-byte words.
__host__ __device__ constexpr size_t attn_slot(int ng, int64_t dim) {
    return size_t(ng) * size_t(dim) + size_t(ng == 1 ? 4 : 2 * ng);
}

struct AttnParams {
    AttnArgs a;
    int nb, gsz;          // blocks of query heads a K/V head, heads a block
    int tile_its;         // stages a warp takes in one tile
    int64_t cap;          // entries of a row that can be visible
    float* part;          // [2 * CTAs][attn_slot(NG, D)]: o [NG][D], then (r, l) [NG]
    float2* ml;           // [rows][heads]: reference and 1 / sum (acc)
    float* scores;        // [rows][heads][cap] (acc)
    float qscale;         // scale * log2(e)
    int* err;
};

// The visible entries in order: entry v of nvis is cache row v + (v < ns ? 0 : gap).
struct Visible {
    uint32_t nvis, ns, gap;
};

__device__ __forceinline__ Visible visible(int pos, int64_t n_pos, int64_t window, int64_t sinks) {
    if (pos < -1 || pos >= n_pos) return {0, 0, 0};
    const uint32_t n = uint32_t(pos) + 1;
    if (window < 0 || window >= n) return {n, n, 0};
    const uint32_t rest = n - uint32_t(window), ns = sinks < rest ? uint32_t(sinks) : rest;
    return {ns + uint32_t(window), ns, rest - ns};
}

typedef unsigned long long f32x2;   // two binary32 values

__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float ex2(float x) {   // within 2^-22 of 2^x, relative
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 16 bytes from global to shared memory, or 16 zero bytes (nothing is read).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool read) {
    const int n = read ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The 16 bytes of a chunk as pairs of binary32 (both 16-bit types convert exactly).
template <int KV>
__device__ __forceinline__ void chunk_pairs(int4 c, f32x2* out) {
    if constexpr (KV == Q8_KV_F32) {
        out[0] = pack2(__int_as_float(c.x), __int_as_float(c.y));
        out[1] = pack2(__int_as_float(c.z), __int_as_float(c.w));
    } else {
        const int w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (KV == Q8_KV_BF16) {
                out[i] = pack2(__int_as_float(w[i] << 16), __int_as_float(w[i] & int(0xffff0000)));
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                out[i] = pack2(f.x, f.y);
            }
        }
    }
}

// What a warp computes of a segment: its own entries KT of every TK from v_begin
// on, for the block's query heads.
struct Segment {
    const AttnParams& p;
    int row, g0, ng;
    Visible vis;
    uint32_t pitch;          // bytes from one entry to the next
    int64_t off;             // of the row and K/V head in the caches (head-major ones: in entries)
    uint32_t v_end, v_begin;
    int its;                 // stages
    int half;                // of V's values, where two warps share them
    unsigned char* ring;
    float* q;                // shared: the block's query heads [NG][DMAX]
    float *m, *l;            // the warp's references and sums; its o goes to the ring [NG][DMAX]
};

// q by way of shared memory, scaled; zero behind D and behind the block's heads.
template <class T>
__device__ __forceinline__ void stage_q(const Segment& s) {
    const AttnArgs& a = s.p.a;
    const int D = int(a.dim);
#pragma unroll 4
    for (int e = threadIdx.x; e < T::NG * T::DMAX; e += kAttnThreads) {
        const int g = e / T::DMAX, d = e % T::DMAX;
        s.q[e] = g < s.ng && d < D ? a.q[s.row * a.ldq + int64_t(s.g0 + g) * D + d] * s.p.qscale : 0.0f;
    }
    __syncthreads();
}

template <class T>
__device__ __forceinline__ void lanes_states(const Segment& s) {
    constexpr int NG = T::NG, LPK = T::LPK, KV = T::KV;
    const AttnParams& p = s.p;
    const AttnArgs& a = p.a;
    const int lane = threadIdx.x & 31, D = int(a.dim), ng = s.ng, its = s.its;
    const int sl = lane % LPK, grp = lane / LPK, grp0 = lane - sl;
    const int gl = sl / T::LG;                             // this lane's query head of the block
    const int u0 = (sl / T::DUP) * T::R % T::U;            // and its first of R entry steps
    const int swz = LPK == 4 ? (grp & 1) * 4 : 0;          // rows next to each other on other banks
    const uint32_t ring_s = smem_u32(s.ring), v_begin = s.v_begin, v_end = s.v_end, pitch = s.pitch;
    const Visible vis = s.vis;
    // (a lane copies the same 16-byte column of every row it copies)
    constexpr int CPR = T::PITCH / 16, RPI = CPR < 32 ? 32 / CPR : 1;   // chunks a row, rows at a time
    const int r0 = CPR < 32 ? lane / CPR : 0, c0 = lane % CPR;
    const unsigned char* kp = static_cast<const unsigned char*>(a.k) + s.off + c0 * 16;
    const unsigned char* vp = static_cast<const unsigned char*>(a.v) + s.off + c0 * 16;
    const uint32_t dst0 = ring_s + r0 * T::PITCH + (LPK == 4 ? c0 ^ (r0 & 1) * 4 : c0) * 16;

    // (where the weights are accumulated: one lane of those that hold a score)
    float* const scores = p.scores && gl < ng && sl % T::DUP == 0
                              ? p.scores + (int64_t(s.row) * a.heads + s.g0 + gl) * p.cap
                              : nullptr;
    float ref = -INFINITY, l = 0.0f;    // of query head gl, over this lane group's entries

    int in_slot = 0, out_slot = 0;
    const auto load = [&](int it) {
        if (it < its) {
            const uint32_t st = dst0 + in_slot * (2 * T::HALF), vb = v_begin + uint32_t(it) * T::TK + r0;
            in_slot = in_slot + 1 == T::S ? 0 : in_slot + 1;
#pragma unroll
            for (int r = 0; r < T::KT; r += RPI) {
                const uint32_t v = vb + r, i = v + (v < vis.ns ? 0 : vis.gap);
                const bool in = v < v_end;
                const uint64_t at = in ? uint64_t(i) * pitch : 0;
#pragma unroll
                for (int c = 0; c < CPR; c += 32) {
                    static_assert(LPK != 4 || RPI % 2 == 0, "a lane's rows swap their halves alike");
                    if ((c0 + c) * T::CD < D) {
                        cp16(st + r * T::PITCH + c * 16, kp + at + c * 16, in);
                        cp16(st + T::HALF + r * T::PITCH + c * 16, vp + at + c * 16, in);
                    }
                }
            }
        }
        cp_commit();
    };
#pragma unroll 1
    for (int i = 0; i < T::S - 1; ++i) load(i);

    stage_q<T>(s);
    f32x2 q[NG][T::NP], o[NG][T::NP];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < T::NP; ++i) {
            const int d = (i / (T::CD / 2) * LPK + sl) * T::CD + i % (T::CD / 2) * 2;
            q[g][i] = *reinterpret_cast<const f32x2*>(s.q + g * T::DMAX + d);
            o[g][i] = 0ull;
        }
    for (int it = 0; it < its; ++it) {
        cp_wait<T::S - 2>();
        __syncwarp();
        load(it + T::S - 1);
        const uint32_t st = ring_s + out_slot * (2 * T::HALF);
        out_slot = out_slot + 1 == T::S ? 0 : out_slot + 1;
        const uint32_t vb = v_begin + uint32_t(it) * T::TK;
        // partial scores over this lane's values, x[g * U + u]
        float x[T::NV];
#pragma unroll
        for (int u = 0; u < T::U; ++u) {
            f32x2 k[T::NP];
#pragma unroll
            for (int c = 0; c < T::NC; ++c)
                chunk_pairs<KV>(lds128(st + (u * T::KPS + grp) * T::PITCH + ((c * LPK + sl) ^ swz) * 16),
                                k + c * (T::CD / 2));
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f32x2 dot = mul2(q[g][0], k[0]);
#pragma unroll
                for (int i = 1; i < T::NP; ++i) dot = fma2(q[g][i], k[i], dot);
                const float2 f = unpack2(dot);
                x[g * T::U + u] = f.x + f.y;
            }
        }
        // sum over the LPK lanes; lane sl keeps x[R * (sl / DUP) ...], R of them
        int n = T::NV;
#pragma unroll
        for (int mask = LPK / 2; mask; mask >>= 1) {
            if (n > 1) {
                n /= 2;
                const bool up = sl & mask;
#pragma unroll
                for (int i = 0; i < T::NV / 2; ++i) {
                    if (i >= n) break;
                    const float give = up ? x[i] : x[i + n], mine = up ? x[i + n] : x[i];
                    x[i] = mine + __shfl_xor_sync(0xffffffffu, give, mask);
                }
            } else {
                x[0] += __shfl_xor_sync(0xffffffffu, x[0], mask);
            }
        }
        bool moves = false;
#pragma unroll
        for (int r = 0; r < T::R; ++r) {
            const uint32_t v = vb + (u0 + r) * T::KPS + grp;
            if (scores && v < v_end) scores[v] = x[r];
            x[r] = v < v_end ? x[r] : -INFINITY;
            moves = moves || x[r] > ref + 8.0f;
        }
        if (__any_sync(0xffffffffu, moves)) {
            float top = ref;
#pragma unroll
            for (int r = 0; r < T::R; ++r) top = fmaxf(top, x[r]);
#pragma unroll
            for (int mask = T::LG / 2; mask; mask >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, mask));
            const float f = top == ref ? 1.0f : ex2(ref - top);
            ref = top;
            l *= f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float fg = __shfl_sync(0xffffffffu, f, grp0 + g * T::LG);
#pragma unroll
                for (int i = 0; i < T::NP; ++i) o[g][i] = mul2(o[g][i], pack2(fg, fg));
            }
        }
#pragma unroll
        for (int r = 0; r < T::R; ++r) {
            x[r] = x[r] == -INFINITY ? 0.0f : ex2(x[r] - ref);
            l += x[r];
        }
#pragma unroll
        for (int u = 0; u < T::U; ++u) {
            f32x2 v[T::NP];
#pragma unroll
            for (int c = 0; c < T::NC; ++c)
                chunk_pairs<KV>(
                    lds128(st + T::HALF + (u * T::KPS + grp) * T::PITCH + ((c * LPK + sl) ^ swz) * 16),
                    v + c * (T::CD / 2));
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float w = __shfl_sync(0xffffffffu, x[u % T::R],
                                            grp0 + (g * T::U + u) / T::R * T::DUP);
                const f32x2 ww = pack2(w, w);
#pragma unroll
                for (int i = 0; i < T::NP; ++i) o[g][i] = fma2(ww, v[i], o[g][i]);
            }
        }
    }
    cp_wait<0>();
    __syncwarp();

    // join the warp's lane groups, then the warps
    {
        float top = ref;
#pragma unroll
        for (int mask = LPK; mask < 32; mask <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, mask));
        const float f = ref == -INFINITY ? 0.0f : ex2(ref - top);
        // (l stays NaN where a score was NaN before any other)
        l = ref == -INFINITY ? l : l * f;
        const float fo = ref == -INFINITY ? 1.0f : f;   // o is 0 or NaN there
#pragma unroll
        for (int mask = LPK; mask < 32; mask <<= 1) l += __shfl_xor_sync(0xffffffffu, l, mask);
#pragma unroll
        for (int mask = T::LG / 2; mask; mask >>= 1) l += __shfl_xor_sync(0xffffffffu, l, mask);
        l *= 1.0f / T::DUP;
        if (grp == 0 && sl % T::LG == 0) {
            s.m[gl] = top;
            s.l[gl] = l;
        }
        f32x2 z[NG * T::NP];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const float fg = __shfl_sync(0xffffffffu, fo, grp0 + g * T::LG);
#pragma unroll
            for (int i = 0; i < T::NP; ++i) z[g * T::NP + i] = mul2(o[g][i], pack2(fg, fg));
        }
        constexpr int P = NG * T::NP, KEEP = P / T::KPS;
        int n = P;
#pragma unroll
        for (int mask = 16; mask >= LPK; mask >>= 1) {
            n /= 2;
            const bool up = lane & mask;
#pragma unroll
            for (int i = 0; i < P / 2; ++i) {
                if (i >= n) break;
                const f32x2 give = up ? z[i] : z[i + n], mine = up ? z[i + n] : z[i];
                const float2 y = unpack2(__shfl_xor_sync(0xffffffffu, give, mask)), w = unpack2(mine);
                z[i] = pack2(w.x + y.x, w.y + y.y);
            }
        }
        float* so = reinterpret_cast<float*>(s.ring);     // [NG][DMAX]
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int at = grp * KEEP + i, g = at / T::NP, pr = at % T::NP;
            const int d = (pr / (T::CD / 2) * LPK + sl) * T::CD + pr % (T::CD / 2) * 2;
            *reinterpret_cast<float2*>(so + g * T::DMAX + d) = unpack2(z[i]);
        }
    }
}

template <int KV_, int NG_, int LPK_>
struct AttnLanes {
    static constexpr int KV = KV_, NG = NG_, LPK = LPK_;
    static constexpr int ELT = KV == Q8_KV_F32 ? 4 : 2;
    static constexpr int CD = 16 / ELT;                       // values a 16-byte chunk
    static constexpr int DPL = NG <= 4 ? 16 : 8;              // values a lane
    static constexpr int NC = DPL / CD;                       // chunks a lane
    static constexpr int NP = DPL / 2;                        // pairs a lane
    static constexpr int DMAX = DPL * LPK, DV = DMAX, SPLIT = 1;
    static constexpr int PITCH = DMAX * ELT;                  // bytes an entry in a stage
    static constexpr int KPS = 32 / LPK;                      // entries a warp takes at a time
    static constexpr int U = KV == Q8_KV_F32 ? 2 : 4;
    static constexpr int KT = KPS * U;                        // entries a stage
    static constexpr int HALF = KT * PITCH;                   // bytes of K (and of V) a stage
    static constexpr int S0 = kAttnRing / (2 * HALF);
    static constexpr int S = S0 > 6 ? 6 : S0;                 // stages
    static constexpr int TK = kAttnWarps * KT;                // entries a stage of all warps
    static constexpr int EXTRA = (128 * 1024 + kAttnWarps * 2 * HALF - 1) / (kAttnWarps * 2 * HALF);
    static constexpr int NV = U * NG;                         // scores of an entry group a stage
    static constexpr int R = NV > LPK ? NV / LPK : 1;         // scores a lane ends with
    static constexpr int DUP = LPK > NV ? LPK / NV : 1;       // lanes holding the same scores
    static constexpr int LG = LPK / NG;                       // lanes a query head
    static constexpr int LEAST = NG == 8 ? 1 : 2;             // tiles a CTA, at least
    static constexpr int CTAS = 2, RING = kAttnRing, MAX_CTAS = kAttnMaxCtas;
    static constexpr bool HEAD_MAJOR = false;
    static_assert(S >= 2 && LG >= 1 && U % R == 0 && R * LPK >= NV, "attention tile");
    static_assert(NG * DMAX * 4 <= kAttnRing, "a warp's state fits its ring");

    static __device__ __forceinline__ void states(const Segment& s) { lanes_states<AttnLanes>(s); }
};

template <class T>
__global__ void __launch_bounds__(kAttnThreads, T::CTAS) attn_kernel(const AttnParams p) {
    constexpr int NG = T::NG, WARPS = kAttnWarps / T::SPLIT;      // warps that share a stage's entries
    static_assert(T::TK >= kAttnLeastStage && T::EXTRA <= kAttnMostExtra, "launch_attn's bound on the tiles of a call");
    extern __shared__ __align__(256) unsigned char ring_raw[];
    unsigned char* const ring_all = ring_raw + (512 - (smem_u32(ring_raw) & 511) & 511);   // stages on whole rows
    __shared__ uint32_t s_pre[Q8_MAX_ROWS + 1];   // tiles before each row
    __shared__ uint32_t s_warp[kAttnWarps];
    __shared__ int s_pos[Q8_MAX_ROWS];
    __shared__ __align__(16) float s_q[NG * T::DMAX];
    __shared__ float s_m[kAttnWarps][NG], s_l[kAttnWarps][NG];
    __shared__ int s_last;
    const AttnArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = int(a.dim), rows = int(a.rows);
    const uint32_t per_row = uint32_t(a.kv_heads) * p.nb;
    const int TT = T::TK * p.tile_its;                     // entries a tile
    unsigned char* ring = ring_all + warp * T::RING;
    const uint32_t ring_s = smem_u32(ring);

    // values behind D are never copied; they stay zero
    if (D < T::DMAX) {
        for (int i = lane; i < T::RING / 16; i += 32) reinterpret_cast<int4*>(ring)[i] = int4{0, 0, 0, 0};
    }
    pdl_wait();
    pdl_launch_dependents();

    // tiles of each row (a row with nothing visible has one, which writes its zeros)
    {
        constexpr int PER = (Q8_MAX_ROWS + kAttnThreads - 1) / kAttnThreads;
        uint32_t n[PER], x = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int m = tid * PER + i;
            if (m < rows) {
                const int pos = a.pos[m];
                s_pos[m] = pos;
                if (blockIdx.x == 0 && (pos < -1 || pos >= a.n_pos)) atomicExch(p.err, Q8_DEVERR_POSITION);
                // (up to 2^31 - 1 entries, so 32 bits hold the rounding up)
                const uint32_t nvis = visible(pos, a.n_pos, a.window, a.sinks).nvis;
                x += (nvis ? (nvis + TT - 1) / TT : 1) * per_row;
            }
            n[i] = x;
        }
        const uint32_t own = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        for (int w = 0; w < warp; ++w) x += s_warp[w];
        if (tid == 0) s_pre[0] = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) s_pre[tid * PER + i + 1] = x - own + n[i];
        __syncthreads();
    }
    // CTA c has tiles [first(c), first(c + 1)): all of them in equal shares, the
    // first ones one longer.  Small problems: a tile or two a CTA (fewer cost more
    // to join than they save; one where a tile is fewer bytes and more work), or a
    // unit.  Few units: of T tiles cut in P parts, one CTA's tiles take T / P and
    // the join P, so P grows with the root of T (one row's K/V head with 8 query
    // heads, on all CTAs and so: 48000 bf16 entries of 128 values 67 and 28 us, 3408
    // f32 entries of 80 values 34 and 16 us; factors of 2 to 20 tried).
    const uint32_t real = s_pre[rows], units = uint32_t(rows) * per_row;
    const uint32_t extra = real >= 4 * gridDim.x ? T::EXTRA : 1, W = real + extra * units;
    constexpr float ROOT = NG * T::DMAX > 512 ? 5.0f : 8.0f;
    const uint32_t best = uint32_t(__fsqrt_rn(ROOT * float(real) * float(units)));
    const uint32_t ctas = min(max(min(real / T::LEAST, best), units), gridDim.x), cta = blockIdx.x;
    __syncthreads();
    for (int i = tid; i <= rows; i += kAttnThreads) s_pre[i] += extra * i * per_row;
    __syncthreads();
    if (cta >= ctas) return;
    const uint32_t share = W / ctas, longer = W % ctas;
    const auto first = [&](uint32_t c) { return c * share + min(c, longer); };
    const auto owner = [&](uint32_t tile) {
        const uint32_t edge = longer * (share + 1);
        return tile < edge ? tile / (share + 1) : longer + (tile - edge) / share;
    };
    const uint32_t t_begin = first(cta), t_end = first(cta + 1);
    uint32_t t0 = t_begin;

    while (t0 < t_end) {
        // the segment: tiles [t0, t1) of unit (m, h, b)
        int lo = 0, hi = rows - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (s_pre[mid] <= t0) lo = mid; else hi = mid - 1;
        }
        const int m = lo;
        const uint32_t span = (s_pre[m + 1] - s_pre[m]) / per_row, tiles = span - extra;
        const uint32_t unit = (t0 - s_pre[m]) / span;
        const uint32_t unit0 = s_pre[m] + unit * span;              // the unit's first tile
        if (t0 >= unit0 + tiles) {                                  // in its extra ones
            t0 = unit0 + span;
            continue;
        }
        const uint32_t t1 = min(unit0 + tiles, t_end);
        const int h = int(unit / p.nb), b = int(unit % p.nb);
        const int group = int(uint32_t(a.heads) / uint32_t(a.kv_heads));
        const int g0 = h * group + b * p.gsz;                       // the block's first query head
        const int ng = min(p.gsz, group - b * p.gsz);
        const Visible vis = visible(s_pos[m], a.n_pos, a.window, a.sinks);
        uint32_t pitch;
        int64_t off;
        if constexpr (T::HEAD_MAJOR) {
            pitch = T::ROW;
            off = (int64_t(m) * a.kv_heads + h) * a.n_pos;
        } else {
            pitch = uint32_t(a.kv_heads) * D * T::ELT;                 // (below 2^21)
            off = (int64_t(m) * a.n_pos * a.kv_heads + h) * D * T::ELT;
        }
        // this warp's entries: KT of every TK from v_begin on.  At most 2^31 - 1 are
        // visible, so 32 bits hold every index and a tile more.
        const uint64_t upto = uint64_t(t1 - unit0) * TT;
        const uint32_t v_end = uint32_t(vis.nvis < upto ? vis.nvis : upto);
        const int half = warp / WARPS;
        const uint64_t v_from = uint64_t(t0 - unit0) * TT + (warp - half * WARPS) * T::KT;
        const uint32_t v_begin = uint32_t(v_from);
        const int its = v_end > v_from ? int((v_end - v_begin + T::TK - 1) / T::TK) : 0;
        const Segment seg{p, m, g0, ng, vis, pitch, off, v_end, v_begin, its, half, ring, s_q, s_m[warp], s_l[warp]};
        T::states(seg);
        __syncthreads();

        // the CTA's state of the segment, and the whole unit's where it is all here
        const auto put = [&](int g, int d, float4 v, float sum, bool any) {
            float* out = a.out + m * a.ldo + int64_t(g0 + g) * D + d;      // (ldo may be odd)
            out[0] = any ? v.x / sum : 0.0f;
            out[1] = any ? v.y / sum : 0.0f;
            out[2] = any ? v.z / sum : 0.0f;
            out[3] = any ? v.w / sum : 0.0f;
        };
        const bool whole = t0 == unit0 && t1 == unit0 + tiles;
        const uint32_t c_first = owner(unit0), c_last = owner(unit0 + tiles - 1);
        const size_t slot = attn_slot(NG, D);
        float* part = p.part + (2 * cta + (t_begin >= unit0 ? 0 : 1)) * slot;
        const int D4 = D / 4;
        for (int e = tid; e < ng * D4; e += kAttnThreads) {
            const int g = e / D4, d = (e - g * D4) * 4;
            float top = s_m[0][g];
#pragma unroll
            for (int w = 1; w < kAttnWarps; ++w) top = fmaxf(top, s_m[w][g]);
            float sum = 0.0f;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const int h0 = d / T::DV * WARPS;                     // the first warp that holds these values
#pragma unroll
            for (int i = 0; i < WARPS; ++i) {
                const int w = h0 + i;
                const float f = s_m[w][g] == -INFINITY ? 1.0f : ex2(s_m[w][g] - top);   // l and o: 0 or NaN
                const float4 o4 =
                    *reinterpret_cast<const float4*>(ring_all + w * T::RING + (g * T::DV + d % T::DV) * 4);
                sum += s_l[w][g] * f;
                v.x += o4.x * f, v.y += o4.y * f, v.z += o4.z * f, v.w += o4.w * f;
            }
            if (whole) {
                put(g, d, v, sum, vis.nvis != 0);
                if (d == 0 && p.ml) p.ml[int64_t(m) * a.heads + g0 + g] = make_float2(top, 1.0f / sum);
            } else {
                *reinterpret_cast<float4*>(part + g * D + d) = v;
                if (d == 0) *reinterpret_cast<float2*>(part + NG * D + 2 * g) = make_float2(top, sum);
            }
        }
        if (!whole) {
            unsigned* ticket = static_cast<unsigned*>(a.ws) + c_first;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const unsigned before = atomicAdd(ticket, 1u);
                s_last = before == c_last - c_first;
                if (s_last) *ticket = 0u;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                // a CTA's state is in its first slot if it begins inside the unit, as
                // every one behind c_first does
                const float* p0 = p.part + (2 * c_first + (first(c_first) < unit0 ? 1 : 0)) * slot;
                const float* p1 = p.part + 2 * (c_first + 1) * slot;
                const int n = int(c_last - c_first) + 1;
                const auto from = [&](int i) { return i ? p1 + (i - 1) * 2 * slot : p0; };
                const auto state = [&](int i, int g) {      // reference and sum of part i
                    return __ldcg(reinterpret_cast<const float2*>(from(i) + NG * D + 2 * g));
                };
                // (the states in the ring have been read) the factors, then as many
                // parts' o at a time as fit, copied by all threads: one CTA's plain
                // loads in turn would be the time of a unit that many share
                float* const s_f = reinterpret_cast<float*>(ring_all);
                constexpr int FACTORS = T::MAX_CTAS * NG * 4;
                constexpr int FIT = (kAttnWarps * T::RING - FACTORS) / (NG * T::DMAX * 4);
                const float4* const s_x = reinterpret_cast<const float4*>(ring_all + FACTORS);
                const int E = ng * D4;
                const auto fetch = [&](int i0) {
                    const int end = min(i0 + FIT, n);
                    for (int i = i0 + warp; i < end; i += kAttnWarps) {
                        const float* src = from(i);
                        const uint32_t dst = smem_u32(s_x + (i - i0) * E);
#pragma unroll 4
                        for (int e = lane; e < E; e += 32) cp16(dst + 16 * e, src + 4 * e, true);
                    }
                    cp_commit();
                };
                fetch(0);
                // one warp a query head: factors 2^(r_i - r), the sum and 1 / sum
                for (int g = warp; g < ng; g += kAttnWarps) {
                    const float2 mine = lane < n ? state(lane, g) : make_float2(-INFINITY, 0.0f);
                    float top = mine.x, sum = 0.0f;
                    for (int i = lane + 32; i < n; i += 32) top = fmaxf(top, state(i, g).x);
#pragma unroll
                    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    for (int i = lane; i < n; i += 32) {
                        const float2 rl = i == lane ? mine : state(i, g);
                        const float f = rl.x == -INFINITY ? 1.0f : ex2(rl.x - top);
                        s_f[i * NG + g] = f;
                        sum += rl.y * f;
                    }
#pragma unroll
                    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                    if (lane == 0) {
                        s_l[0][g] = sum;
                        if (p.ml) p.ml[int64_t(m) * a.heads + g0 + g] = make_float2(top, 1.0f / sum);
                    }
                }
                // where there are at most half as many float4 as threads, several threads
                // share one, each every share-th part
                constexpr int NE = (NG * T::DMAX / 4 + kAttnThreads - 1) / kAttnThreads;
                const int bits = E <= kAttnThreads / 2 ? 32 - __clz(E - 1) : 31;    // (E >= 2)
                const int share = E <= kAttnThreads / 2 ? kAttnThreads >> bits : 1, sub = tid >> bits;
                const int mine = tid - (sub << bits);
                float4 v[NE];
#pragma unroll
                for (int j = 0; j < NE; ++j) v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int i0 = 0; i0 < n; i0 += FIT) {
                    if (i0) fetch(i0);
                    cp_wait<0>();
                    __syncthreads();
                    const int end = min(FIT, n - i0);
#pragma unroll
                    for (int j = 0; j < NE; ++j) {
                        const int e = mine + j * kAttnThreads;
                        if (e >= E) continue;
                        const int g = e / D4;
#pragma unroll 4
                        for (int i = sub; i < end; i += share) {
                            const float4 x = s_x[i * E + e];
                            const float f = s_f[(i0 + i) * NG + g];
                            v[j].x += x.x * f, v[j].y += x.y * f, v[j].z += x.z * f, v[j].w += x.w * f;
                        }
                    }
                    __syncthreads();
                }
                if (share > 1) {
                    float4* const s_v = reinterpret_cast<float4*>(ring_all + FACTORS);
                    s_v[tid] = v[0];
                    __syncthreads();
                    for (int k = 1; tid < E && k < share; ++k) {
                        const float4 x = s_v[tid + (k << bits)];
                        v[0].x += x.x, v[0].y += x.y, v[0].z += x.z, v[0].w += x.w;
                    }
                }
#pragma unroll
                for (int j = 0; j < NE; ++j) {
                    const int e = tid + j * kAttnThreads;
                    if (e < E) put(e / D4, e % D4 * 4, v[j], s_l[0][e / D4], true);
                }
                if (D < T::DMAX) {     // values behind D are zero again
                    __syncthreads();
                    for (int i = tid; i < kAttnWarps * T::RING / 16; i += kAttnThreads)
                        reinterpret_cast<int4*>(ring_all)[i] = int4{0, 0, 0, 0};
                }
            }
        }
        __syncthreads();
        if (D < T::DMAX) {   // the states overwrote values behind D
            for (int i = lane; i < NG * T::DMAX / 4; i += 32) reinterpret_cast<int4*>(ring)[i] = int4{0, 0, 0, 0};
            __syncwarp();
        }
        t0 = t1;
    }
}

template <class T>
cudaError_t launch_attn_kernel(const AttnParams& p, const LaunchCtx& ctx) {
    static std::atomic<bool> ready[kMaxDevices];
    const auto kern = attn_kernel<T>;
    constexpr size_t smem = size_t(kAttnWarps) * T::RING + 512;
    const cudaError_t e = set_smem_once(kern, smem, ctx.dev, ready);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attrs[1];
    cfg.gridDim = dim3(unsigned(T::CTAS * ctx.num_sms < T::MAX_CTAS ? T::CTAS * ctx.num_sms : T::MAX_CTAS));
    cfg.blockDim = dim3(kAttnThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = ctx.stream;
    cfg.numAttrs = pdl_attrs(ctx, attrs);
    cfg.attrs = attrs;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// LPK, the lanes that hold an entry's values, by head_dim.
template <int KV, int NG>
cudaError_t launch_attn_lanes(const AttnParams& p, const LaunchCtx& ctx) {
    constexpr int SHARE = AttnLanes<KV, NG, 8>::DPL == 16 ? 1 : 2;
    if (p.a.dim <= 64) return launch_attn_kernel<AttnLanes<KV, NG, 4 * SHARE>>(p, ctx);
    if (p.a.dim <= 128) return launch_attn_kernel<AttnLanes<KV, NG, 8 * SHARE>>(p, ctx);
    return launch_attn_kernel<AttnLanes<KV, NG, 16 * SHARE>>(p, ctx);
}

template <int KV>
cudaError_t launch_attn_type(const AttnParams& p, const LaunchCtx& ctx) {
    if (p.gsz == 1) return launch_attn_lanes<KV, 1>(p, ctx);
    if (p.gsz == 2) return launch_attn_lanes<KV, 2>(p, ctx);
    if constexpr (KV == Q8_KV_F32)
        if (p.gsz > kAttnLanesHeads) return launch_attn_lanes<KV, 8>(p, ctx);
    return launch_attn_lanes<KV, 4>(p, ctx);
}

}  // namespace q8
