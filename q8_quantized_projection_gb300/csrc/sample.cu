// sample.cu -- sampling of one token a row from the head's logits.
//
// Mathematics.  A token's weight is an integer, 2^((x - M) log2(e) / T) in
// units of 2^-shift rounded down, so every sum is exact and independent of its
// order: what is drawn depends on nothing but the row and its settings.  The
// filters cut the tokens in order of x (ties: the lowest index first), so what
// they leave is "x > t, or x = t and index <= last".  Shares of a sum (top_p,
// u) are exact products of integers too.
//
// Layout.  A cluster of 1 to 8 CTAs takes a row, each an equal part of it in
// index order, read once into shared memory (parts past 46 K logits are read
// again from L2 instead).  The CTAs hand sums to one another through
// distributed shared memory: one cluster barrier an exchange.
//
// Top-k of up to some hundreds: the lanes' maxima give a logit (`reach`) that
// at least k tokens reach; the tokens that reach it, 600 of 128256 for k = 50,
// are listed, and the first CTA does the rest on the list alone (what a
// histogram leaves of it, up to 128 tokens, by comparing every pair).
//
// Otherwise a cut (the k-th largest; the end of the nucleus) is found without
// sorting the row: a histogram of 1024 bins linear in x (counts, or masses to
// 2^-21) names the bin that holds it; an exact pass sums what lies above that
// bin and lists the bin's tokens (some hundreds); every CTA takes the whole list,
// and each of its own tokens adds up what goes before it, which says whether it
// stays and whether it is the cut.  Longer lists are sorted by the first CTA.
// Where the list is too long (thousands of equal logits), a binary search over
// the 32 bits of the ordered logits finds the cut instead, with exact sums at
// each step.
//
// What bounds it.  One row: latency, of exchanges and of code that runs once
// (no arithmetic of 64-bit floats: at 2 lanes a clock and SM, one division in
// every thread cost 5 us).  A batch: the same latency, 17 of a CTA's 39 us, in two
// waves of clusters (64 rows of 128256, two CTAs an SM), then the instructions, 45
// for an exact weight and about 170 a token in all against 4 bytes read, at 0.49
// issued a clock and scheduler, and the histogram's shared atomics, 5 of the 39.
// (An exponent of 5 instructions in place of 16 gained 0.2 us of the 84.)  64
// registers for two CTAs an SM: 48 bytes are spilled.
//
// Measured (device time): 3 rows of 1001 tokens 9 us, one of 128256 with every
// filter 15 us, 64 of 128256 with top-p 85 us, 256 of 32003 with settings of
// their own 69 us.  CTAs of 512 threads and two CTAs an SM: on an earlier form at
// 100 us for the 64 rows, 256 threads and parts of 8 K (clusters of 16) took 137
// us, 1024 and 32 K 103 us, and 86 and 93 on the 256 rows at 75 us.
#include <cooperative_groups.h>
#include <float.h>
#include <math.h>

#include "common.cuh"
#include "launch.h"

namespace q8 {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarpsN = kThreads / 32;
constexpr int kTile = 128;                  // logits a warp takes at a time, four a lane
constexpr int kPart = kWarpsN * kTile;      // a CTA's part is a multiple of this
constexpr int kMaxPart = 46 * 1024;         // logits of a part held in shared memory
constexpr int kPairPart = 18 * 1024;        // the same with two CTAs an SM
constexpr int kBins = 1024, kList = 2048, kMaxCluster = 8;
constexpr uint32_t kPairs = kBins / 2, kPairsOne = 128;   // lists up to these are compared pair by pair (one CTA a row)
constexpr int kShort = kThreads / 4;        // a longer list is cut by a histogram, and what is longer then is sorted
typedef unsigned long long u64;

// What the CTAs of a cluster exchange: sums a, b, g, e and e2, the largest c
// and c2, the smallest d; s: a sum of weights as a float, of which a logit of
// key c weighs 1 (0: none).  A slot a CTA, two sets used in turn, so that a slot
// is written again only after a barrier behind its last reader.
struct Slot {
    u64 a = 0, b = 0, g = 0;
    uint32_t e = 0, e2 = 0, c = 0, c2 = 0, d = 0xffffffffu;
    float s = 0.0f;
};
enum { kA = 1, kB = 2, kG = 4, kE = 8, kE2 = 16, kC = 32, kC2 = 64, kD = 128, kS = 256 };

struct Shared {
    Slot slot[2][kMaxCluster];
    Slot warp[kWarpsN];                     // the same by warp of this CTA
    u64 scan[kWarpsN];
    uint32_t hist[kBins];
    u64 list[kList];                        // (ordered logit, ~index) of listed tokens
    u64 mine[kList];                        // this CTA's part of the list; then weights, or what a histogram left
    uint32_t listed;                        // tokens this CTA listed
    float cut_x;                            // the cut that the first CTA found
    uint32_t cut_i;
    uint32_t found;                         // an index, bin or place that one thread found
    uint2 pow2[64];                         // 2^(j/64): in units of 2^-31, and as a float of those
};

// The dynamic shared memory: Shared, then the CTA's part of the row.
extern __shared__ __align__(16) unsigned char smem[];
__device__ __forceinline__ Shared& sh() { return *reinterpret_cast<Shared*>(smem); }
__device__ __forceinline__ float* sh_x() { return reinterpret_cast<float*>(smem + sizeof(Shared)); }
static_assert(sizeof(Shared) % 16 == 0 && sizeof(Shared) + 4 * kMaxPart <= 227 * 1024, "shared memory");
static_assert(2 * (sizeof(Shared) + 4 * kPairPart + 1024) <= 228 * 1024, "two CTAs an SM");

// A logit as it is taken: NaN as -inf (never drawn), +inf as the largest float.
__device__ __forceinline__ float clean(float v) { return v > -INFINITY ? fminf(v, FLT_MAX) : -INFINITY; }

// Order of the logits as unsigned integers; 0: NaN or -inf, never drawn.
__device__ __forceinline__ uint32_t logit_key(float x) {
    if (!(x > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ float exp2_rough(float y) {      // to about 2^-22; 0 below 2^-126
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
    return r;
}

// 2^(j/64) in units of 2^-31.
__constant__ uint32_t kPow2[64] = {
    2147483648u, 2170868212u, 2194507417u, 2218404036u, 2242560872u, 2266980759u, 2291666561u, 2316621173u,
    2341847524u, 2367348571u, 2393127307u, 2419186755u, 2445529972u, 2472160047u, 2499080105u, 2526293303u,
    2553802834u, 2581611923u, 2609723834u, 2638141863u, 2666869345u, 2695909648u, 2725266179u, 2754942382u,
    2784941738u, 2815267765u, 2845924021u, 2876914102u, 2908241642u, 2939910317u, 2971923842u, 3004285971u,
    3037000500u, 3070071267u, 3103502151u, 3137297074u, 3171459999u, 3205994934u, 3240905930u, 3276197082u,
    3311872529u, 3347936457u, 3384393094u, 3421246719u, 3458501653u, 3496162267u, 3534232978u, 3572718252u,
    3611622603u, 3650950594u, 3690706840u, 3730896002u, 3771522796u, 3812591987u, 3854108391u, 3896076880u,
    3938502376u, 3981389855u, 4024744348u, 4068570940u, 4112874773u, 4157661043u, 4202935003u, 4248701965u};

// Weights of a row.  The exponent y = (x - M) log2(e) / T is carried as an
// unevaluated sum of two floats (the difference by the exact two-term sum, its
// product with a two-term constant), split into J/64 + h with |h| <= 1/128 and
// a little; 2^h - 1 is its Taylor polynomial to degree 3 (remainder 2^-34).
// The largest error is that polynomial's and h's own rounding, 2^-29 of the
// weight; sums over n tokens average it, so that fewer than one draw in 10^7
// has a border within it.
struct Weights {
    float M, pre, ch, cl;   // pre: 1/2 where differences could overflow
    int shift;

    // 2^y as mantissa (in units of 2^-31, up to 2^32) * 2^n; false: below one unit
    __device__ __forceinline__ bool parts(float x, uint32_t& mant, int& n) const {
        const float a = x * pre, s = a - M, bb = s - a;
        const float err = (a - (s - bb)) + (-M - bb);
        const float p = __fmul_rn(s, ch);                // (rounded: e is what it lost)
        float e = fmaf(s, ch, -p);
        e = fmaf(s, cl, e);
        e = fmaf(err, ch, e);
        const float kRound = 196608.0f;                  // 1.5 * 2^17: one step is 1/64
        const float r = p + kRound;
        const int J = __float_as_int(r) - __float_as_int(kRound);
        const float h = (p - (r - kRound)) + e;
        float q = fmaf(h, 0.05550411f, 0.2402265f);      // ln(2)^3/6, ln(2)^2/2, ln(2)
        q = fmaf(h, q, 0.6931472f);
        q *= h;
        const uint2 t = sh().pow2[J & 63];
        mant = t.x + uint32_t(__float2int_rn(__uint_as_float(t.y) * q));
        n = J >> 6;
        return p > -float(shift);
    }
    __device__ __forceinline__ u64 operator()(float x) const {
        uint32_t mant;
        int n;
        const bool any = parts(x, mant, n);
        return (u64(any ? mant : 0u) << 31) >> ((62 - shift - n) & 63);
    }
    // the histogram's coordinate: bin b holds b <= y < b + 1, the last one all that lies lower
    __device__ __forceinline__ float depth(float x, float scale) const {
        return (M - x * pre) * scale;
    }
    // the histogram's bin: (M - x) * scale, the last one for all that lies lower
    __device__ __forceinline__ int bin(float x, float scale) const {
        // (added to 2^23 rounded down: whole units; a quarter of the time of a conversion)
        const float y = fminf(depth(x, scale), float(kBins - 1));
        return __float_as_int(__fadd_rd(y, 8388608.0f)) - 0x4b000000;
    }
    // 2^y to about 2^-21, for the histogram; 0 below 2^-126
    __device__ __forceinline__ float rough(float x) const {
        return exp2_rough((x * pre - M) * ch);
    }
};

struct Cut {
    float t;         // kept: x > t, or x = t and index <= last
    uint32_t last;
    __device__ __forceinline__ bool has(float x, uint32_t i) const { return x > t || (x == t && i <= last); }
};

// f * S for 0 <= f <= 1 as an integer, rounded down or up, exactly.
__device__ __forceinline__ u64 share(float f, u64 S, bool up) {
    const uint32_t bits = __float_as_uint(f), eb = bits >> 23;
    const u64 m = (bits & 0x7fffffu) | (eb ? 0x800000u : 0u);        // f = m * 2^-k
    const int k = 150 - int(max(eb, 1u));
    const u64 lo = m * S, hi = __umul64hi(m, S);
    u64 q = 0, rest = lo | hi;
    if (k < 64) {
        q = (hi << (64 - k)) | (lo >> k);
        rest = lo << (64 - k);
    } else if (k == 64) {
        q = hi;
        rest = lo;
    } else if (k < 128) {
        q = hi >> (k - 64);
        rest = lo | (hi << (128 - k));
    }
    return q + (up && rest);
}

// Sum over the warp, in three fields that 32 lanes cannot overflow.
__device__ __forceinline__ u64 warp_sum(u64 v) {
    const uint32_t lo = __reduce_add_sync(0xffffffffu, uint32_t(v) & 0x7ffffffu);
    const uint32_t mid = __reduce_add_sync(0xffffffffu, uint32_t(v >> 27) & 0x7ffffffu);
    const uint32_t hi = __reduce_add_sync(0xffffffffu, uint32_t(v >> 54));
    return u64(lo) + (u64(mid) << 27) + (u64(hi) << 54);
}

__device__ __forceinline__ u64 warp_scan(u64 v) {     // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += y;
    }
    return v;
}

// Exclusive prefix sum over the CTA's threads; the whole sum in *all.
__device__ __noinline__ u64 block_scan(u64 v, u64* all) {
    Shared& s = sh();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const u64 up = warp_scan(v);
    __syncthreads();
    if (lane == 31) s.scan[warp] = up;
    __syncthreads();
    const u64 w = warp_scan(lane < kWarpsN ? s.scan[lane] : 0);
    *all = __shfl_sync(0xffffffffu, w, 31);
    const u64 before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return (warp ? before : 0) + up - v;
}

// (c: the exponent's factor, for s)
template <int F>
__device__ __forceinline__ void warp_reduce(Slot& v, float c = 0.0f) {
    if constexpr (F & kS) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, v.c);
        v.s = v.c == top ? v.s : v.c ? v.s * exp2_rough((key_logit(v.c) - key_logit(top)) * c) : 0.0f;
        v.c = top;
#pragma unroll
        for (int d = 16; d; d >>= 1) v.s += __shfl_xor_sync(0xffffffffu, v.s, d);
    }
    if constexpr (F & kA) v.a = warp_sum(v.a);
    if constexpr (F & kB) v.b = warp_sum(v.b);
    if constexpr (F & kG) v.g = warp_sum(v.g);
    if constexpr (F & kE) v.e = __reduce_add_sync(0xffffffffu, v.e);
    if constexpr (F & kE2) v.e2 = __reduce_add_sync(0xffffffffu, v.e2);
    if constexpr ((F & kC) && !(F & kS)) v.c = __reduce_max_sync(0xffffffffu, v.c);
    if constexpr (F & kC2) v.c2 = __reduce_max_sync(0xffffffffu, v.c2);
    if constexpr (F & kD) v.d = __reduce_min_sync(0xffffffffu, v.d);
}

// The fields F of every thread's Slot over the cluster as one; before (if
// given) receives the sum of a over the CTAs before this one.
template <int F>
__device__ __forceinline__ Slot exchange(Slot v, int& phase, u64* before = nullptr, float c = 0.0f) {
    Shared& s = sh();
    cg::cluster_group cl = cg::this_cluster();
    const unsigned rank = cl.block_rank(), size = cl.num_blocks();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    warp_reduce<F>(v, c);
    if (lane == 0) s.warp[warp] = v;
    __syncthreads();
    Slot* const slots = s.slot[phase];
    phase ^= 1;
    if (warp == 0) {
        v = Slot();
        if (lane < kWarpsN) v = s.warp[lane];
        warp_reduce<F>(v, c);
        if (lane < int(size)) *cl.map_shared_rank(&slots[rank], lane) = v;
    }
    cluster_sync(size);
    v = Slot();
    if (lane < int(size)) v = slots[lane];
    if (before) *before = warp_sum(lane < int(rank) ? v.a : 0);
    warp_reduce<F>(v, c);
    return v;
}

// Bitonic steps k (all of j = 32 .. 1) on the 64 numbers a[lane], a[lane + 32]
// of a warp, which begin at place `at` of what is sorted; the largest first.
__device__ __forceinline__ void warp_steps(u64& lo, u64& hi, int at, int k, int j0) {
    const int lane = threadIdx.x & 31;
    for (int j = j0; j; j >>= 1) {
        if (j == 32) {
            const bool down = ((at + lane) & k) == 0;
            if ((lo < hi) == down) {
                const u64 t = lo;
                lo = hi;
                hi = t;
            }
        } else {
            const u64 l2 = __shfl_xor_sync(0xffffffffu, lo, j), h2 = __shfl_xor_sync(0xffffffffu, hi, j);
            const bool first = !(lane & j);
            const bool lmax = first == (((at + lane) & k) == 0), hmax = first == (((at + lane + 32) & k) == 0);
            lo = (lo < l2) == lmax ? l2 : lo;
            hi = (hi < h2) == hmax ? h2 : hi;
        }
    }
}

// Sorts a[0, n) from the largest down (n <= kList) with the CTA's threads: 64
// numbers a warp in registers, longer steps through shared memory.
__device__ __noinline__ void sort_down(u64* a, int n) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n2 = 64;
    while (n2 < n) n2 *= 2;
    __syncthreads();
    for (int at = warp * 64; at < n2; at += kWarpsN * 64) {
        u64 lo = at + lane < n ? a[at + lane] : 0, hi = at + lane + 32 < n ? a[at + lane + 32] : 0;
        for (int k = 2; k <= 64; k *= 2) warp_steps(lo, hi, at, k, k / 2);
        a[at + lane] = lo;
        a[at + lane + 32] = hi;
    }
    __syncthreads();
    for (int k = 128; k <= n2; k *= 2) {
        for (int j = k / 2; j >= 64; j /= 2) {
            for (int p = threadIdx.x; p < n2 / 2; p += kThreads) {
                const int i = 2 * p - (p & (j - 1));
                const u64 x = a[i], y = a[i + j];
                if ((x < y) == ((i & k) == 0)) {
                    a[i] = y;
                    a[i + j] = x;
                }
            }
            __syncthreads();
        }
        for (int at = warp * 64; at < n2; at += kWarpsN * 64) {
            u64 lo = a[at + lane], hi = a[at + lane + 32];
            warp_steps(lo, hi, at, k, 32);
            a[at + lane] = lo;
            a[at + lane + 32] = hi;
        }
        __syncthreads();
    }
}

__device__ __forceinline__ float list_x(u64 v) { return key_logit(uint32_t(v >> 32)); }
__device__ __forceinline__ uint32_t list_i(u64 v) { return ~uint32_t(v); }

// One CTA's view of its row.  RES: the part lies in shared memory, padded with
// -inf to whole tiles of every warp; else it is read from global memory.
template <bool RES>
struct Row {
    const float* x;            // the part in global memory
    uint32_t base, n;          // its first index and length
    int tiles;                 // tiles of each warp
    unsigned rank, size;
    int phase;

    // f(four logits, index of the first) for each of this lane's quads
    template <typename F>
    __device__ __forceinline__ void quads(F f) const {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        uint32_t e = warp * tiles * kTile + lane * 4;
#pragma unroll 1
        for (int k = 0; k < tiles; ++k, e += kTile) f(quad(e), base + e);
    }
    // f(logit, index) for each of this lane's logits
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        quads([&](float4 v, uint32_t i) { f(v.x, i), f(v.y, i + 1), f(v.z, i + 2), f(v.w, i + 3); });
    }
    __device__ __forceinline__ float4 quad(uint32_t e) const {
        if constexpr (RES) return *reinterpret_cast<const float4*>(sh_x() + e);
        return make_float4(at(e), at(e + 1), at(e + 2), at(e + 3));
    }
    __device__ __forceinline__ float at(uint32_t e) const {
        return e < n ? clean(x[e]) : -INFINITY;
    }

    // Lists those of a lane's four tokens that `in` names (all lanes call);
    // whether the warp had any.
    __device__ __forceinline__ bool list(const bool (&in)[4], float4 v, uint32_t i) {
        if (!__any_sync(0xffffffffu, in[0] | in[1] | in[2] | in[3])) return false;
        const float x[4] = {v.x, v.y, v.z, v.w};
        Shared& s = sh();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (in[j]) {
                const uint32_t at = atomicAdd(&s.listed, 1u);
                if (at < kList) s.mine[at] = (u64(logit_key(x[j])) << 32) | uint32_t(~(i + j));
            }
        return true;
    }
    // Behind the exchange (of e2: tokens listed) that ended the listing: the
    // parts as one list of n <= kList tokens, got(place, token) for each.  The
    // CTAs keep their parts until the next barrier.
    template <typename G>
    __device__ __forceinline__ void gather(uint32_t n, G got) {
        Shared& s = sh();
        cg::cluster_group cl = cg::this_cluster();
        for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
            uint32_t at = i;
            unsigned r = 0;
            for (; r + 1 < size && at >= s.slot[phase ^ 1][r].e2; ++r) at -= s.slot[phase ^ 1][r].e2;
            const u64 t = cl.map_shared_rank(s.mine, r)[at];
            s.list[i] = t;
            got(i, t);
        }
        __syncthreads();
    }

    // The index whose running sum of w(x, index) in index order first reaches
    // e, where `before` is the sum of the CTAs before this one and s.warp[].a
    // the sums of its warps (1 <= e <= the whole sum).
    template <typename W>
    __device__ __forceinline__ uint32_t pick(u64 e, u64 before, W w) {
        Shared& s = sh();
        u64 run = before;
        int k = 0;       // the warp whose tokens hold it, if one of this CTA's does
        while (k < kWarpsN && run + s.warp[k].a < e) run += s.warp[k++].a;
        if (run < e && k < kWarpsN) {
            const uint32_t of_warp = uint32_t(tiles) * kTile;
            // that warp's tokens, over the whole CTA
            for (uint32_t at0 = 0; at0 < of_warp; at0 += kThreads * 4) {
                const uint32_t at = at0 + threadIdx.x * 4, el = k * of_warp + at, i = base + el;
                u64 w0 = 0, w1 = 0, w2 = 0, w3 = 0, sum;
                if (at < of_warp) {
                    const float4 v = quad(el);
                    w0 = w(v.x, i), w1 = w0 + w(v.y, i + 1), w2 = w1 + w(v.z, i + 2), w3 = w2 + w(v.w, i + 3);
                }
                const u64 lo = run + block_scan(w3, &sum);
                if (run + sum < e) {
                    run += sum;
                    continue;
                }
                if (lo < e && lo + w3 >= e) {
                    const uint32_t hit = lo + w0 >= e ? 0 : lo + w1 >= e ? 1 : lo + w2 >= e ? 2 : 3;
                    cg::cluster_group cl = cg::this_cluster();
                    for (unsigned r = 0; r < size; ++r) *cl.map_shared_rank(&s.found, r) = i + hit;
                }
                break;
            }
        }
        cluster_sync(size);
        return s.found;
    }

    // The cut by exact sums of f(x, index) over what reaches a bound, bit by
    // bit: the largest bound whose sum is at least `need`.  e_of(sum above, one
    // tie's f) says how many of the tokens equal to the bound are taken.
    template <typename F, typename E>
    __device__ __noinline__ Cut search(uint32_t top, F f, u64 need, E e_of) {
        uint32_t t = 0;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t cand = t | (1u << bit);
            if (cand > top) continue;
            Slot v;
            each([&](float x, uint32_t i) {
                if (logit_key(x) >= cand) v.a += f(x, i);
            });
            if (exchange<kA>(v, phase).a >= need) t = cand;
        }
        if (t == 0) t = 1;
        Slot v;
        u64 tie = 0;
        each([&](float x, uint32_t i) {
            const uint32_t k = logit_key(x);
            const u64 w = k >= t ? f(x, i) : 0;
            if (k > t) v.a += w;
            if (k == t && w) {
                tie = w;
                ++v.e;
            }
        });
        v.g = tie * v.e;       // ties weigh the same
        const Slot all = exchange<kA | kG | kE>(v, phase);
        const float x = key_logit(t);
        if (all.e == 0) return {x, 0xffffffffu};
        const u64 e = min(max(e_of(all.a, all.g / all.e), u64(1)), u64(all.e));
        const auto is_tie = [&](float y, uint32_t i) { return u64(y == x && f(y, i)); };
        Slot ties;
        each([&](float y, uint32_t i) { ties.a += is_tie(y, i); });
        u64 before;
        exchange<kA>(ties, phase, &before);
        return {x, pick(e, before, is_tie)};
    }
};

// A cut by histogram, exact pass and sorted list.  f(x, i): what is summed (0:
// not among the tokens); rough(x, i): f for the histogram, whose sum from the
// top reaches rough_need in the cut's bin; need_of(sum of all f): the sum that
// the cut reaches; scale: bins a unit of M - x.  False: not found this way.
// True: s.cut_x and s.cut_i hold the cut behind the next cluster barrier, and
// kept and kept_n are a thread's part of the sum and number of the tokens that
// it keeps (summed over a warp: those of its own part of the row).
template <bool RES, typename F, typename R, typename P>
__device__ __forceinline__ bool cut_by_bins(Row<RES>& row, const Weights& w, float scale, F f, R rough, u64 rough_need,
                                            P need_of, u64* kept, uint32_t* kept_n) {
    cg::cluster_group cl = cg::this_cluster();
    Shared& s = sh();
    const int tid = threadIdx.x;
    for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
    if (tid == 0) s.found = kBins;
    __syncthreads();
    // (the last bin holds all that lies lower: summed in a register)
    uint32_t rest = 0;
    row.each([&](float x, uint32_t i) {
        const uint32_t r = rough(x, i);
        const int b = w.bin(x, scale);
        if (b == kBins - 1) rest += r;
        else if (r) atomicAdd(&s.hist[b], r);
    });
    rest = __reduce_add_sync(0xffffffffu, rest);
    if ((tid & 31) == 0 && rest) atomicAdd(&s.hist[kBins - 1], rest);
    cluster_sync(row.size);
    // every CTA sums the cluster's bins and finds the one that holds the cut
    static_assert(kBins == 2 * kThreads, "two bins a thread");
    u64 b0 = 0, b1 = 0, all_bins;
#pragma unroll 8
    for (unsigned r = 0; r < row.size; ++r) {
        const uint2 h = reinterpret_cast<const uint2*>(cl.map_shared_rank(s.hist, r))[tid];
        b0 += h.x;
        b1 += h.y;
    }
    const u64 before = block_scan(b0 + b1, &all_bins);
    if (before < rough_need && before + b0 + b1 >= rough_need) s.found = 2 * tid + (before + b0 < rough_need);
    if (tid == 0) s.listed = 0;
    __syncthreads();
    int B = int(s.found);
    // (nobody reads another CTA's bins, or this CTA's `found`, behind the next barrier)
    for (int attempt = 0; attempt < 3; ++attempt) {
        Slot v;
        const float y0 = float(B), y1 = B < kBins - 1 ? float(B + 1) : INFINITY;
        row.quads([&](float4 x4, uint32_t i) {
            const float x[4] = {x4.x, x4.y, x4.z, x4.w};
            bool in[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u64 fx = f(x[j], i + j);
                const float y = w.depth(x[j], scale);
                v.a += fx;
                const bool up = y < y0 && fx != 0;
                v.b += up ? fx : 0;
                v.e += up;
                in[j] = !(y < y0) && y <= y1 && fx != 0 && (y < y1 || B == kBins - 1);
            }
            if (row.list(in, x4, i)) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (in[j]) {
                        v.g += f(x[j], i + j);
                        ++v.e2;
                    }
            }
        });
        const Slot all = exchange<kA | kB | kG | kE2>(v, row.phase);
        const u64 need = need_of(all.a);
        const bool deep = all.b >= need;
        if (deep || all.b + all.g < need) {      // the histogram's rounding named a neighbour
            __syncthreads();
            if (tid == 0) {
                s.listed = 0;
                s.found = deep ? 0 : kBins - 1;
            }
            __syncthreads();
            // the nearest bin on the side of the cut that holds anything
            const uint32_t at[2] = {2u * tid, 2u * tid + 1};
            const u64 holds[2] = {b0, b1};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (holds[j] && deep && int(at[j]) < B) atomicMax(&s.found, at[j]);
                if (holds[j] && !deep && int(at[j]) > B) atomicMin(&s.found, at[j]);
            }
            __syncthreads();
            B = int(s.found);
            continue;
        }
        if (all.e2 > kList) return false;
        const uint32_t n = all.e2;
        const int lane = tid & 31, warp = tid >> 5;
        const uint32_t of_warp = uint32_t(row.tiles) * kTile;
        if (n <= (row.size == 1 ? kPairsOne : kPairs)) {
            // every CTA takes the whole list; a token of its own is kept if what
            // goes before it falls short, and is the cut if it makes that up
            u64* const fs = reinterpret_cast<u64*>(s.hist);
            if (tid < kWarpsN) s.scan[tid] = 0;
            row.gather(n, [&](uint32_t i, u64 t) { fs[i] = f(list_x(t), list_i(t)); });
            // eight lanes a token
            const uint32_t own = s.listed, sub = lane & 7;
            for (uint32_t j0 = 0; j0 < own; j0 += kThreads / 8) {
                const uint32_t j = j0 + tid / 8;
                const u64 t = j < own ? s.mine[j] : ~u64(0);
                u64 sum = 0;
#pragma unroll 4
                for (uint32_t i = sub; i < n; i += 8) sum += s.list[i] > t ? fs[i] : 0;
#pragma unroll
                for (int d = 4; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                sum += all.b;
                if (sub == 0 && j < own && sum < need) {
                    const float x = list_x(t);
                    const uint32_t at = list_i(t);
                    const u64 fx = f(x, at);
                    atomicAdd(&s.scan[(at - row.base) / of_warp], fx);
                    ++v.e;
                    if (sum + fx >= need)
                        for (unsigned r = 0; r < row.size; ++r) {
                            *cl.map_shared_rank(&s.cut_x, r) = x;
                            *cl.map_shared_rank(&s.cut_i, r) = at;
                        }
                }
            }
            __syncthreads();
            if (lane == 0) v.b += s.scan[warp];
        } else {
            if (row.rank == 0) {
                row.gather(n, [](uint32_t, u64) {});
                sort_down(s.list, int(n));
                // the first place whose sum, itself included, is enough
                const int per = (n + kThreads - 1) / kThreads, at0 = tid * per, at1 = min(at0 + per, int(n));
                u64 part = 0, sum;
                for (int j = at0; j < at1; ++j) part += f(list_x(s.list[j]), list_i(s.list[j]));
                u64 run = all.b + block_scan(part, &sum);
                for (int j = at0; j < at1; ++j) {
                    const u64 fx = f(list_x(s.list[j]), list_i(s.list[j]));
                    if (run < need && run + fx >= need) {
                        for (unsigned r = 0; r < row.size; ++r) {
                            *cl.map_shared_rank(&s.cut_x, r) = list_x(s.list[j]);
                            *cl.map_shared_rank(&s.cut_i, r) = list_i(s.list[j]);
                        }
                    }
                    run += fx;
                }
            }
            cluster_sync(row.size);
            const Cut cut{s.cut_x, s.cut_i};
            const uint32_t first = row.base + warp * of_warp;
            for (uint32_t j = lane; j < s.listed; j += 32) {
                const float x = list_x(s.mine[j]);
                const uint32_t i = list_i(s.mine[j]);
                if (i - first < of_warp && cut.has(x, i)) {
                    v.b += f(x, i);
                    ++v.e;
                }
            }
        }
        *kept = v.b;
        *kept_n = v.e;
        return true;
    }
    return false;
}

// What one row is given.
struct Settings {
    float p, u;
    u64 floor_w;     // the smallest weight that min-p keeps
    int k;
};

// The same on at most kShort tokens a, every pair of them compared, four threads
// a token, in place of two sorts (wt: n words of shared memory).
__device__ __noinline__ void draw_from_pairs(const Weights& w, const Settings& g, const u64* a, u64* wt, int n,
                                             uint32_t* tok, u64* mass, uint32_t* kept) {
    Shared& s = sh();
    const int i = threadIdx.x >> 2, sub = threadIdx.x & 3;
    const bool has = i < n, writes = has && sub == 0;
    const u64 t = has ? a[i] : 0, wi = has ? w(list_x(t)) : 0;
    if (writes) wt[i] = wi;
    __syncthreads();
    // what goes before it: the k-th says the k's mass, and who falls short of p of that stays
    u64 above = 0;
    int rank = 0;
    for (int j = sub; j < n; j += 4) {
        const bool more = a[j] > t;
        above += more ? wt[j] : 0;
        rank += more;
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        above += __shfl_xor_sync(0xffffffffu, above, d);
        rank += __shfl_xor_sync(0xffffffffu, rank, d);
    }
    if (writes && rank == 0) s.found = list_i(t);
    if (writes && rank == g.k - 1) s.scan[0] = above + wi;
    __syncthreads();
    const u64 need = g.p < 1.0f ? share(g.p, s.scan[0], true) : ~u64(0);
    const bool in = has && rank < g.k && above < need && (rank == 0 || wi >= g.floor_w);
    // (a weight is at most 2^61 here; bit 62: not 0 in binary32)
    const u64 positive = w.rough(list_x(t)) > 0.0f ? u64(1) << 62 : 0;
    if (writes) wt[i] = in ? wi | positive | u64(1) << 63 : 0;
    __syncthreads();
    const auto counts = [&](u64 v) { return g.u > 0.0f ? v & ((u64(1) << 62) - 1) : v >> 62 & 1; };
    u64 sum = 0, run = 0;
    uint32_t cnt = 0;
    for (int j = sub; j < n; j += 4) {
        const u64 v = wt[j];
        sum += v & ((u64(1) << 62) - 1);
        cnt += uint32_t(v >> 63);
        run += list_i(a[j]) < list_i(t) ? counts(v) : 0;
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
        run += __shfl_xor_sync(0xffffffffu, run, d);
        cnt += __shfl_xor_sync(0xffffffffu, cnt, d);
    }
    // the first sum above u * S; u = 0: the first whose weight is not 0
    const u64 e = g.u >= 1.0f ? sum : g.u > 0.0f ? share(g.u, sum, false) + 1 : 1;
    if (writes && in && run < e && run + counts(wi | positive) >= e) s.found = list_i(t);
    __syncthreads();
    *tok = s.found;
    *mass = sum;
    *kept = cnt;
}

// The first CTA alone, on a list of n tokens that holds the row's k largest
// (k <= n): the filters and the draw.  scale: bins over the list's logits.
__device__ __noinline__ void draw_from_list(const Weights& w, const Settings& g, int n, float scale, uint32_t* tok,
                                            u64* mass, uint32_t* kept) {
    Shared& s = sh();
    const int tid = threadIdx.x, k = g.k;
    u64* a = s.list;       // the tokens
    u64* wt = s.mine;      // their weights
    u64 sum;
    if (n > kShort) {
        // those in the bins up to the one that holds the k-th
        for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
        if (tid == 0) s.listed = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) atomicAdd(&s.hist[w.bin(list_x(a[i]), scale)], 1u);
        __syncthreads();
        const uint32_t b0 = s.hist[2 * tid], b1 = s.hist[2 * tid + 1];
        const u64 before = block_scan(b0 + b1, &sum);
        if (before < u64(k) && before + b0 + b1 >= u64(k)) s.found = 2 * tid + (before + b0 < u64(k));
        __syncthreads();
        const int B = int(s.found);
        for (int i = tid; i < n; i += kThreads)
            if (w.bin(list_x(a[i]), scale) <= B) s.mine[atomicAdd(&s.listed, 1u)] = a[i];
        __syncthreads();
        n = int(s.listed);
        a = s.mine;
        wt = s.list;
    }
    if (n <= kShort) return draw_from_pairs(w, g, a, wt, n, tok, mass, kept);
    sort_down(a, n);
    const int per = (k + kThreads - 1) / kThreads, at0 = tid * per, at1 = min(at0 + per, k);
    u64 part = 0;
    for (int j = at0; j < at1; ++j) {
        const u64 x = w(list_x(a[j]));
        wt[j] = x;
        part += x;
    }
    u64 run = block_scan(part, &sum);
    if (tid == 0) s.found = uint32_t(k);
    __syncthreads();
    if (g.p < 1.0f) {
        // the shortest beginning that holds p of the mass
        const u64 need = share(g.p, sum, true);
        for (int j = at0; j < at1; ++j) {
            if (run < need && run + wt[j] >= need) s.found = uint32_t(j + 1);
            run += wt[j];
        }
    }
    __syncthreads();
    n = int(s.found);
    // what is left, in index order: (~index, weight not 0 in binary32, place); 0
    // for what min-p drops
    part = 0;
    uint32_t cnt = 0;
    for (int j = at0; j < at1; ++j) {
        const bool in = j < n && (j == 0 || wt[j] >= g.floor_w);
        if (in) {
            part += wt[j];
            ++cnt;
        }
        const uint32_t positive = w.rough(list_x(a[j])) > 0.0f ? 0x10000u : 0u;
        a[j] = in ? (a[j] << 32) | positive | uint32_t(j) : 0;
    }
    block_scan(part, &sum);
    u64 cnt_all;
    block_scan(cnt, &cnt_all);
    sort_down(a, n);
    const int at2 = min(at0 + per, int(cnt_all));
    // the first sum above u * S; u = 0: the first whose weight is not 0
    const u64 e = g.u >= 1.0f ? sum : g.u > 0.0f ? share(g.u, sum, false) + 1 : 1;
    const auto counts = [&](u64 v) { return g.u > 0.0f ? wt[v & 0xffffu] : v >> 16 & 1; };
    part = 0;
    for (int j = at0; j < at2; ++j) part += counts(a[j]);
    u64 whole;
    run = block_scan(part, &whole);
    for (int j = at0; j < at2; ++j) {
        const u64 x = counts(a[j]);
        if (run < e && run + x >= e) s.found = uint32_t(j);
        run += x;
    }
    __syncthreads();
    *tok = ~uint32_t(a[s.found] >> 32);
    *mass = sum;
    *kept = uint32_t(cnt_all);
}

template <bool RES>
__global__ void __launch_bounds__(kThreads, RES ? 2 : 1) sample_kernel(const SampleArgs a, int part, int shift, int* err) {
    Shared& s = sh();
    cg::cluster_group cl = cg::this_cluster();
    const unsigned rank = cl.block_rank(), size = cl.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t m = blockIdx.x / size;
    if (tid < 64) s.pow2[tid] = make_uint2(kPow2[tid], __float_as_uint(float(kPow2[tid])));
    if (tid == 0) s.listed = 0;
    pdl_wait();
    pdl_launch_dependents();

    const float T = a.temperature ? a.temperature[m] : 1.0f;
    const int32_t k = a.top_k ? a.top_k[m] : 0;
    const float p = a.top_p ? a.top_p[m] : 1.0f, mp = a.min_p ? a.min_p[m] : 0.0f;
    const float u = a.u[m];
    const auto give = [&](int64_t tok, float prob, int32_t kept) {
        a.tok[m] = int32_t(tok);
        if (a.prob) a.prob[m] = prob;
        if (a.kept) a.kept[m] = kept;
    };
    const bool writes = rank == 0 && tid == 0;
    if (!(T >= 0.0f) || isnan(p) || isnan(mp)) {      // the whole cluster alike
        if (writes) {
            atomicExch(err, Q8_DEVERR_PARAM);
            give(0, 0.0f, 0);
        }
        return;
    }

    cluster_arrive(size);    // (waited for below: every CTA has begun before another writes to it)

    // the part: [base, base + n) of the row
    const uint32_t base = rank * uint32_t(part), N = uint32_t(a.N);
    const uint32_t n = base < N ? min(uint32_t(part), N - base) : 0;
    const float* gx = a.x + m * a.ldx + base;
    Row<RES> row{gx, base, n, part / kPart, rank, size, 0};
    const uint32_t of_warp = uint32_t(row.tiles) * kTile;      // tokens of a warp

    // (Ordinary loads, here and where rows are read again: this grid may have begun while
    // the one that writes the logits ran, and the read-only path is for what nobody writes
    // while a grid runs.)
    // Seen once while they are loaded: the largest and the smallest that can be
    // drawn, how many can, and for the nucleus of the whole row the sum of their
    // weights (a lane's in units of its own largest).
    const bool early = p < 1.0f && k <= 0 && T <= 1e30f;       // (T: so that no difference overflows but to weight 0)
    const float early_c = __fdividef(1.44269502f, T);
    float best = -INFINITY, least = INFINITY, est = 0.0f;
    uint32_t some = 0;
    const auto look = [&](float4 q, uint32_t) {
        const float x[4] = {q.x, q.y, q.z, q.w};
        const float now = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), best);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (x[j] > -INFINITY) {
                least = fminf(least, x[j]);
                ++some;
            }
        if (early) {
            if (now > best) est = best > -INFINITY ? est * exp2_rough((best - now) * early_c) : 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (x[j] > -INFINITY) est += exp2_rough((x[j] - now) * early_c);
        }
        best = now;
    };
    if constexpr (RES) {
        float* x = sh_x();
        if ((reinterpret_cast<uintptr_t>(gx) & 15) == 0) {
            // each warp its own tiles
            const int end = (tid >> 5) * int(of_warp) + int(of_warp);
#pragma unroll 8
            for (int e = end - int(of_warp) + lane * 4; e < end; e += kTile) {
                float4 v;
                if (e + 3 < int(n)) {
                    v = *reinterpret_cast<const float4*>(gx + e);
                } else {
                    v.x = e < int(n) ? gx[e] : -INFINITY;
                    v.y = e + 1 < int(n) ? gx[e + 1] : -INFINITY;
                    v.z = e + 2 < int(n) ? gx[e + 2] : -INFINITY;
                    v.w = -INFINITY;
                }
                v = make_float4(clean(v.x), clean(v.y), clean(v.z), clean(v.w));
                *reinterpret_cast<float4*>(x + e) = v;
                look(v, 0);
            }
            __syncthreads();
        } else {
            // a row that begins off a 16-byte boundary: whole words, stored a float at
            // a time (behind the first row only, so the word before it is the row before's)
            const int off = int(reinterpret_cast<uintptr_t>(gx) >> 2 & 3);
#pragma unroll 8
            for (int e = tid * 4 - off; e < part; e += kThreads * 4) {
                float f[4];
                if (e + 3 < int(n)) {
                    const float4 v = *reinterpret_cast<const float4*>(gx + e);
                    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[j] = e + j < int(n) && e + j >= 0 ? gx[e + j] : -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (e + j >= 0 && e + j < part) x[e + j] = clean(f[j]);
            }
            __syncthreads();
            row.quads(look);
        }
    } else {
        row.quads(look);
    }
    Slot v;
    v.c = logit_key(best);
    v.d = least < INFINITY ? logit_key(least) - 1 : 0xffffffffu;
    v.e = some;
    v.s = est;
    // with top-k: a logit that at least k reach, from the lanes' maxima: the
    // q-th largest of each full warp, the smallest of those over the warps
    uint32_t reach = 0xffffffffu;
    const uint32_t full = N / of_warp;      // warps whose logits all exist
    const uint32_t q = k > 0 && full ? (uint32_t(k) + full - 1) / full : 0;
    if (q >= 1 && q <= 32 && base / of_warp + (tid >> 5) < full) {
        uint32_t key = v.c;
        for (uint32_t j = 1; j < q; ++j) {
            const uint32_t most = __reduce_max_sync(0xffffffffu, key);
            const unsigned who = __ballot_sync(0xffffffffu, key == most);
            if (lane == __ffs(who) - 1) key = 0;
        }
        reach = __reduce_max_sync(0xffffffffu, key);
    }
    v.c2 = ~reach;
    cluster_wait(size);
    const Slot all = exchange<kE | kC | kC2 | kD | kS>(v, row.phase, nullptr, early_c);
    const uint32_t top = all.c, low = all.d + 1;
    reach = ~all.c2;
    if (top == 0) {
        if (writes) give(0, 0.0f, 0);
        return;
    }
    const float M = key_logit(top);
    if (T < 0x1p-60f || p <= 0.0f || mp > 1.0f) {      // the first alone
        v = Slot();
        row.each([&](float x, uint32_t i) {
            if (x == M) v.d = min(v.d, i);
        });
        const uint32_t first = exchange<kD>(v, row.phase).d;
        if (writes) give(first, 1.0f, 1);
        return;
    }

    Weights w;
    w.pre = fmaxf(fabsf(M), fabsf(key_logit(low))) > 1e38f ? 0.5f : 1.0f;
    w.M = M * w.pre;
    // log2(e) / T in two floats, from log2(e) in two
    const float c = __fdiv_rn(1.44269502f, T);
    const float c2 = isinf(T) ? 0.0f : __fdiv_rn(fmaf(-c, T, 1.44269502f) + 1.925963e-8f, T);
    w.ch = c / w.pre;
    w.cl = c2 / w.pre;
    w.shift = shift;
    const u64 one = u64(1) << shift;
    Settings set{p, u, mp > 0.0f ? share(mp, one, true) : 0, k};
    const auto finish = [&](uint32_t tok, u64 S, uint32_t kept) {
        // the weight's mantissa over the sum's 48 leading bits, both in two floats
        uint32_t mant;
        int e;
        w.parts(clean(a.x[m * a.ldx + tok]), mant, e);
        const int z = __clzll(S);
        const u64 top48 = S << z >> 16;                                // S = top48 * 2^(16 - z)
        const float nh = float(mant & 0xffffff00u), nl = float(mant & 255u);
        const float dh = float(uint32_t(top48 >> 24)) * 16777216.0f, dl = float(uint32_t(top48) & 0xffffffu);
        const float q = __fdiv_rn(nh, dh), r = fmaf(-q, dh, nh) + fmaf(-q, dl, nl);
        const int by = e - 31 + shift - 16 + z;                        // mant * 2^(e - 31 + shift) / S
        const float prob = q + __fdiv_rn(r, dh);                       // (of 2^-17 to 2^-14)
        give(tok, ldexpf(prob, by), int32_t(kept));
    };
    const float span = w.M - key_logit(low) * w.pre;      // of all logits (0: all equal)
    const auto bins_over = [&](float d) {
        d = fminf(d, span);
        return d > 0.0f && d < INFINITY ? fminf(float(kBins) / d, FLT_MAX) : 0.0f;
    };
    const bool by_k = k > 0 && uint32_t(k) < all.e;
    const bool reached = reach > 0 && reach <= top;
    // a row of which few can be drawn, as a grammar's mask leaves, is a list whole (60
    // of 128256, top-p: 1 row 25 us without, 13 so, 64 rows 71 and 31; not short rows
    // without top-p: 153 rows of 120 8 us, 12 so)
    const bool few = all.e <= uint32_t(kShort) && N > 1 && (p < 1.0f || N > uint32_t(kPart));
    const float bound = few ? -FLT_MAX : reached ? key_logit(reach) : M;
    const float k_scale = reached && bound < M ? bins_over((w.M - bound * w.pre) * 1.001f) : bins_over(span);
    if (few || (by_k && k <= kList && reached)) {
        // every token that reaches `bound`, at least k of them
        if (!by_k) set.k = int(all.e);
        v = Slot();
        row.quads([&](float4 x, uint32_t i) {
            const bool in[4] = {x.x >= bound, x.y >= bound, x.z >= bound, x.w >= bound};
            v.e2 += in[0] + in[1] + in[2] + in[3];
            row.list(in, x, i);
        });
        const uint32_t listed = exchange<kE2>(v, row.phase).e2;
        if (listed <= kList) {
            if (rank == 0) {
                row.gather(listed, [](uint32_t, u64) {});
                uint32_t tok, kept;
                u64 S;
                draw_from_list(w, set, int(listed), k_scale, &tok, &S, &kept);
                if (writes) finish(tok, S, kept);
            }
            cluster_sync(size);      // (the first CTA has read the others' parts of the list)
            return;
        }
    }

    Cut cut{-FLT_MAX, 0xffffffffu};      // everything above -inf
    const auto cut_found = [&] {
        cluster_sync(size);
        cut = {s.cut_x, s.cut_i};
    };
    u64 kept = 0;
    uint32_t kept_n = 0;
    if (by_k) {
        const auto counted = [&](float x, uint32_t) { return uint32_t(x > -INFINITY); };
        if (cut_by_bins(row, w, k_scale, counted, counted, u64(k), [&](u64) { return u64(k); }, &kept, &kept_n))
            cut_found();
        else
            cut = row.search(top, counted, u64(k), [&](u64 sum, u64) { return u64(k) - sum; });
    }
    bool summed = false;                 // kept, kept_n are the nucleus's
    if (p < 1.0f) {
        // bins hold masses in units of 2^-31 of the sum, by its estimate
        const Cut before = cut;
        float S = all.s;                 // at least 1: M itself
        if (!early) {
            est = 0.0f;
            row.each([&](float x, uint32_t i) {
                if (before.has(x, i)) est += w.rough(x);
            });
            v = Slot();
            v.a = u64(est * 16777216.0f);
            S = float(exchange<kA>(v, row.phase).a) * 0x1p-24f;
        }
        const float unit = 2147483648.0f / S;
        // tokens of less than (1 - p) S / N hold less than the share 1 - p
        // together, so the nucleus ends above them: the bins stop there
        const float lowest = (1.0f - p) * S / float(all.e) * 0.99f;
        const float scale = bins_over(-log2f(lowest) / w.ch);
        // (the weight of -inf is 0: without a cut before, every logit may be asked)
        const auto f = [&](float x, uint32_t i) {
            const u64 wx = w(x);
            return !by_k || before.has(x, i) ? wx : 0;
        };
        const auto rough = [&](float x, uint32_t i) {
            const uint32_t r = __float2uint_rn(w.rough(x) * unit);
            return !by_k || before.has(x, i) ? r : 0u;
        };
        u64 need = 0;
        const auto need_of = [&](u64 sum) { return need = share(p, sum, true); };
        summed = cut_by_bins(row, w, scale, f, rough, u64(share(p, u64(1) << 31, true)), need_of, &kept, &kept_n);
        if (!summed)
            // (`need` is of the exact sum by now) the fewest ties that reach the mass
            cut = row.search(top, f, need, [&](u64 sum, u64 tie) { return (need - sum + tie - 1) / tie; });
    }

    // what is kept: its mass and number, and its lowest index
    const u64 floor_w = set.floor_w;
    const auto kept_w = [&](float x, uint32_t i) -> u64 {
        const u64 wx = w(x);
        return cut.has(x, i) && wx >= floor_w ? wx : 0;
    };
    v = Slot();
    const bool whole = summed && floor_w == 0 && u > 0.0f;
    if (whole) {
        v.a = kept;
        v.e = kept_n;
    } else {
        if (summed) cut_found();
        row.each([&](float x, uint32_t i) {
            const u64 wx = w(x);
            const bool in = cut.has(x, i) && wx >= floor_w;
            v.a += in ? wx : 0;
            v.e += in;
            v.d = in && w.rough(x) > 0.0f ? min(v.d, i) : v.d;
        });
    }
    u64 before;
    const Slot fin = exchange<kA | kE | kD>(v, row.phase, &before);
    if (whole) cut = {s.cut_x, s.cut_i};
    uint32_t tok = fin.d;
    if (u > 0.0f) {
        // the first sum above u * S
        const u64 e = u >= 1.0f ? fin.a : share(u, fin.a, false) + 1;
        tok = row.pick(e, before, kept_w);
    }
    if (writes) finish(tok, fin.a, fin.e);
    cluster_sync(size);      // nobody leaves while another may still write here
}

template <bool RES>
cudaError_t launch_sample_kernel(const SampleArgs& a, int size, int part, int shift, const LaunchCtx& ctx) {
    static std::atomic<bool> ready[kMaxDevices];
    const cudaError_t e =
        set_smem_once(sample_kernel<RES>, sizeof(Shared) + (RES ? size_t(kMaxPart) * 4 : 0), ctx.dev, ready);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attrs[2];
    cfg.gridDim = dim3(unsigned(a.rows * size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared) + (RES ? size_t(part) * 4 : 0);
    cfg.stream = ctx.stream;
    cfg.numAttrs = pdl_attrs(ctx, attrs);
    attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attrs[cfg.numAttrs].val.clusterDim.x = unsigned(size);
    attrs[cfg.numAttrs].val.clusterDim.y = 1;
    attrs[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
    cfg.attrs = attrs;
    return cudaLaunchKernelEx(&cfg, sample_kernel<RES>, a, part, shift, ctx.dev_err);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, const LaunchCtx& ctx) {
    int bits = 0;
    while ((int64_t(1) << bits) < a.N) ++bits;
    const auto part_of = [&](int size) {
        const int64_t tiles = (a.N + int64_t(size) * kPart - 1) / (int64_t(size) * kPart);
        return int(tiles * kPart);
    };
    // CTAs a row: parts of which an SM holds two where 8 CTAs reach that (248 rows
    // of 33098: 2 of 18 K 80 us, 4 of 10 K 101 us); more, down to parts of one tile
    // a warp, while the GPU has SMs to spare.  Past 8 parts of 18 K an SM holds one
    // CTA (64 rows, top-p: of 147456 92 us, of 147457 164), past 8 of 46 K none's part
    // fits and every pass reads L2 (one row of 2^20, every filter: 58 us)
    int size = 1;
    while (size < kMaxCluster && (part_of(size) > kPairPart ||
                                  (a.rows * size * 2 <= ctx.num_sms && part_of(size) > kPart)))
        size *= 2;
    const int part = part_of(size);
    if (part <= kMaxPart) return launch_sample_kernel<true>(a, size, part, 62 - bits, ctx);
    return launch_sample_kernel<false>(a, size, part, 62 - bits, ctx);
}

}  // namespace q8
