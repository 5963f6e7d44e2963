// sample.cu -- sampling of one token a row from the head's logits.
//
// Mathematics.  A token's weight is an integer, 2^((x - M) log2(e) / T) in
// units of 2^-shift rounded down, so every sum is exact and independent of its
// order: what is drawn depends on nothing but the row and its settings.  The
// filters cut the tokens in order of x (ties: the lowest index first), so what
// they leave is "x > t, or x = t and index <= last".
//
// Layout.  A cluster of 1 to 8 CTAs takes a row, each an equal part of it in
// index order, read once into shared memory (rows past 8 x 48 K logits are read
// again from L2 instead).  The CTAs hand sums to one another through
// distributed shared memory: one cluster barrier an exchange.
//
// A cut (the k-th largest; the end of the nucleus) is found without sorting
// the row: a histogram of 1024 bins linear in x between M and a bound below the
// cut (counts, or masses to 2^-22) names the bin that holds it; an exact pass
// sums what lies above that bin and lists the bin's tokens in the first CTA,
// which sorts them (some hundreds) and finds the cut's place.  Where the list
// is too long (thousands of equal logits) or the histogram's rounding named a
// neighbour, a binary search over the 32 bits of the ordered logits finds the
// cut instead, with exact sums at each step.
//
// What bounds it.  One row: latency (about ten exchanges).  A batch: the exact
// weights, about 30 instructions each against 4 bytes read.
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
constexpr int kMaxPart = 48 * 1024;         // logits of a part held in shared memory
constexpr int kBins = 1024, kList = 2048, kMaxCluster = 8;
constexpr float kOctaves = 48.0f;           // below 2^-48 of the largest a nucleus never ends
typedef unsigned long long u64;

// What the CTAs of a cluster exchange: a slot a CTA, two sets used in turn, so
// that a slot is written again only after a barrier behind its last reader.
struct Slot {
    u64 a, b, g;
    uint32_t c, d;
};

struct Shared {
    Slot slot[2][kMaxCluster];
    u64 warp_a[kWarpsN], warp_b[kWarpsN], warp_g[kWarpsN];
    uint32_t warp_c[kWarpsN], warp_d[kWarpsN];
    uint32_t hist[kBins];
    u64 list[kList];
    uint32_t listed[2];                     // in the first CTA: tokens offered to the list, by attempt
    float cut_x;                            // the cut that the first CTA found
    uint32_t cut_i, cut_ok;
    uint32_t found;                         // an index that one CTA found
    uint2 pow2[32];                         // 2^(j/32): in units of 2^-31, and as a float of those
};

// Order of the logits as unsigned integers; 0: NaN or -inf, never drawn.
__device__ __forceinline__ uint32_t logit_key(float x) {
    if (!(x > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// 2^(j/32) in units of 2^-31.
__constant__ uint32_t kPow2[32] = {
    2147483648u, 2194507417u, 2242560872u, 2291666561u, 2341847524u, 2393127307u,
    2445529972u, 2499080105u, 2553802834u, 2609723834u, 2666869345u, 2725266179u,
    2784941738u, 2845924021u, 2908241642u, 2971923842u, 3037000500u, 3103502151u,
    3171459999u, 3240905930u, 3311872529u, 3384393094u, 3458501653u, 3534232978u,
    3611622603u, 3690706840u, 3771522796u, 3854108391u, 3938502376u, 4024744348u,
    4112874773u, 4202935003u};

// Weights of a row.  The exponent y = (x - M) log2(e) / T is carried as an
// unevaluated sum of two floats (the difference by the exact two-term sum, its
// product with a two-term constant), split into J/32 + h with |h| <= 1/64 and
// a little; 2^h - 1 is its Taylor polynomial to degree 4 (remainder 2^-40).
// The largest error is that polynomial's and h's own rounding, 2^-29 of the
// weight; with 2^-30 typical, one draw in 10^7 falls next to a border that
// this moves.
struct Weights {
    float M, pre, ch, cl;   // pre: 1/2 where differences could overflow
    int shift;
    bool inf;               // M is +inf
    const uint2* pow2;

    __device__ __forceinline__ u64 operator()(float x) const {
        if (inf) return x == INFINITY ? u64(1) << shift : 0;
        const float a = x * pre, s = a - M, bb = s - a;
        const float err = (a - (s - bb)) + (-M - bb);
        const float p = __fmul_rn(s, ch);       // (rounded: e is what it lost)
        if (!(p > -float(shift))) return 0;
        float e = fmaf(s, ch, -p);
        e = fmaf(s, cl, e);
        e = fmaf(err, ch, e);
        const float kRound = 393216.0f;                 // 1.5 * 2^18: one step is 1/32
        const float r = p + kRound;
        const int J = __float_as_int(r) - __float_as_int(kRound);
        const float h = (p - (r - kRound)) + e;
        float q = fmaf(h, 0.009618129f, 0.05550411f);   // ln(2)^4/24, ln(2)^3/6, ...
        q = fmaf(h, q, 0.2402265f);
        q = fmaf(h, q, 0.6931472f);
        q *= h;
        const uint2 t = pow2[J & 31];
        const uint32_t m = t.x + uint32_t(__float2int_rn(__uint_as_float(t.y) * q));
        return (u64(m) << 31) >> (62 - shift - (J >> 5));
    }
    // 2^y to about 2^-21, for the histogram
    __device__ __forceinline__ float rough(float x) const {
        if (inf) return x == INFINITY ? 1.0f : 0.0f;
        return exp2f((x * pre - M) * ch);
    }
};

struct Cut {
    float t;         // kept: x > t, or x = t and index <= last
    uint32_t last;
    __device__ __forceinline__ bool has(float x, uint32_t i) const { return x > t || (x == t && i <= last); }
};

// One CTA's view of its row.  RES: the part lies in shared memory, padded with
// -inf to whole tiles of every warp; else it is read from global memory.
template <bool RES>
struct Row {
    Shared& s;
    const float* x;            // the part
    uint32_t base, n;          // its first index and length
    int tiles;                 // tiles of each warp
    unsigned rank, size;
    int phase;

    // f(four logits, index of the first) for each of this lane's quads, in index order a warp
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const uint32_t e0 = warp * tiles * kTile + lane * 4;
#pragma unroll 2
        for (int k = 0; k < tiles; ++k) f(quad(e0 + k * kTile), base + e0 + k * kTile);
    }
    __device__ __forceinline__ float4 quad(uint32_t e) const {
        if constexpr (RES) return *reinterpret_cast<const float4*>(x + e);
        float4 v;
        v.x = at(e), v.y = at(e + 1), v.z = at(e + 2), v.w = at(e + 3);
        return v;
    }
    __device__ __forceinline__ float at(uint32_t e) const {
        if constexpr (RES) return x[e];
        const float v = e < n ? __ldg(x + e) : -INFINITY;
        return v > -INFINITY ? v : -INFINITY;       // NaN too
    }

    // Sums a, b and g, the largest c and the smallest d over the cluster's
    // threads; before (if given) receives the sums of a over the CTAs before this one.
    __device__ __forceinline__ Slot exchange(u64 a, u64 b, u64 g, uint32_t c, uint32_t d, u64* before = nullptr) {
        cg::cluster_group cl = cg::this_cluster();
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int k = 16; k; k >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, k);
            b += __shfl_xor_sync(0xffffffffu, b, k);
            g += __shfl_xor_sync(0xffffffffu, g, k);
        }
        c = __reduce_max_sync(0xffffffffu, c);
        d = __reduce_min_sync(0xffffffffu, d);
        if (lane == 0) {
            s.warp_a[warp] = a;
            s.warp_b[warp] = b;
            s.warp_g[warp] = g;
            s.warp_c[warp] = c;
            s.warp_d[warp] = d;
        }
        __syncthreads();
        Slot(&slots)[kMaxCluster] = s.slot[phase];
        phase ^= 1;
        if (warp == 0) {
            a = lane < kWarpsN ? s.warp_a[lane] : 0;
            b = lane < kWarpsN ? s.warp_b[lane] : 0;
            g = lane < kWarpsN ? s.warp_g[lane] : 0;
            c = __reduce_max_sync(0xffffffffu, lane < kWarpsN ? s.warp_c[lane] : 0u);
            d = __reduce_min_sync(0xffffffffu, lane < kWarpsN ? s.warp_d[lane] : 0xffffffffu);
#pragma unroll
            for (int k = 8; k; k >>= 1) {
                a += __shfl_xor_sync(0xffffffffu, a, k);
                b += __shfl_xor_sync(0xffffffffu, b, k);
                g += __shfl_xor_sync(0xffffffffu, g, k);
            }
            if (lane < size) *cl.map_shared_rank(&slots[rank], lane) = Slot{a, b, g, c, d};
        }
        cl.sync();
        Slot all = slots[0];
        u64 sum = rank > 0 ? slots[0].a : 0;
        for (unsigned r = 1; r < size; ++r) {
            if (r < rank) sum += slots[r].a;
            all.a += slots[r].a;
            all.b += slots[r].b;
            all.g += slots[r].g;
            all.c = max(all.c, slots[r].c);
            all.d = min(all.d, slots[r].d);
        }
        if (before) *before = sum;
        return all;
    }

    // The index whose running sum of w(x, index) in index order first reaches
    // e (1 <= e <= the whole sum, which the caller knows is reached).
    template <typename W>
    __device__ __forceinline__ uint32_t locate(u64 e, W w) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        u64 mine = 0, before;
        each([&](float4 v, uint32_t i) { mine += w(v.x, i) + w(v.y, i + 1) + w(v.z, i + 2) + w(v.w, i + 3); });
        exchange(mine, 0, 0, 0, 0, &before);
        // (warp_a: this CTA's sums by warp, until the next exchange)
        u64 at_warp = before;
        for (int k = 0; k < warp; ++k) at_warp += s.warp_a[k];
        if (at_warp < e && at_warp + s.warp_a[warp] >= e) {
            u64 run = at_warp;
            for (int k = 0; k < tiles; ++k) {
                const uint32_t el = (warp * tiles + k) * kTile + lane * 4, i = base + el;
                const float4 v = quad(el);
                const u64 w0 = w(v.x, i), w1 = w0 + w(v.y, i + 1), w2 = w1 + w(v.z, i + 2), w3 = w2 + w(v.w, i + 3);
                u64 up = w3;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const u64 y = __shfl_up_sync(0xffffffffu, up, d);
                    if (lane >= d) up += y;
                }
                const u64 lo = run + up - w3;
                if (lo < e && run + up >= e) {
                    const uint32_t hit = lo + w0 >= e ? 0 : lo + w1 >= e ? 1 : lo + w2 >= e ? 2 : 3;
                    cg::cluster_group cl = cg::this_cluster();
                    for (unsigned r = 0; r < size; ++r) *cl.map_shared_rank(&s.found, r) = i + hit;
                }
                run += __shfl_sync(0xffffffffu, up, 31);
                if (run >= e) break;
            }
        }
        cg::this_cluster().sync();
        return s.found;
    }

    // The cut by exact sums of f(x, index) over what reaches a bound, bit by
    // bit; goal(sum): whether the sum is enough.  e_of(sum above, one tie's f,
    // ties) says how many of the tokens equal to the bound are taken.
    template <typename F, typename G, typename E>
    __device__ __noinline__ Cut search(uint32_t top, F f, G goal, E e_of) {
        uint32_t t = 0;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t cand = t | (1u << bit);
            if (cand > top) continue;
            u64 sum = 0;
            each([&](float4 v, uint32_t i) {
                if (logit_key(v.x) >= cand) sum += f(v.x, i);
                if (logit_key(v.y) >= cand) sum += f(v.y, i + 1);
                if (logit_key(v.z) >= cand) sum += f(v.z, i + 2);
                if (logit_key(v.w) >= cand) sum += f(v.w, i + 3);
            });
            if (goal(exchange(sum, 0, 0, 0, 0).a)) t = cand;
        }
        if (t == 0) t = 1;
        u64 above = 0, tie = 0;
        uint32_t ties = 0;
        const auto one = [&](float x, uint32_t i) {
            const uint32_t k = logit_key(x);
            const u64 w = k >= t ? f(x, i) : 0;
            if (k > t) above += w;
            if (k == t && f(x, i)) {
                tie = w;
                ++ties;
            }
        };
        each([&](float4 v, uint32_t i) { one(v.x, i), one(v.y, i + 1), one(v.z, i + 2), one(v.w, i + 3); });
        // (ties weigh the same: the sum of their weights by their number)
        const Slot all = exchange(above, ties, u64(ties) * tie, 0, 0);
        const float x = key_logit(t);
        const u64 n = all.b;
        const u64 e = n ? min(max(e_of(all.a, all.g / n, n), u64(1)), n) : 1;
        if (n == 0) return {x, 0xffffffffu};
        const uint32_t last = locate(e, [&](float v, uint32_t i) { return u64(v == x && f(v, i)); });
        return {x, last};
    }
};

// Sorts s.list[0, n) from the largest down (n <= kList) with the CTA's threads.
__device__ __forceinline__ void sort_list(Shared& s, int n) {
    int n2 = 2;
    while (n2 < n) n2 *= 2;
    for (int i = n + threadIdx.x; i < n2; i += kThreads) s.list[i] = 0;
    __syncthreads();
    for (int k = 2; k <= n2; k *= 2)
        for (int j = k / 2; j; j /= 2) {
            for (int p = threadIdx.x; p < n2 / 2; p += kThreads) {
                const int i = 2 * p - (p & (j - 1));
                const u64 a = s.list[i], b = s.list[i + j];
                if ((a < b) == ((i & k) == 0)) {
                    s.list[i] = b;
                    s.list[i + j] = a;
                }
            }
            __syncthreads();
        }
}

// A cut by histogram, exact pass and sorted list.  f(x, i): what is summed (0:
// not among the tokens); rough(x, i): f for the histogram; scale: bins a unit
// of M - x; goal(sum): whether a sum from the top is enough; prep(total): called
// with the exact sum of all f before goal.  False: not found this way.
template <bool RES, typename F, typename R, typename P, typename G>
__device__ __forceinline__ bool cut_by_bins(Row<RES>& row, const Weights& w, float scale, F f, R rough, u64 rough_goal,
                                            P prep, G goal, Cut* cut) {
    cg::cluster_group cl = cg::this_cluster();
    Shared& s = row.s;
    const int tid = threadIdx.x, lane = tid & 31;
    const auto bin = [&](float x) {
        const float y = w.inf ? (x == INFINITY ? 0.0f : float(kBins)) : (w.M - x * w.pre) * scale;
        return y < float(kBins - 1) ? int(y) : kBins - 1;
    };
    for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
    if (tid < 2) s.listed[tid] = 0;
    __syncthreads();
    row.each([&](float4 v, uint32_t i) {
        const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t r = rough(x[j], i + j);
            if (r) atomicAdd(&s.hist[bin(x[j])], r);
        }
    });
    cl.sync();
    // every CTA sums the cluster's bins and finds the one that holds the cut
    constexpr int PER = kBins / kThreads;
    u64 mine[PER], sum = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        mine[j] = 0;
        for (unsigned r = 0; r < row.size; ++r) mine[j] += cl.map_shared_rank(s.hist, r)[tid * PER + j];
        sum += mine[j];
    }
    u64 up = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, up, d);
        if (lane >= d) up += y;
    }
    if (lane == 31) s.warp_a[tid >> 5] = up;
    if (tid == 0) s.found = kBins;
    __syncthreads();
    u64 before = up - sum;
    for (int k = 0; k < tid >> 5; ++k) before += s.warp_a[k];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (before < rough_goal && before + mine[j] >= rough_goal) s.found = tid * PER + j;
        before += mine[j];
    }
    __syncthreads();
    int B = int(s.found);
    // (nobody reads another CTA's bins, or this CTA's `found`, behind the next barrier)
    u64* const list = cl.map_shared_rank(s.list, 0);
    for (int attempt = 0; attempt < 3; ++attempt) {
        uint32_t* const listed = cl.map_shared_rank(&s.listed[attempt & 1], 0);
        u64 total = 0, above = 0, within = 0;
        row.each([&](float4 v, uint32_t i) {
            const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u64 fx = f(x[j], i + j);
                const int b = bin(x[j]);
                const bool in = b == B && fx != 0;
                total += fx;
                if (b < B) above += fx;
                if (in) within += fx;
                const unsigned who = __ballot_sync(0xffffffffu, in);
                if (who) {
                    const int lead = __ffs(who) - 1;
                    uint32_t at = 0;
                    if (lane == lead) at = atomicAdd(listed, uint32_t(__popc(who)));
                    at = __shfl_sync(0xffffffffu, at, lead) + __popc(who & ((1u << lane) - 1));
                    if (in && at < kList) list[at] = (u64(logit_key(x[j])) << 32) | uint32_t(~(i + j));
                }
            }
        });
        const Slot all = row.exchange(total, above, within, 0, 0);
        prep(all.a);
        if (goal(all.b) || !goal(all.b + all.g)) {      // the histogram's rounding named a neighbour
            B += goal(all.b) ? -1 : 1;
            if (tid == 0) s.listed[attempt & 1] = 0;    // (for the attempt after the next)
            continue;
        }
        if (row.rank == 0) {
            const int n = int(s.listed[attempt & 1]);
            if (tid == 0) s.cut_ok = n <= kList;
            if (n <= kList) {
                sort_list(s, n);
                // the first place whose sum, itself included, is enough
                const int per = (n + kThreads - 1) / kThreads;
                u64 part = 0;
                for (int j = 0; j < per; ++j) {
                    const int at = tid * per + j;
                    if (at < n) part += f(key_logit(uint32_t(s.list[at] >> 32)), ~uint32_t(s.list[at]));
                }
                u64 upto = part;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const u64 y = __shfl_up_sync(0xffffffffu, upto, d);
                    if (lane >= d) upto += y;
                }
                if (lane == 31) s.warp_b[tid >> 5] = upto;
                __syncthreads();
                u64 run = all.b + upto - part;
                for (int k = 0; k < tid >> 5; ++k) run += s.warp_b[k];
                for (int j = 0; j < per; ++j) {
                    const int at = tid * per + j;
                    if (at >= n) break;
                    const float x = key_logit(uint32_t(s.list[at] >> 32));
                    const uint32_t i = ~uint32_t(s.list[at]);
                    const u64 fx = f(x, i);
                    if (!goal(run) && goal(run + fx)) {
                        s.cut_x = x;
                        s.cut_i = i;
                    }
                    run += fx;
                }
            }
            __syncthreads();
            if (tid < int(row.size) && tid > 0) {
                *cl.map_shared_rank(&s.cut_x, tid) = s.cut_x;
                *cl.map_shared_rank(&s.cut_i, tid) = s.cut_i;
                *cl.map_shared_rank(&s.cut_ok, tid) = s.cut_ok;
            }
        }
        cl.sync();
        *cut = {s.cut_x, s.cut_i};
        return s.cut_ok != 0;
    }
    return false;
}

template <bool RES>
__global__ void __launch_bounds__(kThreads, RES ? 2 : 1) sample_kernel(const SampleArgs a, int part, int shift, int* err) {
    extern __shared__ __align__(16) float s_x[];
    __shared__ Shared s;
    cg::cluster_group cl = cg::this_cluster();
    const unsigned rank = cl.block_rank(), size = cl.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t m = blockIdx.x / size;
    if (tid < 32) s.pow2[tid] = make_uint2(kPow2[tid], __float_as_uint(float(kPow2[tid])));
    pdl_wait();
    pdl_launch_dependents();

    const float T = a.temperature ? a.temperature[m] : 1.0f;
    const int32_t k = a.top_k ? a.top_k[m] : 0;
    const float p = a.top_p ? a.top_p[m] : 1.0f, mp = a.min_p ? a.min_p[m] : 0.0f;
    const float u = a.u[m];
    const auto give = [&](int64_t tok, float prob, int32_t kept) {
        if (rank == 0 && tid == 0) {
            a.tok[m] = int32_t(tok);
            if (a.prob) a.prob[m] = prob;
            if (a.kept) a.kept[m] = kept;
        }
    };
    if (!(T >= 0.0f) || isnan(p) || isnan(mp)) {      // the whole cluster alike
        if (rank == 0 && tid == 0) atomicExch(err, Q8_DEVERR_PARAM);
        return give(0, 0.0f, 0);
    }

    // the part: [base, base + n) of the row
    const uint32_t base = rank * uint32_t(part), N = uint32_t(a.N);
    const uint32_t n = base < N ? min(uint32_t(part), N - base) : 0;
    const float* gx = a.x + m * a.ldx + base;
    Row<RES> row{s, RES ? s_x : gx, base, n, part / kPart, rank, size, 0};
    if constexpr (RES) {
#pragma unroll 8
        for (int e = tid; e < part; e += kThreads) {
            const float v = e < int(n) ? __ldg(gx + e) : -INFINITY;
            s_x[e] = v > -INFINITY ? v : -INFINITY;   // NaN too
        }
        __syncthreads();
    }

    cl.sync();      // every CTA has begun before another writes to it

    // the largest, the smallest, how many can be drawn
    uint32_t top = 0, low = 0xffffffffu, cnt = 0;
    float best = -INFINITY;
    row.each([&](float4 v, uint32_t) {
        const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            best = fmaxf(best, x[j]);
            const uint32_t key = logit_key(x[j]);
            if (key) {
                low = min(low, key);
                ++cnt;
            }
        }
    });
    top = logit_key(best);
    const Slot all = row.exchange(cnt, 0, 0, top, low);
    top = all.c;
    const u64 count = all.a;
    if (top == 0) return give(0, 0.0f, 0);
    const float M = key_logit(top);
    uint32_t first = 0xffffffffu;
    row.each([&](float4 v, uint32_t i) {
        if (v.w == M) first = min(first, i + 3);
        if (v.z == M) first = min(first, i + 2);
        if (v.y == M) first = min(first, i + 1);
        if (v.x == M) first = min(first, i);
    });
    // with top-k: a logit that at least k reach, from the lanes' maxima: the
    // q-th largest of each full warp, the smallest of those over the warps
    uint32_t reach = 1;
    const bool by_k = k > 0 && u64(k) < count;
    const uint32_t of_warp = uint32_t(row.tiles) * kTile, full = N / of_warp;     // warps whose logits all exist
    const uint32_t q = by_k && full ? (uint32_t(k) + full - 1) / full : 0;
    if (q >= 1 && q <= 32) {
        uint32_t v = logit_key(best);
        for (uint32_t j = 1; j < q; ++j) {
            const uint32_t most = __reduce_max_sync(0xffffffffu, v);
            const unsigned who = __ballot_sync(0xffffffffu, v == most);
            if (lane == __ffs(who) - 1) v = 0;
        }
        reach = __reduce_max_sync(0xffffffffu, v);
        if (base / of_warp + (tid >> 5) >= full) reach = 0xffffffffu;
    }
    {
        // (the smallest over threads of `reach`, and of `first`)
        const Slot r = row.exchange(0, 0, 0, ~reach, first);
        reach = ~r.c;
        first = r.d;
    }
    if (T < 0x1p-60f) {
        return give(first, 1.0f, 1);
    }

    Weights w;
    const double c = 1.4426950408889634 / double(T);
    w.inf = M == INFINITY;
    w.pre = fmaxf(fabsf(M), fabsf(key_logit(all.d))) > 1e38f ? 0.5f : 1.0f;
    w.M = M * w.pre;
    w.ch = float(c / w.pre);
    w.cl = float(c / w.pre - double(w.ch));
    w.shift = shift;
    w.pow2 = s.pow2;
    const float span = w.M - key_logit(all.d) * w.pre;      // of all logits (0: all equal)
    const auto bins_over = [&](float d) {
        d = fminf(d, span);
        return d > 0.0f && d < INFINITY ? fminf(float(kBins) / d, FLT_MAX) : 0.0f;
    };

    Cut cut{-FLT_MAX, 0xffffffffu};      // everything above -inf
    if (by_k) {
        const float d = reach > 1 && reach < top ? (w.M - key_logit(reach) * w.pre) * 1.001f : span;
        const auto one = [&](float x, uint32_t) { return u64(x > -INFINITY); };
        const auto goal = [&](u64 n) { return n >= u64(k); };
        if (!cut_by_bins(row, w, bins_over(d), one, [&](float x, uint32_t) { return uint32_t(x > -INFINITY); }, u64(k),
                         [](u64) {}, goal, &cut))
            cut = row.search(top, one, goal, [&](u64 above, u64, u64) { return u64(k) - above; });
    }
    if (p <= 0.0f) {
        cut = {M, first};
    } else if (p < 1.0f) {
        // bins hold masses in units of 2^-31 of the sum, by its estimate
        float est = 0.0f;
        const Cut before = cut;
        row.each([&](float4 v, uint32_t i) {
            if (before.has(v.x, i)) est += w.rough(v.x);
            if (before.has(v.y, i + 1)) est += w.rough(v.y);
            if (before.has(v.z, i + 2)) est += w.rough(v.z);
            if (before.has(v.w, i + 3)) est += w.rough(v.w);
        });
        const u64 whole = row.exchange(u64(est * 16777216.0f), 0, 0, 0, 0).a;      // at least 2^24: M itself
        const float unit = 2147483648.0f / (float(whole) * 0x1p-24f);
        double P = 0.0;
        u64 S = 0;
        const auto f = [&](float x, uint32_t i) { return before.has(x, i) ? w(x) : 0; };
        const auto rough = [&](float x, uint32_t i) { return before.has(x, i) ? __float2uint_rn(w.rough(x) * unit) : 0u; };
        const auto prep = [&](u64 total) {
            S = total;
            P = double(p) * double(total);
        };
        const auto goal = [&](u64 mass) { return double(mass) >= P; };
        Cut c2;
        if (!cut_by_bins(row, w, bins_over(kOctaves / w.ch), f, rough, u64(double(p) * 2147483648.0) + 1, prep, goal, &c2)) {
            c2 = row.search(top, f, goal, [&](u64 above, u64 tie, u64 ties) {
                // the fewest ties that reach the mass
                u64 lo = 1, hi = ties;
                while (lo < hi) {
                    const u64 e = (lo + hi) / 2;
                    if (goal(above + e * tie)) hi = e; else lo = e + 1;
                }
                return lo;
            });
        }
        cut = c2;
    }
    if (mp > 1.0f) cut = {M, first};
    const double floor_d = ceil(double(mp) * double(u64(1) << shift));
    const u64 floor_w = floor_d >= 1.0 ? (floor_d > double(u64(1) << shift) ? u64(1) << shift : u64(floor_d)) : 0;

    // what is kept: its mass and number, and its lowest index
    u64 mass = 0;
    uint32_t kept = 0, lowest = 0xffffffffu;
    const auto keeps = [&](float x, uint32_t i, u64& wx) {
        wx = 0;
        if (!(x > -INFINITY) || !cut.has(x, i)) return false;
        wx = w(x);
        return wx >= floor_w;
    };
    row.each([&](float4 v, uint32_t i) {
        const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u64 wx;
            if (keeps(x[j], i + j, wx)) {
                mass += wx;
                ++kept;
                // (with +inf among the logits the others weigh nothing)
                if (!w.inf || wx) lowest = min(lowest, i + j);
            }
        }
    });
    const Slot fin = row.exchange(mass, kept, 0, 0, lowest);
    const u64 S = fin.a;
    uint32_t tok = fin.d;
    if (u > 0.0f) {
        const double r = floor(double(u) * double(S));
        const u64 e = r >= double(S) ? S : min(u64(r) + 1, S);       // the first sum above u * S
        tok = row.locate(e, [&](float x, uint32_t i) {
            u64 wx;
            return keeps(x, i, wx) ? wx : 0;
        });
    }
    if (rank == 0 && tid == 0) {
        const float x = a.x[m * a.ldx + tok];
        const double wt = x == M ? 1.0 : exp((double(x) - double(M)) / double(T));
        give(tok, float(wt * double(u64(1) << shift) / double(S)), int32_t(fin.b));
    }
    cl.sync();      // nobody leaves while another may still write here
}

template <bool RES>
cudaError_t launch_sample_kernel(const SampleArgs& a, int size, int part, int shift, const LaunchCtx& ctx) {
    static std::atomic<bool> ready[kMaxDevices];
    const cudaError_t e =
        set_smem_once(sample_kernel<RES>, RES ? size_t(kMaxPart) * 4 : 0, ctx.dev, ready);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attrs[2];
    cfg.gridDim = dim3(unsigned(a.rows * size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = RES ? size_t(part) * 4 : 0;
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
    // CTAs a row: parts of at most 16 K logits where 8 CTAs reach that; more,
    // down to parts of one tile a warp, while the GPU has SMs to spare
    int size = 1;
    while (size < kMaxCluster && (part_of(size) > 16 * 1024 ||
                                  (a.rows * size * 2 <= ctx.num_sms && part_of(size) > kPart)))
        size *= 2;
    const int part = part_of(size);
    if (part <= kMaxPart) return launch_sample_kernel<true>(a, size, part, 62 - bits, ctx);
    return launch_sample_kernel<false>(a, size, part, 62 - bits, ctx);
}

}  // namespace q8
