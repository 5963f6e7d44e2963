// evict.cu -- eviction from the K/V caches by accumulated attention weight.
//
// evict_select_kernel, a cluster of 1 to 8 CTAs a row and K/V head: a radix
// selection over the weights' ordered 32-bit keys (four digits of 8 bits, a
// histogram each, summed over the cluster through distributed shared memory;
// three digits of 11 bits: 64 KB a CTA of 8 reads there, 25 against 17 us at
// 32768 entries) gives the smallest kept key and how many equal to it stay; then
// every warp counts and lists the kept entries of its own range in order.  A
// lane holds its keys in registers where a warp's range is at most 256 entries
// and reads them again (4 bytes against the caches' hundreds) where it is
// longer; the CTA has a lane for eight keys of a row where 256 or 512 threads do
// (2048 of 4096 entries of 8 heads of 128 f32 values, moves included: 1024 threads
// 16.2 us, 512 14.4; 150 of 300 of 64 x 8 heads of 64: 1024 49, 256 30).  Bound by
// the latency of its steps: 12 us at 8192 entries a row and head, 16 at 32768.
//
// evict_move_kernel: K, V and acc to the front, in place and in order.  Entry
// j of the result comes from an entry idx[j] >= j.  A CTA owns a column slice
// of one row and head and walks j upwards in batches: what a batch overwrites
// is read by itself and earlier batches only, so a batch may be written once
// all of it has been read, and the next one's reads go out before that.
// Slices never touch, so CTAs need no order among them; the slice is as wide as
// leaves a CTA an SM, 64 bytes at least (8 heads of 24576 of 32768 f32 entries
// in 4 rows: 128 bytes 246 us; 64 bytes 40 us and 256 bytes 60 us more).  Where
// that leaves few CTAs (few rows and heads) and long walks, a cluster of up to 8
// walks a slice together, with a cluster barrier a batch, and slices are wider.
// Bound: HBM, each moved byte read and written once; measured there 6.6 TB/s
// (read and write), and 9 us for 2048 of 4096 entries of one row.  64 registers
// for two CTAs of 512 threads an SM: 8 to 12 bytes are spilled.
#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.h"
#include "q8proj.h"

namespace q8 {

namespace {

namespace cg = cooperative_groups;

constexpr int kDigit = 256, kMaxCluster = 8;
constexpr int kHeld = 8;                      // keys a lane holds at a time
constexpr int kBatch = 4;                     // pieces a thread has in a batch of moves

// Order of the weights as unsigned integers: NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (isnan(w)) return 0u;
    const uint32_t b = __float_as_uint(w + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The workspace, behind other calls' counters: per row and head the place of
// the first entry that moves (-1: none does), then its list of kept entries.
__device__ __forceinline__ int32_t* first_moved(const EvictArgs& a) {
    return reinterpret_cast<int32_t*>(static_cast<unsigned char*>(a.ws) + kCounterBytes);
}
__device__ __forceinline__ int32_t* kept_list(const EvictArgs& a, int64_t unit) {
    return first_moved(a) + (a.rows * a.kv_heads + 63) / 64 * 64 + unit * a.budget;
}

template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, 1024 / kSelThreads) evict_select_kernel(const EvictArgs a, int* err) {
    constexpr int kSelWarps = kSelThreads / 32;
    static_assert(kSelThreads >= kDigit && kSelWarps <= 32, "a thread a bin, a lane a warp");
    __shared__ uint32_t s_hist[2][kDigit], s_scan[kSelWarps], s_digit, s_above;
    __shared__ uint2 s_warp[kSelWarps];                 // sure ones and ties by warp
    __shared__ uint2 s_cta[kMaxCluster];             // and by CTA
    cg::cluster_group cl = cg::this_cluster();
    const unsigned rank = cl.block_rank(), size = cl.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t unit = blockIdx.x / size, m = unit / a.kv_heads;
    if (tid < kDigit) s_hist[1][tid] = 0;                // (the first digit's)
    pdl_wait();
    pdl_launch_dependents();
    const int pos = a.pos[m];
    const bool bad = pos < -1 || pos >= a.n_pos, writes = rank == 0 && tid == 0;
    if (bad && writes && unit == m * a.kv_heads) atomicExch(err, Q8_DEVERR_POSITION);
    const uint32_t n = bad ? 0 : uint32_t(pos) + 1;      // (n and some steps more fit 32 bits)
    const float* acc = a.acc + unit * a.n_pos;
    int32_t* kept = a.kept ? a.kept + unit * a.budget : nullptr;
    int32_t* idx = kept_list(a, unit);
    const uint32_t budget = uint32_t(a.budget);
    if (n <= budget) {                                   // the whole cluster alike
        if (writes) first_moved(a)[unit] = -1;
        if (kept)
            for (uint32_t i = rank * kSelThreads + tid; i < budget; i += size * kSelThreads) kept[i] = i < n ? int32_t(i) : -1;
        return;
    }
    const uint32_t lo = uint32_t(a.sinks), hi = n - uint32_t(a.recent);
    const uint32_t need = budget - lo - uint32_t(a.recent);
    // this warp's range of all entries, in whole steps of 32
    const uint32_t span = (n + size * kSelWarps * 32 - 1) / (size * kSelWarps * 32) * 32;
    const uint32_t w0 = min((rank * kSelWarps + warp) * span, n), w1 = min(w0 + span, n);
    const bool held = span <= 32 * kHeld;
    uint32_t key[kHeld];                                 // of entries [at, at + 256), lanes in turn
    const auto fetch = [&](uint32_t at) {
        float w[kHeld];
#pragma unroll
        for (int j = 0; j < kHeld; ++j) w[j] = at + 32 * j + lane < w1 ? acc[at + 32 * j + lane] : 0.0f;
#pragma unroll
        for (int j = 0; j < kHeld; ++j) key[j] = weight_key(w[j]);
    };
    if (held) fetch(w0);

    // t: the key of the need-th largest weight in [lo, hi); above: how many are larger
    uint32_t t = 0xffffffffu, above = 0;
    if (need) {
        t = 0;
        uint32_t mask = 0;                               // the digits found so far
        const uint32_t zero = weight_key(0.0f), c1 = min(w1, hi);
#pragma unroll 1
        for (int shift = 24; shift >= 0; shift -= 8) {
            uint32_t* hist = s_hist[shift >> 3 & 1];
            __syncthreads();                             // (the bins are zero)
            // weights of zero, the commonest one, are counted in a register
            uint32_t zeros = 0;
            for (uint32_t at = w0; at < w1; at += 32 * kHeld) {
                if (!held) fetch(at);
#pragma unroll
                for (int j = 0; j < kHeld; ++j) {
                    const uint32_t i = at + 32 * j + lane;
                    if (i < lo || i >= c1 || (key[j] & mask) != t) continue;
                    if (key[j] == zero) ++zeros;
                    else atomicAdd(&hist[(key[j] >> shift) & 255u], 1u);
                }
            }
            zeros = __reduce_add_sync(0xffffffffu, zeros);
            if (lane == 0 && zeros) atomicAdd(&hist[(zero >> shift) & 255u], zeros);
            cluster_sync(size);
            // (the other bins were last read before this barrier's other side)
            if (tid < kDigit) s_hist[~(shift >> 3) & 1][tid] = 0;
            // from the largest digit down: where the cluster's count reaches what is left
            const uint32_t digit = kDigit - 1 - tid, left = need - above;
            uint32_t c = 0, up;
            if (tid < kDigit) {
#pragma unroll 8
                for (unsigned r = 0; r < size; ++r) c += cl.map_shared_rank(hist, r)[digit];
            }
            up = c;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, up, d);
                if (lane >= d) up += y;
            }
            if (lane == 31) s_scan[warp] = up;
            __syncthreads();
            uint32_t before = up - c;
            for (int k = 0; k < min(warp, kDigit / 32); ++k) before += s_scan[k];
            if (tid < kDigit && before < left && before + c >= left) {
                s_digit = digit;
                s_above = before;
            }
            __syncthreads();
            t |= s_digit << shift;
            above += s_above;
            mask |= 255u << shift;
        }
    }
    const uint32_t ties = need - above;      // entries equal to t that stay, the first ones

    // count this warp's kept ones: those that stay for sure, and ties
    const auto judge = [&](uint32_t i, uint32_t k, bool& sure, bool& tie) {
        const bool in = i < w1, mid = i >= lo && i < hi;
        sure = in && (!mid || (need && k > t));
        tie = in && mid && need && k == t;
    };
    uint2 cnt = make_uint2(0, 0);
    for (uint32_t at = w0; at < w1; at += 32 * kHeld) {
        if (!held) fetch(at);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            bool sure, tie;
            judge(at + 32 * j + lane, key[j], sure, tie);
            cnt.x += __popc(__ballot_sync(0xffffffffu, sure));
            cnt.y += __popc(__ballot_sync(0xffffffffu, tie));
        }
    }
    if (lane == 0) s_warp[warp] = cnt;
    if (need == 0) cluster_sync(size);                            // (every CTA runs, else the passes' barriers say so)
    __syncthreads();
    // kept ones before this warp: of the CTA's warps, then of the CTAs before
    const uint2 of = lane < kSelWarps ? s_warp[lane] : make_uint2(0, 0);
    uint2 up = of;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, up.x, d), y = __shfl_up_sync(0xffffffffu, up.y, d);
        if (lane >= d) up.x += x, up.y += y;
    }
    uint2 off = make_uint2(__shfl_sync(0xffffffffu, up.x - of.x, warp), __shfl_sync(0xffffffffu, up.y - of.y, warp));
    if (size > 1) {
        if (warp == 0) {
            const uint2 all = make_uint2(__shfl_sync(0xffffffffu, up.x, 31), __shfl_sync(0xffffffffu, up.y, 31));
            if (lane < int(size)) *cl.map_shared_rank(&s_cta[rank], lane) = all;
        }
        cluster_sync(size);
        for (unsigned r = 0; r < rank; ++r) {
            off.x += s_cta[r].x;
            off.y += s_cta[r].y;
        }
    }
    // list them; the first that does not stay lies in the warp before whose
    // range every entry stays
    const bool all_before = off.x + min(off.y, ties) == w0;
    uint32_t first = n;
    for (uint32_t at = w0; at < w1; at += 32 * kHeld) {
        if (!held) fetch(at);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            const uint32_t i = at + 32 * j + lane, below = (1u << lane) - 1;
            bool sure, tie;
            judge(i, key[j], sure, tie);
            const unsigned vs = __ballot_sync(0xffffffffu, sure), vt = __ballot_sync(0xffffffffu, tie);
            const uint32_t s = off.x + __popc(vs & below), e = off.y + __popc(vt & below);
            if (sure || (tie && e < ties)) {
                const uint32_t to = s + min(e, ties);
                idx[to] = int32_t(i);
                if (kept) kept[to] = int32_t(i);
            } else if (i < w1) {
                first = min(first, i);
            }
            off.x += __popc(vs);
            off.y += __popc(vt);
        }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    if (all_before && first < n && lane == 0) first_moved(a)[unit] = int32_t(first);     // as many stay where they are
}

// Moves items [from, budget) of 16 bytes (caches) or 4 (acc), `pitch` bytes
// apart; src may be dst.  In a batch the cluster has size * kBatch * rows items,
// this thread those that are `mine` of its CTA's rows.
template <bool CLUSTER, typename V>
__device__ __forceinline__ void move_items(const unsigned char* src, unsigned char* dst, int64_t pitch, const int32_t* idx,
                                           int64_t from, int64_t budget, int rows, int mine, bool has, unsigned rank,
                                           unsigned size) {
    V next[kBatch], now[kBatch];
    const int64_t every = int64_t(rows) * size, at0 = int64_t(rank) * rows + mine;
    const auto load = [&](int64_t j0) {
        int at[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int64_t j = j0 + b * every + at0;
            at[b] = has && j < budget ? idx[j] : -1;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (at[b] >= 0) next[b] = *reinterpret_cast<const V*>(src + int64_t(at[b]) * pitch);
    };
    const int64_t step = every * kBatch;
    load(from);
    for (int64_t j0 = from; j0 < budget; j0 += step) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) now[b] = next[b];
        // a barrier: every read of this batch is done
        if (CLUSTER) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
        if (j0 + step < budget) load(j0 + step);
        if (CLUSTER) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        else __syncthreads();
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int64_t j = j0 + b * every + at0;
            if (has && j < budget) *reinterpret_cast<V*>(dst + j * pitch) = now[b];
        }
    }
}

// acc of one row and K/V head, and the row's new position.
template <bool CLUSTER, int kThreads>
__device__ __forceinline__ void move_acc(const EvictArgs& a, int64_t unit, unsigned rank, unsigned size) {
    const int64_t m = unit / a.kv_heads;
    const int tid = threadIdx.x, from = first_moved(a)[unit];
    if (unit == m * a.kv_heads && rank == 0 && tid == 0) {
        // (pos may be new_pos: nobody else reads it in this kernel)
        a.new_pos[m] = from < 0 ? a.pos[m] : int32_t(a.budget - 1);
    }
    const float* acc = a.acc + unit * a.n_pos;
    float* new_acc = a.new_acc + unit * a.n_pos;
    const int64_t as_is = from < 0 ? a.n_pos : from, me = int64_t(rank) * kThreads + tid, all = int64_t(size) * kThreads;
    if (new_acc != acc)
        for (int64_t i = me; i < as_is; i += all) new_acc[i] = acc[i];
    if (from < 0) return;                                // (the whole cluster alike)
    move_items<CLUSTER, float>(reinterpret_cast<const unsigned char*>(acc), reinterpret_cast<unsigned char*>(new_acc), 4,
                         kept_list(a, unit), from, a.budget, kThreads, tid, true, rank, size);
    // (every read ended before the last batch's barrier)
    for (int64_t i = a.budget + me; i < a.n_pos; i += all) new_acc[i] = 0.0f;
}

// Cluster: acc of one row and K/V head (the first ones), or its K or V in one
// column slice of 16 << lanes_log bytes.
template <bool CLUSTER, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    evict_move_kernel(const EvictArgs a, int elt, int lanes_log, int slices) {
    const unsigned rank = CLUSTER ? cg::this_cluster().block_rank() : 0;
    const unsigned size = CLUSTER ? cg::this_cluster().num_blocks() : 1;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t units = a.rows * a.kv_heads, cluster = blockIdx.x / size;
    const int tid = threadIdx.x;
    if (cluster < units) {
        move_acc<CLUSTER, kThreads>(a, cluster, rank, size);
        return;
    }
    const int64_t id = cluster - units;
    const int slice = int(id % slices), kv = int(id / slices % 2);
    const int64_t unit = id / slices / 2, m = unit / a.kv_heads, h = unit % a.kv_heads;
    const int from = first_moved(a)[unit];
    if (from < 0) return;
    const int64_t row_bytes = a.dim * elt, pitch = a.kv_heads * row_bytes;
    const int64_t col = int64_t((slice << lanes_log) + (tid & ((1 << lanes_log) - 1))) * 16;
    unsigned char* base = static_cast<unsigned char*>(kv ? a.v : a.k) + m * a.n_pos * pitch + h * row_bytes + col;
    move_items<CLUSTER, int4>(base, base, pitch, kept_list(a, unit), from, a.budget, kThreads >> lanes_log, tid >> lanes_log,
                        col < row_bytes, rank, size);
}

// The same over quantised caches, head-major.  Cluster: the codes of one row, K/V head and
// one of K and V, in one column slice of `lanes` pieces of 16 bytes; behind those, the words
// of one; behind those, acc.
template <bool CLUSTER, typename V>
__device__ __forceinline__ void move_plane(unsigned char* base, int bytes, int lanes, int slice, const int32_t* idx,
                                           int64_t from, int64_t budget, unsigned rank, unsigned size) {
    const int rows = int(blockDim.x) / lanes, mine = threadIdx.x / lanes;
    const int col = (slice * lanes + threadIdx.x - mine * lanes) * int(sizeof(V));
    move_items<CLUSTER, V>(base + col, base + col, bytes, idx, from, budget, rows, mine, mine < rows && col < bytes, rank,
                           size);
}

template <bool CLUSTER, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    evict_move_kvq_kernel(const EvictArgs a, int row, int lanes, int slices) {
    const unsigned rank = CLUSTER ? cg::this_cluster().block_rank() : 0;
    const unsigned size = CLUSTER ? cg::this_cluster().num_blocks() : 1;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t units = a.rows * a.kv_heads, moves = units * 2 * slices;
    int64_t id = blockIdx.x / size;
    if (id < moves) {
        const int slice = int(id % slices), kv = int(id / slices % 2);
        const int64_t unit = id / slices / 2;
        const int from = first_moved(a)[unit];
        if (from < 0) return;                                // (the whole cluster alike)
        unsigned char* base = static_cast<unsigned char*>(kv ? a.v : a.k) + unit * a.n_pos * row;
        move_plane<CLUSTER, int4>(base, row, lanes, slice, kept_list(a, unit), from, a.budget, rank, size);
        return;
    }
    id -= moves;
    if (id < 2 * units) {
        const int64_t unit = id / 2;
        const int from = first_moved(a)[unit], bytes = int(a.dim) / 8;
        if (from < 0) return;
        unsigned char* base = reinterpret_cast<unsigned char*>(id % 2 ? a.v_words : a.k_words) + unit * a.n_pos * bytes;
        if (bytes % 16 == 0)
            move_plane<CLUSTER, int4>(base, bytes, bytes / 16, 0, kept_list(a, unit), from, a.budget, rank, size);
        else
            move_plane<CLUSTER, int>(base, bytes, bytes / 4, 0, kept_list(a, unit), from, a.budget, rank, size);
        return;
    }
    move_acc<CLUSTER, kThreads>(a, id - 2 * units, rank, size);
}

template <bool CLUSTER, int kThreads>
cudaError_t launch_move_kvq_as(const EvictArgs& a, int size, int row, int lanes, int slices, const LaunchCtx& ctx) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attrs[2];
    cfg.gridDim = dim3(unsigned(a.rows * a.kv_heads * (3 + 2 * slices) * size));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = ctx.stream;
    cfg.numAttrs = pdl_attrs(ctx, attrs);
    if (CLUSTER) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attrs[cfg.numAttrs].val.clusterDim.x = unsigned(size);
        attrs[cfg.numAttrs].val.clusterDim.y = 1;
        attrs[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    cfg.attrs = attrs;
    return cudaLaunchKernelEx(&cfg, evict_move_kvq_kernel<CLUSTER, kThreads>, a, row, lanes, slices);
}

cudaError_t launch_move_kvq(const EvictArgs& a, const LaunchCtx& ctx) {
    const int row = int(a.kv_type == kKvQuantised + Q8_KVQ_U4 ? a.dim / 2 : a.dim), chunks = row / 16;
    // Up to two CTAs an SM that walk codes, first by clusters of three batches a CTA and more
    // (4 x 8 heads of 128 bytes, 24576 of 32768 entries: 171 us alone, 131 in pairs, 98 in
    // fours, 107 in eights), then by slices of 64 bytes at least (1 x 8 heads, 40000 of 65536:
    // eights 65 us, 54 in two slices, 62 in four); 256 threads where even single CTAs are more
    // (64 x 8 heads of 32 bytes, 150 of 300: 24 and 17 us; of 128, 1000 of 2000: 68 and 62).
    const int64_t ctas = a.rows * a.kv_heads * 2, most = 2 * int64_t(ctx.num_sms), batch = int64_t(512 / chunks) * kBatch;
    int size = 1, slices = 1;
    while (size < kMaxCluster && ctas * size * 2 <= most && a.budget >= 3 * batch * size * 2) size *= 2;
    while (ctas * size * slices * 2 <= most && chunks >= 8 * slices) slices *= 2;
    const int lanes = (chunks + slices - 1) / slices;
    slices = (chunks + lanes - 1) / lanes;
    if (size > 1) return launch_move_kvq_as<true, 512>(a, size, row, lanes, slices, ctx);
    if (ctas > most) return launch_move_kvq_as<false, 256>(a, 1, row, lanes, slices, ctx);
    return launch_move_kvq_as<false, 512>(a, 1, row, lanes, slices, ctx);
}

template <int THREADS>
cudaError_t launch_select(const EvictArgs& a, const LaunchCtx& ctx) {
    // CTAs a row and head: so many that lanes hold their keys, where 8 reach that
    // (a barrier of one CTA costs 0.4 thousand cycles, of a cluster 1.8)
    int size = 1;
    while (size < kMaxCluster && a.n_pos > int64_t(size) * THREADS * kHeld) size *= 2;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attrs[2];
    cfg.stream = ctx.stream;
    cfg.numAttrs = pdl_attrs(ctx, attrs);
    attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attrs[cfg.numAttrs].val.clusterDim.x = unsigned(size);
    attrs[cfg.numAttrs].val.clusterDim.y = 1;
    attrs[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
    cfg.attrs = attrs;
    cfg.gridDim = dim3(unsigned(a.rows * a.kv_heads * size));
    cfg.blockDim = dim3(THREADS);
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<THREADS>, a, ctx.dev_err);
}

template <bool CLUSTER, int kThreads>
cudaError_t launch_move(const EvictArgs& a, int size, int elt, int lanes_log, int slices, const LaunchCtx& ctx) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attrs[2];
    cfg.gridDim = dim3(unsigned(a.rows * a.kv_heads * (1 + 2 * slices) * size));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = ctx.stream;
    cfg.numAttrs = pdl_attrs(ctx, attrs);
    if (CLUSTER) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attrs[cfg.numAttrs].val.clusterDim.x = unsigned(size);
        attrs[cfg.numAttrs].val.clusterDim.y = 1;
        attrs[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    cfg.attrs = attrs;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel<CLUSTER, kThreads>, a, elt, lanes_log, slices);
}

}  // namespace

size_t evict_workspace_bytes(int64_t rows, int64_t kv_heads, int64_t budget) {
    const size_t units = size_t(rows * kv_heads);
    return kCounterBytes + ((units + 63) / 64 * 64 + units * size_t(budget)) * sizeof(int32_t);
}

cudaError_t launch_evict(const EvictArgs& a, const LaunchCtx& ctx) {
    const int64_t units = a.rows * a.kv_heads;
    const cudaError_t e = a.n_pos <= 256 * kHeld   ? launch_select<256>(a, ctx)
                          : a.n_pos <= 512 * kHeld ? launch_select<512>(a, ctx)
                                                   : launch_select<1024>(a, ctx);
    if (e != cudaSuccess) return e;
    if (a.kv_type >= kKvQuantised) return launch_move_kvq(a, ctx);
    // the widest slice that leaves a CTA an SM, 64 bytes at least
    const int elt = a.kv_type == Q8_KV_F32 ? 4 : 2, chunks = int(a.dim) * elt / 16;      // 16-byte pieces an entry
    int lanes_log = 5;
    const auto slices_at = [&](int log) { return (chunks + (1 << log) - 1) >> log; };
    while (lanes_log > 2 && ((1 << (lanes_log - 1)) >= chunks || units * 2 * slices_at(lanes_log) < ctx.num_sms))
        --lanes_log;
    // where even those leave an SM one CTA and a long walk, clusters walk
    // together: up to 5 CTAs an SM in all, three batches each at least (1 x 8 heads
    // of 64 f16 values, 41475 of 55887 entries: 123 us alone, 57 in eights; 16 x 8
    // heads of 128, two CTAs an SM: 76 alone, 96 in pairs); and wider slices then,
    // while eights of them leave five CTAs to four SMs (3 x 2 heads of 128 f32 values,
    // 16144 of 47256: 64 bytes 66 us, 128 64, 256, 192 CTAs, 59, 512, 96 CTAs, 93)
    const auto few = [&](int log) { return units * 2 * slices_at(log) <= ctx.num_sms + ctx.num_sms / 10; };
    const auto batch_at = [&](int log) { return int64_t(512 >> log) * kBatch; };
    while (few(lanes_log) && lanes_log < 5 && (1 << lanes_log) < chunks &&
           units * 2 * slices_at(lanes_log + 1) * kMaxCluster * 4 >= 5 * int64_t(ctx.num_sms) &&
           a.budget >= 3 * batch_at(lanes_log + 1) * kMaxCluster)
        ++lanes_log;
    const int slices = slices_at(lanes_log);
    const int64_t ctas = units * 2 * slices, batch = batch_at(lanes_log);
    int size = 1;
    while (size < kMaxCluster && few(lanes_log) && ctas * size * 2 <= 5 * int64_t(ctx.num_sms) &&
           a.budget >= 3 * batch * size * 2)
        size *= 2;
    if (size > 1) return launch_move<true, 512>(a, size, elt, lanes_log, slices, ctx);
    // short walks of more CTAs than two an SM: 256 threads, four an SM (256 x 8 heads
    // of 128 bf16 values, 150 of 300: 104 us with 512, 85 with 256, 80 with 128;
    // 16 x 8, 1000 of 2000: 33, 35)
    if (a.budget <= 512 && ctas > 2 * int64_t(ctx.num_sms))
        return launch_move<false, 256>(a, size, elt, lanes_log, slices, ctx);
    return launch_move<false, 512>(a, size, elt, lanes_log, slices, ctx);
}

}  // namespace q8
