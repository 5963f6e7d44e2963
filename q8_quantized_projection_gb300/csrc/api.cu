// api.cu -- the C ABI of libq8proj (declared in include/q8proj.h): argument
// validation on the host, then launches of the kernels on the caller's stream.
#include <math.h>

#include <atomic>
#include <cfloat>
#include <mutex>

#include "common.cuh"
#include "launch.h"
#include "q8proj.h"

namespace q8 {
cudaError_t launch_gemv_mode0(const GemvArgs& a, const LaunchCtx& ctx);
cudaError_t launch_gemv_mode1(const GemvArgs& a, const LaunchCtx& ctx);
cudaError_t launch_gemv_mode2(const GemvArgs& a, const LaunchCtx& ctx);
cudaError_t launch_gemv_fused_mode0(const GemvArgs& a, const LaunchCtx& ctx);
cudaError_t launch_gemv_fused_mode1(const GemvArgs& a, const LaunchCtx& ctx);
cudaError_t launch_gemv_fused_mode2(const GemvArgs& a, const LaunchCtx& ctx);
}  // namespace q8

using namespace q8;

// Device error word: bounded waits that run out record a code here.
__device__ int g_q8_dev_err;

namespace {

thread_local int t_last_cuda = 0;
std::atomic<int> g_pdl{1};   // q8_set_pdl may race with launches on other threads

struct DevInfo {
    bool ready = false;
    int num_sms = 0;
    int* dev_err = nullptr;
};
DevInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

q8_status cuda_fail(cudaError_t e) {
    t_last_cuda = int(e);
    return Q8_ERR_CUDA;
}

q8_status make_ctx(void* stream, LaunchCtx& ctx) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 0 || dev >= kMaxDevices) return Q8_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lk(g_dev_mu);
    DevInfo& d = g_dev[dev];
    if (!d.ready) {
        e = cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e);
        void* p = nullptr;
        e = cudaGetSymbolAddress(&p, g_q8_dev_err);
        if (e != cudaSuccess) return cuda_fail(e);
        d.dev_err = static_cast<int*>(p);
        d.ready = true;
    }
    ctx.dev = dev;
    ctx.stream = static_cast<cudaStream_t>(stream);
    ctx.pdl = g_pdl.load(std::memory_order_relaxed) != 0;
    ctx.num_sms = d.num_sms;
    ctx.dev_err = d.dev_err;
    return Q8_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

q8_status launched(cudaError_t e) { return e == cudaSuccess ? Q8_OK : cuda_fail(e); }

bool valid_mode(int mode) { return mode >= Q8_ACT_F32 && mode <= Q8_ACT_I8X2; }

q8_status check_shape(int64_t N, int64_t K) {
    if (N < 1 || K < Q8_QK || K % Q8_QK != 0) return Q8_ERR_SHAPE;
    if (N > (int64_t(1) << 31) - 1 || K > (int64_t(1) << 24)) return Q8_ERR_SHAPE;
    return Q8_OK;
}

size_t act_bytes(int mode, int64_t rows, int64_t K) {
    if (mode == Q8_ACT_F32) return size_t(rows) * K * 4;
    if (mode == Q8_ACT_I8) return size_t(rows) * K;
    return size_t(2) * rows * K;
}

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

cudaError_t gemv_dispatch(const GemvArgs& a, const LaunchCtx& ctx) {
    if (a.mode == Q8_ACT_F32) return launch_gemv_mode0(a, ctx);
    if (a.mode == Q8_ACT_I8) return launch_gemv_mode1(a, ctx);
    return launch_gemv_mode2(a, ctx);
}

// The KV-row epilogue's arguments (k_cache NULL: none).
struct KvArgs {
    const int32_t* pos = nullptr;
    int64_t kv_col = 0, kv_dim = 0, n_pos = 0;
    float* k_cache = nullptr;
    float* v_cache = nullptr;
};

// Runs the CUDA-core projection over groups of gemv_group_rows(mode, K)
// activation rows (each group one launch reading the weights once).
q8_status run_projection(int mode, const int8_t* q, const uint16_t* s, int64_t N, int64_t K,
                         const void* xq, const float* xd, int64_t rows, void* y, int out_f64,
                         int32_t* tok, double* maxval, void* ws, const LaunchCtx& ctx) {
    const int64_t nb = K / Q8_QK;
    const int group = gemv_group_rows(mode, K);
    const size_t elem = (mode == Q8_ACT_F32) ? 4 : 1;
    const size_t ysz = (mode == Q8_ACT_F32 && out_f64) ? 8 : 4;
    for (int64_t g0 = 0; g0 < rows; g0 += group) {
        GemvArgs a{};
        a.mode = mode;
        a.q = q;
        a.s = s;
        a.N = N;
        a.K = K;
        a.act = static_cast<const unsigned char*>(xq) + size_t(g0) * K * elem;
        a.xd = xd ? xd + g0 * nb : nullptr;
        a.plane = rows * K;
        a.rows = int(rows - g0 < group ? rows - g0 : group);
        a.y = y ? static_cast<unsigned char*>(y) + size_t(g0) * N * ysz : nullptr;
        a.out_f64 = out_f64;
        a.tok = tok ? tok + g0 : nullptr;
        a.maxval = maxval ? maxval + g0 : nullptr;
        a.ws = ws;
        cudaError_t e = gemv_dispatch(a, ctx);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return Q8_OK;
}

// Plain projection of an activation: the tensor-core chunk kernel from
// chunk_min_rows(mode) rows on (K % 256 == 0), the CUDA-core kernels else.
q8_status project_dispatch(int mode, const int8_t* q, const uint16_t* s, int64_t N, int64_t K,
                           const void* xq, const float* xd, int64_t rows, void* y, int out_f64,
                           const LaunchCtx& ctx) {
    // (f32 at 4 rows runs as two row pairs where the row-per-lane kernel holds
    // a pair: 2 x 87 against 197 us for the d = 4096 layer)
    const bool f32_pairs = mode == Q8_ACT_F32 && rows == 4 && gemv_group_rows(mode, K) == 2;
    if (!f32_pairs && (!out_f64 || mode == Q8_ACT_F32) && rows >= chunk_min_rows(mode) &&
        chunk_supported(mode, N, K, rows))
        return launched(launch_chunk(mode, q, s, N, K, xq, xd, rows, y, out_f64 != 0, ctx));
    return run_projection(mode, q, s, N, K, xq, xd, rows, y, out_f64, nullptr, nullptr, nullptr,
                          ctx);
}

q8_status check_proj_args(int mode, const int8_t* q, const uint16_t* s, int64_t N, int64_t K,
                          const void* xq, const float* xd, int64_t rows, const void* y) {
    if (!valid_mode(mode)) return Q8_ERR_MODE;
    if (!q || !s || !xq || !y || (mode != Q8_ACT_F32 && !xd)) return Q8_ERR_ARG;
    q8_status st = check_shape(N, K);
    if (st != Q8_OK) return st;
    if (rows < 1 || rows > Q8_MAX_ROWS) return Q8_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(s) || !aligned16(xq) || !aligned16(y) ||
        (xd && !aligned16(xd)))
        return Q8_ERR_ALIGN;
    return Q8_OK;
}

}  // namespace

extern "C" {

const char* q8_status_str(int status) {
    switch (status) {
        case Q8_OK: return "Q8_OK";
        case Q8_ERR_ARG: return "Q8_ERR_ARG";
        case Q8_ERR_SHAPE: return "Q8_ERR_SHAPE";
        case Q8_ERR_ALIGN: return "Q8_ERR_ALIGN";
        case Q8_ERR_MODE: return "Q8_ERR_MODE";
        case Q8_ERR_CUDA: return "Q8_ERR_CUDA";
        case Q8_ERR_UNSUPPORTED: return "Q8_ERR_UNSUPPORTED";
        case Q8_ERR_WORKSPACE: return "Q8_ERR_WORKSPACE";
        default: return "Q8_ERR_UNKNOWN";
    }
}

int q8_version(void) { return 106; }

int q8_last_cuda_error(void) { return t_last_cuda; }

void q8_set_pdl(int enable) { g_pdl.store(enable ? 1 : 0, std::memory_order_relaxed); }

q8_status q8_device_error(int32_t* code, void* stream) {
    if (!code) return Q8_ERR_ARG;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e);
    int v = 0;
    e = cudaMemcpyFromSymbol(&v, g_q8_dev_err, sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e);
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_q8_dev_err, &zero, sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e);
    *code = v;
    return Q8_OK;
}

q8_status q8_pack(const float* w, int64_t N, int64_t K, int8_t* q, uint16_t* s,
                  int32_t* overflow, void* stream) {
    if (!w || !q || !s) return Q8_ERR_ARG;
    q8_status st = check_shape(N, K);
    if (st != Q8_OK) return st;
    if (!aligned16(w) || !aligned16(q) || !aligned16(s) || (overflow && !aligned16(overflow)))
        return Q8_ERR_ALIGN;
    LaunchCtx ctx;
    if ((st = make_ctx(stream, ctx)) != Q8_OK) return st;
    return launched(launch_pack(w, N, K, q, s, overflow, ctx));
}

// [a, a + n) and [b, b + n) overlap (either NULL: no)
static bool overlaps(const void* a, const void* b, size_t n) {
    if (!a || !b) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + n && y < x + n;
}

// The residual's arguments: r required; s_out optional, 16-byte aligned and
// disjoint from h and r (every CTA of a fused call reads all of h and r).
static q8_status check_residual(const float* h, const float* r, const float* s_out, int64_t rows,
                                int64_t K) {
    if (!r) return Q8_ERR_ARG;
    if (!aligned16(r) || (s_out && !aligned16(s_out))) return Q8_ERR_ALIGN;
    const size_t n = size_t(rows) * size_t(K) * sizeof(float);
    if (overlaps(s_out, h, n) || overlaps(s_out, r, n)) return Q8_ERR_ARG;
    return Q8_OK;
}

// prod: 0 plain, 1 residual, 2 SwiGLU (h: the gate+up output, rows of 2K)
static q8_status act_quant_impl(int mode, int prod, const float* h, const float* res, float* s_out,
                                int64_t rows, int64_t K, int norm, const float* gain, float eps,
                                void* xq, float* xd, void* stream) {
    if (!valid_mode(mode)) return Q8_ERR_MODE;
    if (!h || !xq || (mode != Q8_ACT_F32 && !xd)) return Q8_ERR_ARG;
    if (norm != 0 && norm != 1) return Q8_ERR_ARG;
    if (!(eps >= 0.0f)) return Q8_ERR_ARG;
    q8_status st = check_shape(1, K);
    if (st != Q8_OK) return st;
    if (rows < 1 || rows > Q8_MAX_ROWS) return Q8_ERR_SHAPE;
    if (!aligned16(h) || !aligned16(xq) || (xd && !aligned16(xd)) || (gain && !aligned16(gain)))
        return Q8_ERR_ALIGN;
    LaunchCtx ctx;
    if ((st = make_ctx(stream, ctx)) != Q8_OK) return st;
    return launched(launch_act_quant(mode, prod, h, res, s_out, rows, K, norm, gain, eps, xq, xd, ctx));
}

q8_status act_quant(int mode, const float* h, int64_t rows, int64_t K, int norm,
                    const float* gain, float eps, void* xq, float* xd, void* stream) {
    return act_quant_impl(mode, 0, h, nullptr, nullptr, rows, K, norm, gain, eps, xq, xd, stream);
}

q8_status act_quant_residual(int mode, const float* h, const float* r, float* s_out, int64_t rows,
                             int64_t K, const float* gain, float eps, void* xq, float* xd,
                             void* stream) {
    if (!h) return Q8_ERR_ARG;
    const q8_status st = check_residual(h, r, s_out, rows, K);
    if (st != Q8_OK) return st;
    return act_quant_impl(mode, 1, h, r, s_out, rows, K, 1, gain, eps, xq, xd, stream);
}

q8_status act_quant_swiglu(int mode, const float* gu, int64_t rows, int64_t K, void* xq, float* xd,
                           void* stream) {
    return act_quant_impl(mode, 2, gu, nullptr, nullptr, rows, K, 0, nullptr, 0.0f, xq, xd, stream);
}

q8_status q8_proj(int mode, const int8_t* q, const uint16_t* s, int64_t N, int64_t K,
                  const void* xq, const float* xd, int64_t rows, void* y, int out_f64,
                  void* stream) {
    q8_status st = check_proj_args(mode, q, s, N, K, xq, xd, rows, y);
    if (st != Q8_OK) return st;
    if (out_f64 && mode != Q8_ACT_F32) return Q8_ERR_MODE;
    LaunchCtx ctx;
    if ((st = make_ctx(stream, ctx)) != Q8_OK) return st;
    return project_dispatch(mode, q, s, N, K, xq, xd, rows, y, out_f64 ? 1 : 0, ctx);
}

q8_status q8_proj_chunk(int mode, const int8_t* q, const uint16_t* s, int64_t N, int64_t K,
                        const void* xq, const float* xd, int64_t T, float* y, void* stream) {
    q8_status st = check_proj_args(mode, q, s, N, K, xq, xd, T, y);
    if (st != Q8_OK) return st;
    LaunchCtx ctx;
    if ((st = make_ctx(stream, ctx)) != Q8_OK) return st;
    return project_dispatch(mode, q, s, N, K, xq, xd, T, y, 0, ctx);
}

q8_status q8_debug_chunk_plan(int mode, int64_t N, int64_t K, int64_t T, int argmax, int64_t* out) {
    if (!out) return Q8_ERR_ARG;
    if (!valid_mode(mode)) return Q8_ERR_MODE;
    if (N < 1 || N > (int64_t(1) << 31) || T < 1 || T > Q8_MAX_ROWS || K < 256 || K % 256 != 0 ||
        K > (int64_t(1) << 24))
        return Q8_ERR_SHAPE;
    LaunchCtx ctx;
    q8_status st = make_ctx(nullptr, ctx);
    if (st != Q8_OK) return st;
    return chunk_plan(mode, N, K, T, argmax != 0, ctx, out) ? Q8_OK : Q8_ERR_UNSUPPORTED;
}

size_t q8_proj_fused_workspace(int mode, int64_t rows, int64_t K) {
    if (!valid_mode(mode) || rows < 1 || K < Q8_QK) return 0;
    return round_up(act_bytes(mode, rows, K), 256) + round_up(size_t(rows) * (K / Q8_QK) * 4, 256);
}

static q8_status proj_fused_impl(int mode, int prod, const int8_t* q, const uint16_t* s, int64_t N,
                                 int64_t K, const float* h, const float* res, float* s_out, int64_t rows,
                                 const float* gain, float eps, void* y, int out_f64, void* workspace,
                                 size_t ws_bytes, void* stream, const KvArgs& kv = KvArgs{}) {
    if (!workspace) return Q8_ERR_WORKSPACE;
    // (h stands in for the scales argument: the fused call has none)
    q8_status st = check_proj_args(mode, q, s, N, K, h, h, rows, y);
    if (st != Q8_OK) return st;
    if (out_f64 && mode != Q8_ACT_F32) return Q8_ERR_MODE;
    if (gain && !aligned16(gain)) return Q8_ERR_ALIGN;
    if (!(eps >= 0.0f)) return Q8_ERR_ARG;
    if (!aligned16(workspace)) return Q8_ERR_ALIGN;
    if (ws_bytes < q8_proj_fused_workspace(mode, rows, K)) return Q8_ERR_WORKSPACE;
    LaunchCtx ctx;
    if ((st = make_ctx(stream, ctx)) != Q8_OK) return st;
    if (rows == 1 && K <= kFusedMaxK) {
        // decode step: one launch, the producer runs inside the projection
        GemvArgs a{};
        a.mode = mode;
        a.q = q;
        a.s = s;
        a.N = N;
        a.K = K;
        a.rows = 1;
        a.plane = K;
        a.y = y;
        a.out_f64 = out_f64 ? 1 : 0;
        a.h = h;
        a.prod = prod;
        a.res = res;
        a.s_out = s_out;
        a.gain = gain;
        a.eps = eps;
        a.pos = kv.pos;
        a.kv_col = kv.kv_col;
        a.kv_dim = kv.kv_dim;
        a.n_pos = kv.n_pos;
        a.k_cache = kv.k_cache;
        a.v_cache = kv.v_cache;
        return launched(mode == Q8_ACT_F32 ? launch_gemv_fused_mode0(a, ctx)
                        : mode == Q8_ACT_I8 ? launch_gemv_fused_mode1(a, ctx)
                                            : launch_gemv_fused_mode2(a, ctx));
    }
    unsigned char* act = static_cast<unsigned char*>(workspace);
    float* xd = reinterpret_cast<float*>(act + round_up(act_bytes(mode, rows, K), 256));
    cudaError_t e = launch_act_quant(mode, prod, h, res, s_out, rows, K, prod == 2 ? 0 : 1, gain, eps,
                                     act, xd, ctx);
    if (e != cudaSuccess) return cuda_fail(e);
    if (kv.k_cache) {
        // batches: the projection, then the K/V slices copied into the caches
        const q8_status st2 = project_dispatch(mode, q, s, N, K, act, mode == Q8_ACT_F32 ? nullptr : xd,
                                               rows, y, 0, ctx);
        if (st2 != Q8_OK) return st2;
        return launched(launch_kv_scatter(static_cast<const float*>(y), rows, N, kv.pos, kv.kv_col,
                                          kv.kv_dim, kv.n_pos, kv.k_cache, kv.v_cache, ctx));
    }
    return project_dispatch(mode, q, s, N, K, act, mode == Q8_ACT_F32 ? nullptr : xd, rows, y,
                            out_f64 ? 1 : 0, ctx);
}

q8_status q8_proj_fused(int mode, const int8_t* q, const uint16_t* s, int64_t N, int64_t K,
                        const float* h, int64_t rows, const float* gain, float eps, void* y,
                        int out_f64, void* workspace, size_t ws_bytes, void* stream) {
    return proj_fused_impl(mode, 0, q, s, N, K, h, nullptr, nullptr, rows, gain, eps, y, out_f64,
                           workspace, ws_bytes, stream);
}

q8_status q8_proj_fused_residual(int mode, const int8_t* q, const uint16_t* s, int64_t N, int64_t K,
                                 const float* h, const float* r, float* s_out, int64_t rows,
                                 const float* gain, float eps, void* y, int out_f64,
                                 void* workspace, size_t ws_bytes, void* stream) {
    if (!h) return Q8_ERR_ARG;
    if (rows < 1 || rows > Q8_MAX_ROWS) return Q8_ERR_SHAPE;
    const q8_status st = check_residual(h, r, s_out, rows, K);
    if (st != Q8_OK) return st;
    return proj_fused_impl(mode, 1, q, s, N, K, h, r, s_out, rows, gain, eps, y, out_f64, workspace,
                           ws_bytes, stream);
}

q8_status q8_proj_fused_kv(int mode, const int8_t* q, const uint16_t* s, int64_t N, int64_t K,
                           const float* h, int64_t rows, const float* gain, float eps, void* y,
                           const int32_t* pos, int64_t kv_col, int64_t kv_dim, float* k_cache,
                           float* v_cache, int64_t n_pos, void* workspace, size_t ws_bytes,
                           void* stream) {
    if (!pos || !k_cache || !v_cache) return Q8_ERR_ARG;
    if (rows < 1 || rows > Q8_MAX_ROWS) return Q8_ERR_SHAPE;
    if (kv_dim < 1 || kv_col < 0 || kv_dim > N / 2 || kv_col > N - 2 * kv_dim) return Q8_ERR_SHAPE;
    // positions are int32; a cache of more than 2^40 bytes exceeds any device
    if (n_pos < 1 || n_pos > INT32_MAX || kv_dim > (int64_t(1) << 38) / (rows * n_pos))
        return Q8_ERR_SHAPE;
    if (K > kFusedMaxK) return Q8_ERR_UNSUPPORTED;   // the decode kernel's K
    if (!aligned16(pos) || !aligned16(k_cache) || !aligned16(v_cache)) return Q8_ERR_ALIGN;
    const size_t cache = size_t(rows) * size_t(n_pos) * size_t(kv_dim) * sizeof(float);
    if (overlaps(k_cache, v_cache, cache)) return Q8_ERR_ARG;
    KvArgs kv;
    kv.pos = pos;
    kv.kv_col = kv_col;
    kv.kv_dim = kv_dim;
    kv.n_pos = n_pos;
    kv.k_cache = k_cache;
    kv.v_cache = v_cache;
    return proj_fused_impl(mode, 0, q, s, N, K, h, nullptr, nullptr, rows, gain, eps, y, 0, workspace,
                           ws_bytes, stream, kv);
}

q8_status q8_proj_fused_swiglu(int mode, const int8_t* q, const uint16_t* s, int64_t N, int64_t K,
                               const float* gu, int64_t rows, void* y, int out_f64, void* workspace,
                               size_t ws_bytes, void* stream) {
    return proj_fused_impl(mode, 2, q, s, N, K, gu, nullptr, nullptr, rows, nullptr, 0.0f, y, out_f64,
                           workspace, ws_bytes, stream);
}

size_t head_argmax_workspace(int64_t rows) {
    if (rows < 1) return 0;
    const int64_t g = rows < kArgmaxGroupRows ? rows : kArgmaxGroupRows;
    return kArgmaxGemvOff + kArgmaxHeader + size_t(kMaxGrid) * size_t(g) * sizeof(ArgmaxCand);
}

q8_status head_argmax(int mode, const int8_t* q, const uint16_t* s, int64_t N, int64_t K,
                      const void* xq, const float* xd, int64_t rows, int32_t* tok,
                      double* maxval, void* logits, void* workspace, size_t ws_bytes,
                      void* stream) {
    if (!valid_mode(mode)) return Q8_ERR_MODE;
    if (!q || !s || !xq || !tok || (mode != Q8_ACT_F32 && !xd)) return Q8_ERR_ARG;
    q8_status st = check_shape(N, K);
    if (st != Q8_OK) return st;
    if (rows < 1 || rows > Q8_MAX_ROWS) return Q8_ERR_SHAPE;
    if (!workspace || ws_bytes < head_argmax_workspace(rows)) return Q8_ERR_WORKSPACE;
    if (!aligned16(q) || !aligned16(s) || !aligned16(xq) || (xd && !aligned16(xd)) ||
        !aligned16(workspace) || (logits && !aligned16(logits)) ||
        (reinterpret_cast<uintptr_t>(tok) & 3u) || (reinterpret_cast<uintptr_t>(maxval) & 7u))
        return Q8_ERR_ALIGN;
    LaunchCtx ctx;
    if ((st = make_ctx(stream, ctx)) != Q8_OK) return st;
    static_assert(kArgmaxKeyBytes >= 8 * Q8_MAX_ROWS, "one arg-max key per row");
    // the tensor-core path from chunk_min_head_rows(mode) rows; in f32 mode up to
    // kArgmaxGroupRows rows and kMaxGrid tiles (its candidates use the
    // CUDA-core layout of the workspace)
    const bool f32_fits = mode != Q8_ACT_F32 || (rows <= kArgmaxGroupRows && (N + 127) / 128 <= kMaxGrid);
    // (f32 row pairs, where they fit, beat the tensor cores up to 7 rows)
    const int64_t min_rows =
        (mode == Q8_ACT_F32 && gemv_group_rows(mode, K) == 2) ? 8 : chunk_min_head_rows(mode);
    if (f32_fits && rows >= min_rows && chunk_supported(mode, N, K, rows))
        return launched(launch_chunk_argmax(mode, q, s, N, K, xq, xd, rows, logits, tok, maxval, workspace,
                                            ctx));
    return run_projection(mode, q, s, N, K, xq, xd, rows, logits, mode == Q8_ACT_F32 ? 1 : 0, tok,
                          maxval, static_cast<unsigned char*>(workspace) + kArgmaxGemvOff, ctx);
}

q8_status q8_debug_block_dots(int mode, const int8_t* q, const void* xq, int64_t N, int64_t K,
                              int64_t rows, int32_t* isum, int path, void* stream) {
    if (mode != Q8_ACT_I8 && mode != Q8_ACT_I8X2) return Q8_ERR_MODE;
    if (!q || !xq || !isum) return Q8_ERR_ARG;
    q8_status st = check_shape(N, K);
    if (st != Q8_OK) return st;
    if (rows < 1 || rows > Q8_MAX_ROWS) return Q8_ERR_SHAPE;
    if (rows * N * (K / Q8_QK) > (int64_t(1) << 26)) return Q8_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(xq) || !aligned16(isum)) return Q8_ERR_ALIGN;
    if (path != 0 && path != 1) return Q8_ERR_ARG;
    LaunchCtx ctx;
    if ((st = make_ctx(stream, ctx)) != Q8_OK) return st;
    if (path == 1) {
        if (!chunk_supported(mode, N, K, rows)) return Q8_ERR_UNSUPPORTED;
        return launched(launch_chunk_debug(mode, q, N, K, xq, rows, isum, ctx));
    }
    return launched(launch_debug_dots(mode, q, xq, N, K, rows, isum, ctx));
}

// ---------------------------------------------- the decode step's other operators

// Sizes of a K/V cache [rows][n_pos][kv_heads * dim]: what attn_decode and
// kv_evict take; *bytes receives one cache's size.
static q8_status check_cache(int kv_type, int64_t rows, int64_t n_pos, int64_t kv_heads, int64_t dim,
                             size_t* bytes) {
    if (kv_type < Q8_KV_F32 || kv_type > Q8_KV_BF16) return Q8_ERR_MODE;
    if (rows < 1 || rows > Q8_MAX_ROWS || n_pos < 1 || n_pos > INT32_MAX) return Q8_ERR_SHAPE;
    if (kv_heads < 1 || kv_heads > kMaxHeads || dim < 8 || dim > 256 || dim % 8) return Q8_ERR_SHAPE;
    const int64_t elt = kv_type == Q8_KV_F32 ? 4 : 2;
    // (in values, so that attn_decode_workspace, which is given no type, refuses the same)
    if (n_pos > (int64_t(1) << 39) / (rows * kv_heads * dim)) return Q8_ERR_SHAPE;
    *bytes = size_t(rows) * size_t(n_pos) * size_t(kv_heads * dim * elt);
    return Q8_OK;
}

// [a, a + na) and [b, b + nb) overlap (either NULL: no)
static bool overlaps2(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

static q8_status check_attn(int kv_type, int64_t rows, int64_t n_pos, int64_t heads, int64_t kv_heads,
                            int64_t dim, int64_t window, int64_t sinks, size_t* cache) {
    const q8_status st = check_cache(kv_type, rows, n_pos, kv_heads, dim, cache);
    if (st != Q8_OK) return st;
    if (heads < kv_heads || heads > kMaxHeads || heads % kv_heads) return Q8_ERR_SHAPE;
    if (window < -1 || sinks < 0) return Q8_ERR_SHAPE;
    return Q8_OK;
}

size_t attn_decode_workspace(int64_t rows, int64_t heads, int64_t kv_heads, int64_t head_dim,
                             int64_t n_pos, int64_t window, int64_t sinks, int with_acc) {
    size_t cache;
    if (check_attn(Q8_KV_F16, rows, n_pos, heads, kv_heads, head_dim, window, sinks, &cache) != Q8_OK)
        return 0;
    return attn_workspace_bytes(rows, heads, kv_heads, head_dim, n_pos, window, sinks, with_acc != 0, false);
}

q8_status attn_decode(const float* q, int64_t ldq, const void* k_cache, const void* v_cache,
                      int kv_type, int64_t rows, int64_t n_pos, int64_t heads, int64_t kv_heads,
                      int64_t head_dim, const int32_t* pos, int64_t window, int64_t sinks,
                      float scale, float* out, int64_t ldo, float* acc, void* workspace,
                      size_t ws_bytes, void* stream) {
    if (!q || !k_cache || !v_cache || !pos || !out) return Q8_ERR_ARG;
    size_t cache;
    q8_status st = check_attn(kv_type, rows, n_pos, heads, kv_heads, head_dim, window, sinks, &cache);
    if (st != Q8_OK) return st;
    const int64_t width = heads * head_dim, max_ld = int64_t(1) << 31;
    if (ldq < width || ldo < width || ldq > max_ld || ldo > max_ld) return Q8_ERR_SHAPE;
    // (its product with log2(e) is to be a normal binary32)
    if (scale != 0.0f && !(fabsf(scale) >= FLT_MIN && fabsf(scale) <= 0x1p127f)) return Q8_ERR_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(pos) ||
        !aligned16(out) || (acc && !aligned16(acc)))
        return Q8_ERR_ALIGN;
    const size_t qn = size_t((rows - 1) * ldq + width) * 4, on = size_t((rows - 1) * ldo + width) * 4;
    const size_t an = size_t(rows * kv_heads) * size_t(n_pos) * 4, pn = size_t(rows) * 4;
    if (overlaps2(out, on, q, qn) || overlaps2(out, on, k_cache, cache) ||
        overlaps2(out, on, v_cache, cache) || overlaps2(out, on, acc, an) || overlaps2(out, on, pos, pn) ||
        overlaps2(acc, an, q, qn) || overlaps2(acc, an, k_cache, cache) ||
        overlaps2(acc, an, v_cache, cache) || overlaps2(acc, an, pos, pn))
        return Q8_ERR_ARG;
    const size_t wn =
        attn_workspace_bytes(rows, heads, kv_heads, head_dim, n_pos, window, sinks, acc != nullptr, false);
    if (!workspace || ws_bytes < wn) return Q8_ERR_WORKSPACE;
    if (!aligned16(workspace)) return Q8_ERR_ALIGN;
    if (overlaps2(workspace, wn, q, qn) || overlaps2(workspace, wn, k_cache, cache) ||
        overlaps2(workspace, wn, v_cache, cache) || overlaps2(workspace, wn, pos, pn) ||
        overlaps2(workspace, wn, out, on) || overlaps2(workspace, wn, acc, an))
        return Q8_ERR_ARG;
    LaunchCtx ctx;
    if ((st = make_ctx(stream, ctx)) != Q8_OK) return st;
    const AttnArgs a{q,   ldq,    k_cache, v_cache, kv_type, rows, n_pos, heads, kv_heads, head_dim,
                     pos, window, sinks,   scale,   out,     ldo,  acc,   workspace};
    return launched(launch_attn(a, ctx));
}

size_t kv_evict_workspace(int64_t rows, int64_t kv_heads, int64_t budget) {
    if (rows < 1 || rows > Q8_MAX_ROWS || kv_heads < 1 || kv_heads > kMaxHeads || budget < 1 ||
        budget > INT32_MAX)
        return 0;
    return evict_workspace_bytes(rows, kv_heads, budget);
}

q8_status kv_evict(void* k_cache, void* v_cache, int kv_type, int64_t rows, int64_t n_pos,
                   int64_t kv_heads, int64_t head_dim, const int32_t* pos, const float* acc,
                   int64_t budget, int64_t sinks, int64_t recent, int32_t* new_pos, float* new_acc,
                   int32_t* kept, void* workspace, size_t ws_bytes, void* stream) {
    if (!k_cache || !v_cache || !pos || !acc || !new_pos || !new_acc) return Q8_ERR_ARG;
    size_t cache;
    q8_status st = check_cache(kv_type, rows, n_pos, kv_heads, head_dim, &cache);
    if (st != Q8_OK) return st;
    if (budget < 1 || budget > n_pos || sinks < 0 || recent < 0 || sinks > budget ||
        recent > budget - sinks)
        return Q8_ERR_SHAPE;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(pos) || !aligned16(acc) ||
        !aligned16(new_pos) || !aligned16(new_acc) || (kept && !aligned16(kept)))
        return Q8_ERR_ALIGN;
    const size_t an = size_t(rows * kv_heads) * size_t(n_pos) * 4, pn = size_t(rows) * 4;
    const size_t kn = size_t(rows * kv_heads) * size_t(budget) * 4;
    const size_t wn = evict_workspace_bytes(rows, kv_heads, budget);
    if (!workspace || ws_bytes < wn) return Q8_ERR_WORKSPACE;
    if (!aligned16(workspace)) return Q8_ERR_ALIGN;
    // every buffer that is written is disjoint from every other one
    const struct { const void* p; size_t n; bool written; } b[] = {
        {k_cache, cache, true}, {v_cache, cache, true}, {pos, pn, false}, {acc, an, false},
        {new_pos, pn, true},    {new_acc, an, true},    {kept, kn, true}, {workspace, wn, true}};
    for (int i = 0; i < 8; ++i)
        for (int j = 0; j < i; ++j) {
            if (!b[i].written && !b[j].written) continue;
            if ((i == 4 && j == 2 && new_pos == pos) || (i == 5 && j == 3 && new_acc == acc)) continue;
            if (overlaps2(b[i].p, b[i].n, b[j].p, b[j].n)) return Q8_ERR_ARG;
        }
    LaunchCtx ctx;
    if ((st = make_ctx(stream, ctx)) != Q8_OK) return st;
    const EvictArgs a{k_cache, v_cache, kv_type, rows,    n_pos,   kv_heads, head_dim, pos,
                      acc,     budget,  sinks,   recent,  new_pos, new_acc,  kept,     workspace};
    return launched(launch_evict(a, ctx));
}

q8_status head_sample(const float* logits, int64_t ldl, int64_t rows, int64_t N, const float* u,
                      const float* temperature, const int32_t* top_k, const float* top_p,
                      const float* min_p, int32_t* tok, float* prob, int32_t* kept, void* stream) {
    if (!logits || !u || !tok) return Q8_ERR_ARG;
    if (rows < 1 || rows > Q8_MAX_ROWS || N < 1 || N > kSampleMaxN || ldl < N ||
        ldl > (int64_t(1) << 31))
        return Q8_ERR_SHAPE;
    const void* per_row[] = {u, temperature, top_k, top_p, min_p, tok, prob, kept};
    for (const void* p : per_row)
        if (reinterpret_cast<uintptr_t>(p) & 3u) return Q8_ERR_ALIGN;
    if (!aligned16(logits)) return Q8_ERR_ALIGN;
    // every output is disjoint from every other buffer: a row's first CTA may write its
    // results while the others have not read the row's settings yet
    const size_t rn = size_t(rows) * 4;
    for (int i = 5; i < 8; ++i) {
        if (overlaps2(per_row[i], rn, logits, size_t((rows - 1) * ldl + N) * 4)) return Q8_ERR_ARG;
        for (int j = 0; j < i; ++j)
            if (overlaps2(per_row[i], rn, per_row[j], rn)) return Q8_ERR_ARG;
    }
    LaunchCtx ctx;
    q8_status st = make_ctx(stream, ctx);
    if (st != Q8_OK) return st;
    const SampleArgs a{logits, ldl, rows, N, u, temperature, top_k, top_p, min_p, tok, prob, kept};
    return launched(launch_sample(a, ctx));
}

// ------------------------------------------------------------ quantised K/V caches

namespace {

// A buffer of a call and whether the call writes it.
struct Span {
    const void* p;
    size_t n;
    bool written;
};

// A written buffer among these overlaps another one.
bool any_overlap(const Span* b, int n) {
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < i; ++j)
            if ((b[i].written || b[j].written) && overlaps2(b[i].p, b[i].n, b[j].p, b[j].n)) return true;
    return false;
}

// Sizes of a quantised cache; *codes and *words receive the bytes of one plane of each.
q8_status check_kvq(int kind, int64_t rows, int64_t n_pos, int64_t kv_heads, int64_t dim, size_t* codes,
                    size_t* words) {
    if (kind != Q8_KVQ_I8 && kind != Q8_KVQ_U4) return Q8_ERR_MODE;
    if (dim % Q8_QK) return Q8_ERR_SHAPE;
    size_t n;
    const q8_status st = check_cache(Q8_KV_F16, rows, n_pos, kv_heads, dim, &n);
    if (st != Q8_OK) return st;
    *codes = kind == Q8_KVQ_I8 ? n / 2 : n / 4;
    *words = n / 16;
    return Q8_OK;
}

// What kvq_store reads and kvq_load writes: one of K's and V's floats.
q8_status check_floats(int type, int64_t rows, int64_t T, int64_t width, int64_t ld_row, int64_t ld_tok, bool written,
                       size_t* bytes) {
    if (type < Q8_KV_F32 || type > Q8_KV_BF16) return Q8_ERR_MODE;
    const int64_t elt = type == Q8_KV_F32 ? 4 : 2, most = int64_t(1) << 40;
    if (T < 1 || T > INT32_MAX) return Q8_ERR_SHAPE;
    if ((T > 1 && (ld_tok < width || ld_tok > most / T)) || (rows > 1 && (ld_row < width || ld_row > most / rows)))
        return Q8_ERR_SHAPE;
    if ((T > 1 && ld_tok * elt % 16) || (rows > 1 && ld_row * elt % 16)) return Q8_ERR_ALIGN;
    const int64_t tokens = T > 1 ? (T - 1) * ld_tok : 0, all = rows > 1 ? (rows - 1) * ld_row : 0;
    // (rows that are written lie behind one another, or between one another's tokens)
    if (written && T > 1 && rows > 1 && ld_row < tokens + width && ld_tok < all + width) return Q8_ERR_SHAPE;
    *bytes = size_t(tokens + all + width) * size_t(elt);
    return Q8_OK;
}

// What kvq_load writes of K, and again of V: runs of n bytes, an inner line of them, those lines one
// behind another (check_floats' two orders of rows and tokens).
struct Runs {
    int64_t n, inner, inners, outer, outers;
};

Runs float_runs(int64_t elt, int64_t rows, int64_t T, int64_t width, int64_t ld_row, int64_t ld_tok) {
    const int64_t row = rows > 1 ? ld_row * elt : 1, tok = T > 1 ? ld_tok * elt : 1;   // (a stride of one says nothing)
    return row < tok ? Runs{width * elt, row, rows, tok, T} : Runs{width * elt, tok, T, row, rows};
}

int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }

// Whether one of the runs from a on overlaps [b, b + nb), or, with again, one of the same runs from b on:
// whether some o * outer + i * inner lies in [lo, hi].  Lines have gaps, so a line may reach over
// that interval and miss it, but only the few at its ends do.
bool runs_overlap(const Runs& r, const void* a, const void* b, int64_t nb, bool again) {
    const int64_t d = int64_t(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
    const int64_t lo = d - r.n + 1, hi = d + nb - 1, i0 = again ? 1 - r.inners : 0, o0 = again ? 1 - r.outers : 0;
    const int64_t first = -floor_div((r.inners - 1) * r.inner - lo, r.outer), last = floor_div(hi - i0 * r.inner, r.outer);
    for (int64_t o = first < o0 ? o0 : first; o <= last && o < r.outers; ++o) {
        const int64_t from = -floor_div(o * r.outer - lo, r.inner), to = floor_div(hi - o * r.outer, r.inner);
        if ((from < i0 ? i0 : from) <= (to < r.inners ? to : r.inners - 1)) return true;
    }
    return false;
}

q8_status kvq_io(bool store, void* k, void* v, int type, int64_t ld_row, int64_t ld_tok, int64_t rows, int64_t T,
                 int64_t kv_heads, int64_t dim, const int32_t* pos, const int32_t* lens, int kind, void* k_codes,
                 void* k_words, void* v_codes, void* v_words, int64_t n_pos, void* stream) {
    if (!k || !v || (store && !pos) || !k_codes || !k_words || !v_codes || !v_words) return Q8_ERR_ARG;
    size_t codes, words, floats;
    q8_status st = check_kvq(kind, rows, n_pos, kv_heads, dim, &codes, &words);
    if (st != Q8_OK) return st;
    if ((st = check_floats(type, rows, T, kv_heads * dim, ld_row, ld_tok, !store, &floats)) != Q8_OK) return st;
    const void* all[] = {k, v, pos, lens, k_codes, k_words, v_codes, v_words};
    for (const void* p : all)
        if (!aligned16(p)) return Q8_ERR_ALIGN;
    const size_t pn = size_t(rows) * 4;
    const Span b[] = {{k, floats, !store},     {v, floats, !store},     {pos, pn, false},        {lens, pn, false},
                      {k_codes, codes, store}, {k_words, words, store}, {v_codes, codes, store}, {v_words, words, store}};
    if (store) {
        if (any_overlap(b, sizeof(b) / sizeof(b[0]))) return Q8_ERR_ARG;
    } else {
        // K and V that are written may be columns of the same rows, and anything may lie between their runs
        const Runs r = float_runs(type == Q8_KV_F32 ? 4 : 2, rows, T, kv_heads * dim, ld_row, ld_tok);
        if (runs_overlap(r, k, v, r.n, true)) return Q8_ERR_ARG;
        for (const Span& x : b)
            if (x.p && !x.written && (runs_overlap(r, k, x.p, int64_t(x.n), false) || runs_overlap(r, v, x.p, int64_t(x.n), false)))
                return Q8_ERR_ARG;
    }
    LaunchCtx ctx;
    if ((st = make_ctx(stream, ctx)) != Q8_OK) return st;
    const KvqIoArgs a{k,    v,    type, ld_row,  ld_tok,  rows,    T,       kv_heads, dim,
                      pos,  lens, kind, k_codes, k_words, v_codes, v_words, n_pos};
    return launched(store ? launch_kvq_store(a, ctx) : launch_kvq_load(a, ctx));
}

}  // namespace

q8_status kvq_store(const void* k, const void* v, int src_type, int64_t ld_row, int64_t ld_tok, int64_t rows, int64_t T,
                    int64_t kv_heads, int64_t head_dim, const int32_t* pos, const int32_t* lens, int kvq_type,
                    void* k_codes, void* k_words, void* v_codes, void* v_words, int64_t n_pos, void* stream) {
    return kvq_io(true, const_cast<void*>(k), const_cast<void*>(v), src_type, ld_row, ld_tok, rows, T, kv_heads, head_dim,
                  pos, lens, kvq_type, k_codes, k_words, v_codes, v_words, n_pos, stream);
}

q8_status kvq_load(int kvq_type, const void* k_codes, const void* k_words, const void* v_codes, const void* v_words,
                   int64_t rows, int64_t n_pos, int64_t kv_heads, int64_t head_dim, const int32_t* pos, int64_t T,
                   const int32_t* lens, int dst_type, void* k, void* v, int64_t ld_row, int64_t ld_tok, void* stream) {
    return kvq_io(false, k, v, dst_type, ld_row, ld_tok, rows, T, kv_heads, head_dim, pos, lens, kvq_type,
                  const_cast<void*>(k_codes), const_cast<void*>(k_words), const_cast<void*>(v_codes),
                  const_cast<void*>(v_words), n_pos, stream);
}

static q8_status check_kvq_attn(int kind, int64_t rows, int64_t n_pos, int64_t heads, int64_t kv_heads, int64_t dim,
                                int64_t window, int64_t sinks, size_t* codes, size_t* words) {
    const q8_status st = check_kvq(kind, rows, n_pos, kv_heads, dim, codes, words);
    if (st != Q8_OK) return st;
    size_t n;
    return check_attn(Q8_KV_F16, rows, n_pos, heads, kv_heads, dim, window, sinks, &n);
}

size_t kvq_attn_decode_workspace(int64_t rows, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t n_pos,
                                 int64_t window, int64_t sinks, int with_acc) {
    size_t codes, words;
    if (check_kvq_attn(Q8_KVQ_I8, rows, n_pos, heads, kv_heads, head_dim, window, sinks, &codes, &words) != Q8_OK)
        return 0;
    return attn_workspace_bytes(rows, heads, kv_heads, head_dim, n_pos, window, sinks, with_acc != 0, true);
}

q8_status kvq_attn_decode(const float* q, int64_t ldq, int kvq_type, const void* k_codes, const void* k_words,
                          const void* v_codes, const void* v_words, int64_t rows, int64_t n_pos, int64_t heads,
                          int64_t kv_heads, int64_t head_dim, const int32_t* pos, int64_t window, int64_t sinks,
                          float scale, float* out, int64_t ldo, float* acc, void* workspace, size_t ws_bytes,
                          void* stream) {
    if (!q || !k_codes || !k_words || !v_codes || !v_words || !pos || !out) return Q8_ERR_ARG;
    size_t codes, words;
    q8_status st = check_kvq_attn(kvq_type, rows, n_pos, heads, kv_heads, head_dim, window, sinks, &codes, &words);
    if (st != Q8_OK) return st;
    const int64_t width = heads * head_dim, max_ld = int64_t(1) << 31;
    if (ldq < width || ldo < width || ldq > max_ld || ldo > max_ld) return Q8_ERR_SHAPE;
    if (scale != 0.0f && !(fabsf(scale) >= FLT_MIN && fabsf(scale) <= 0x1p127f)) return Q8_ERR_ARG;   // (as attn_decode)
    const void* all[] = {q, k_codes, k_words, v_codes, v_words, pos, out, acc};
    for (const void* p : all)
        if (!aligned16(p)) return Q8_ERR_ALIGN;
    const size_t wn =
        attn_workspace_bytes(rows, heads, kv_heads, head_dim, n_pos, window, sinks, acc != nullptr, true);
    const Span b[] = {{q, size_t((rows - 1) * ldq + width) * 4, false}, {out, size_t((rows - 1) * ldo + width) * 4, true},
                      {acc, size_t(rows * kv_heads) * size_t(n_pos) * 4, true}, {pos, size_t(rows) * 4, false},
                      {k_codes, codes, false}, {k_words, words, false}, {v_codes, codes, false}, {v_words, words, false}};
    if (any_overlap(b, sizeof(b) / sizeof(b[0]))) return Q8_ERR_ARG;
    if (!workspace || ws_bytes < wn) return Q8_ERR_WORKSPACE;
    if (!aligned16(workspace)) return Q8_ERR_ALIGN;
    for (const Span& s : b)
        if (overlaps2(workspace, wn, s.p, s.n)) return Q8_ERR_ARG;
    LaunchCtx ctx;
    if ((st = make_ctx(stream, ctx)) != Q8_OK) return st;
    const AttnArgs a{q,      ldq,   k_codes, v_codes, kKvQuantised + kvq_type,
                     rows,   n_pos, heads,   kv_heads, head_dim, pos, window, sinks, scale, out, ldo, acc, workspace,
                     static_cast<const uint32_t*>(k_words), static_cast<const uint32_t*>(v_words)};
    return launched(launch_attn(a, ctx));
}

size_t kvq_evict_workspace(int64_t rows, int64_t kv_heads, int64_t budget) {
    return kv_evict_workspace(rows, kv_heads, budget);
}

q8_status kvq_evict(int kvq_type, void* k_codes, void* k_words, void* v_codes, void* v_words, int64_t rows,
                    int64_t n_pos, int64_t kv_heads, int64_t head_dim, const int32_t* pos, const float* acc,
                    int64_t budget, int64_t sinks, int64_t recent, int32_t* new_pos, float* new_acc, int32_t* kept,
                    void* workspace, size_t ws_bytes, void* stream) {
    if (!k_codes || !k_words || !v_codes || !v_words || !pos || !acc || !new_pos || !new_acc) return Q8_ERR_ARG;
    size_t codes, words;
    q8_status st = check_kvq(kvq_type, rows, n_pos, kv_heads, head_dim, &codes, &words);
    if (st != Q8_OK) return st;
    if (budget < 1 || budget > n_pos || sinks < 0 || recent < 0 || sinks > budget || recent > budget - sinks)
        return Q8_ERR_SHAPE;
    const void* all[] = {k_codes, k_words, v_codes, v_words, pos, acc, new_pos, new_acc, kept};
    for (const void* p : all)
        if (!aligned16(p)) return Q8_ERR_ALIGN;
    const size_t an = size_t(rows * kv_heads) * size_t(n_pos) * 4, pn = size_t(rows) * 4;
    const size_t wn = evict_workspace_bytes(rows, kv_heads, budget);
    if (!workspace || ws_bytes < wn) return Q8_ERR_WORKSPACE;
    if (!aligned16(workspace)) return Q8_ERR_ALIGN;
    // (in place: the old one counts as the new)
    const Span b[] = {{k_codes, codes, true}, {k_words, words, true}, {v_codes, codes, true}, {v_words, words, true},
                      {new_pos == pos ? nullptr : pos, pn, false},    {new_acc == acc ? nullptr : acc, an, false},
                      {new_pos, pn, true},    {new_acc, an, true},
                      {kept, size_t(rows * kv_heads) * size_t(budget) * 4, true}, {workspace, wn, true}};
    if (any_overlap(b, sizeof(b) / sizeof(b[0]))) return Q8_ERR_ARG;
    LaunchCtx ctx;
    if ((st = make_ctx(stream, ctx)) != Q8_OK) return st;
    const EvictArgs a{k_codes, v_codes, kKvQuantised + kvq_type, rows,    n_pos,   kv_heads, head_dim, pos,
                      acc,     budget,  sinks, recent, new_pos, new_acc, kept, workspace,
                      static_cast<uint32_t*>(k_words), static_cast<uint32_t*>(v_words)};
    return launched(launch_evict(a, ctx));
}

}  // extern "C"
