// q8_api.cu -- the C ABI of libq8: argument checks (host only, before any
// CUDA call), device checks, and dispatch to the kernels.
#include <mutex>

#include <algorithm>

#include "q8_internal.h"

namespace q8 {

namespace {
constexpr int kMaxDevices = 64;
DeviceInfo g_info[kMaxDevices];
std::once_flag g_once[kMaxDevices];
int g_ok[kMaxDevices];

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
}  // namespace

const DeviceInfo *device_info() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::call_once(g_once[dev], [dev]() {
        DeviceInfo &d = g_info[dev];
        d.device = dev;
        g_ok[dev] = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
                    cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev) == cudaSuccess &&
                    cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, dev) == cudaSuccess;
    });
    return g_ok[dev] ? &g_info[dev] : nullptr;
}

q8_status check_arch(const DeviceInfo **out) {
    const DeviceInfo *di = device_info();
    if (!di) return Q8_ERR_CUDA;
    if (di->cc_major != 10 || di->cc_minor != 3) return Q8_ERR_ARCH;
    *out = di;
    return Q8_OK;
}

static q8_status check_weights(const int8_t *q, const uint16_t *s, int64_t N, int64_t K) {
    if (N < 0 || K <= 0 || (K % 32) != 0 || N > INT32_MAX || K > INT32_MAX) return Q8_ERR_SHAPE;
    if (N == 0) return Q8_OK;
    if (!q || !s) return Q8_ERR_ARG;
    if (!aligned(q, 16) || !aligned(s, 16)) return Q8_ERR_ALIGN;
    return Q8_OK;
}

static q8_status check_desc(const q8_linear_desc &d, int32_t M) {
    q8_status st = check_weights(d.q, d.s, d.N, d.K);
    if (st != Q8_OK) return st;
    if (d.N == 0) return Q8_OK;
    if (!d.x || !d.y) return Q8_ERR_ARG;
    if (d.ldx < d.K || (M > 1 && d.ldy < d.N) || d.ldy < 1) return Q8_ERR_SHAPE;
    if (!aligned(d.x, 16) || (d.ldx % 8) != 0 || !aligned(d.y, 4)) return Q8_ERR_ALIGN;
    return Q8_OK;
}

// Host-only argument check of one skinny matmul (no CUDA call).
q8_status check_skinny_args(const q8_linear_desc &d, int32_t M) {
    if (M < 0 || M > Q8_SKINNY_MAX_M) return Q8_ERR_SHAPE;
    return check_desc(d, M);
}

}  // namespace q8

using namespace q8;

extern "C" {

int32_t q8_abi_version(void) { return Q8_ABI_VERSION; }

const char *q8_status_str(q8_status st) {
    switch (st) {
        case Q8_OK: return "ok";
        case Q8_ERR_ARG: return "invalid argument (null pointer or bad count)";
        case Q8_ERR_ALIGN: return "misaligned pointer or leading dimension";
        case Q8_ERR_SHAPE: return "bad shape (K must be a positive multiple of 32; check M and leading dimensions)";
        case Q8_ERR_WORKSPACE: return "workspace missing or too small";
        case Q8_ERR_ARCH: return "current device is not sm_103 (GB300)";
        case Q8_ERR_CUDA: return "CUDA runtime error";
        case Q8_ERR_UNSUPPORTED: return "not supported by this build";
    }
    return "unknown status";
}

q8_status q8_quantize_rows(const float *w, int64_t rows, int64_t K, int8_t *q, uint16_t *s,
                           uint32_t *dev_status, q8_stream_t stream) {
    return q8_quantize_rows_ex(w, rows, K, q, s, Q8_QUANT_EXACT, dev_status, stream);
}

q8_status q8_quantize_rows_ex(const float *w, int64_t rows, int64_t K, int8_t *q, uint16_t *s, int32_t mode,
                              uint32_t *dev_status, q8_stream_t stream) {
    if (mode != Q8_QUANT_EXACT && mode != Q8_QUANT_FL32) return Q8_ERR_ARG;
    if (rows < 0 || K <= 0 || (K % 32) != 0) return Q8_ERR_SHAPE;
    if (rows == 0) return Q8_OK;
    if (!w || !q || !s) return Q8_ERR_ARG;
    if (!aligned(w, 16) || !aligned(q, 16) || !aligned(s, 16)) return Q8_ERR_ALIGN;
    if (dev_status && !aligned(dev_status, 4)) return Q8_ERR_ALIGN;
    const DeviceInfo *di;
    q8_status st = check_arch(&di);
    if (st != Q8_OK) return st;
    return launch_quantize(w, rows, K, q, s, dev_status, reinterpret_cast<cudaStream_t>(stream), mode);
}

q8_status q8_gguf_to_planar(const void *blocks, int64_t rows, int64_t K, int8_t *q, uint16_t *s,
                            q8_stream_t stream) {
    if (rows < 0 || K <= 0 || (K % 32) != 0) return Q8_ERR_SHAPE;
    if (rows == 0) return Q8_OK;
    if (!blocks || !q || !s) return Q8_ERR_ARG;
    if (!aligned(blocks, 16) || !aligned(q, 16) || !aligned(s, 16)) return Q8_ERR_ALIGN;
    if (rows > INT64_MAX / K) return Q8_ERR_SHAPE;
    const DeviceInfo *di;
    q8_status st = check_arch(&di);
    if (st != Q8_OK) return st;
    return launch_gguf_ingest(blocks, rows * (K / 32), q, s, reinterpret_cast<cudaStream_t>(stream));
}

q8_status q8_planar_to_gguf(const int8_t *q, const uint16_t *s, int64_t rows, int64_t K, void *blocks,
                            q8_stream_t stream) {
    if (rows < 0 || K <= 0 || (K % 32) != 0) return Q8_ERR_SHAPE;
    if (rows == 0) return Q8_OK;
    if (!blocks || !q || !s) return Q8_ERR_ARG;
    if (!aligned(blocks, 16) || !aligned(q, 16) || !aligned(s, 16)) return Q8_ERR_ALIGN;
    if (rows > INT64_MAX / K) return Q8_ERR_SHAPE;
    const DeviceInfo *di;
    q8_status st = check_arch(&di);
    if (st != Q8_OK) return st;
    return launch_gguf_export(q, s, rows * (K / 32), blocks, reinterpret_cast<cudaStream_t>(stream));
}

q8_status q8_selftest_wait_timeout(uint64_t limit_ns, uint32_t *dev_status, uint64_t *dev_elapsed_ns,
                                   q8_stream_t stream) {
    if (limit_ns == 0 || limit_ns > 1000000000ull) return Q8_ERR_ARG;
    if (dev_status && !aligned(dev_status, 4)) return Q8_ERR_ALIGN;
    if (dev_elapsed_ns && !aligned(dev_elapsed_ns, 8)) return Q8_ERR_ALIGN;
    const DeviceInfo *di;
    q8_status st = check_arch(&di);
    if (st != Q8_OK) return st;
    return launch_selftest_wait_timeout(limit_ns, dev_status, dev_elapsed_ns, reinterpret_cast<cudaStream_t>(stream));
}

size_t q8_stream_read_out_words(void) {
    const DeviceInfo *di = device_info();
    return di ? static_cast<size_t>(stream_read_grid(di)) : 0;
}

q8_status q8_stream_read(const void *src, size_t bytes, uint32_t *out, q8_stream_t stream) {
    if (bytes == 0) return Q8_OK;
    if (!src || !out) return Q8_ERR_ARG;
    if (!aligned(src, 16) || (bytes % 16) != 0 || !aligned(out, 4)) return Q8_ERR_ALIGN;
    const DeviceInfo *di;
    q8_status st = check_arch(&di);
    if (st != Q8_OK) return st;
    return launch_stream_read(src, bytes, out, reinterpret_cast<cudaStream_t>(stream));
}

size_t q8_workspace_size(int64_t N, int64_t K, int32_t M) {
    if (N <= 0 || K <= 0 || (K % 32) != 0 || M < 1 || M > Q8_SKINNY_MAX_M) return 0;
    q8_linear_desc d{};
    d.N = N;
    d.K = K;
    SplitPlan pl;
    size_t sched_off;
    return skinny_workspace(&d, 1, M, &pl, &sched_off);
}

size_t q8_linear_batch_workspace_size_ex(const q8_linear_desc *descs, int32_t count, int32_t M, int32_t variant) {
    if (variant != Q8_VARIANT_W8A8 && variant != Q8_VARIANT_BATCH_INVARIANT)
        return q8_linear_batch_workspace_size(descs, count, M);
    if (!descs || count < 1 || count > Q8_MAX_BATCH || M < 1 || M > Q8_SKINNY_MAX_M) return 0;
    q8_linear_desc tmp[Q8_MAX_BATCH];
    int n = 0;
    if (variant == Q8_VARIANT_BATCH_INVARIANT) {
        // the general kernel's partial sums for the matrices off the 256 grid
        for (int i = 0; i < count; ++i)
            if (descs[i].N > 0 && descs[i].K > 0 && descs[i].K % 256) tmp[n++] = descs[i];
        SplitPlan pl[Q8_MAX_BATCH];
        return n > 0 ? plan_skinny(tmp, n, M, pl, true) : 0;
    }
    for (int i = 0; i < count; ++i) {
        if (descs[i].N <= 0 || descs[i].K <= 0 || descs[i].K % 32) continue;
        tmp[n++] = descs[i];
    }
    return n > 0 ? w8a8_workspace(tmp, n, M) : 0;
}

size_t q8_linear_batch_workspace_size(const q8_linear_desc *descs, int32_t count, int32_t M) {
    if (!descs || count < 1 || count > Q8_MAX_BATCH || M < 1 || M > Q8_SKINNY_MAX_M) return 0;
    q8_linear_desc tmp[Q8_MAX_BATCH];
    int n = 0;
    for (int i = 0; i < count; ++i) {
        if (descs[i].N <= 0 || descs[i].K <= 0 || descs[i].K % 32) continue;
        tmp[n++] = descs[i];
    }
    if (n == 0) return 0;
    SplitPlan pl[Q8_MAX_BATCH];
    size_t sched_off;
    return skinny_workspace(tmp, n, M, pl, &sched_off);
}

namespace {

q8_status linear_batch(const q8_linear_desc *descs, int32_t count, int32_t M, int32_t variant, void *ws,
                       size_t ws_bytes, uint32_t *dev_status, q8_stream_t stream, bool chained) {
    if (!descs || count < 0 || count > Q8_MAX_BATCH) return Q8_ERR_ARG;
    if (variant < Q8_VARIANT_AUTO || variant > Q8_VARIANT_W8A8) return Q8_ERR_ARG;
    if (M < 0 || M > Q8_SKINNY_MAX_M) return Q8_ERR_SHAPE;
    if (dev_status && !aligned(dev_status, 4)) return Q8_ERR_ALIGN;
    // drop empty matrices; check the rest
    q8_linear_desc live[Q8_MAX_BATCH];
    int n = 0;
    for (int i = 0; i < count; ++i) {
        q8_status st = check_desc(descs[i], M);
        if (st != Q8_OK) return st;
        if (descs[i].N > 0) live[n++] = descs[i];
    }
    if (M == 0 || n == 0) return Q8_OK;
    const DeviceInfo *di;
    q8_status st = check_arch(&di);
    if (st != Q8_OK) return st;
    return launch_skinny(live, n, M, variant, ws, ws_bytes, dev_status, reinterpret_cast<cudaStream_t>(stream),
                         chained);
}

}  // namespace

q8_status q8_linear_batch_ex(const q8_linear_desc *descs, int32_t count, int32_t M, int32_t variant,
                             void *ws, size_t ws_bytes, uint32_t *dev_status, q8_stream_t stream) {
    return linear_batch(descs, count, M, variant, ws, ws_bytes, dev_status, stream, false);
}

q8_status q8_linear_batch_chained(const q8_linear_desc *descs, int32_t count, int32_t M, void *ws,
                                  size_t ws_bytes, uint32_t *dev_status, q8_stream_t stream) {
    return linear_batch(descs, count, M, Q8_VARIANT_AUTO, ws, ws_bytes, dev_status, stream, true);
}

q8_status q8_linear_chain(const q8_chain_step *steps, int32_t count, int32_t M, void *ws, size_t ws_bytes,
                          uint32_t *dev_status, q8_stream_t stream) {
    q8_status st = check_chain(steps, count, M);
    if (st != Q8_OK) return st;
    if (dev_status && !aligned(dev_status, 4)) return Q8_ERR_ALIGN;
    const size_t need = chain_workspace(steps, count, M);
    if (need > 0 && (ws == nullptr || ws_bytes < need)) return Q8_ERR_WORKSPACE;
    if (need > 0 && !aligned(ws, 256)) return Q8_ERR_ALIGN;
    const DeviceInfo *di;
    st = check_arch(&di);
    if (st != Q8_OK) return st;
    return launch_chain(steps, count, M, ws, ws_bytes, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

size_t q8_linear_chain_workspace_size(const q8_chain_step *steps, int32_t count, int32_t M) {
    if (check_chain(steps, count, M) != Q8_OK) return 0;
    return chain_workspace(steps, count, M);
}

q8_status q8_linear_batch(const q8_linear_desc *descs, int32_t count, int32_t M,
                          void *ws, size_t ws_bytes, uint32_t *dev_status, q8_stream_t stream) {
    return q8_linear_batch_ex(descs, count, M, Q8_VARIANT_AUTO, ws, ws_bytes, dev_status, stream);
}

q8_status q8_gemm_skinny(const int8_t *q, const uint16_t *s, int64_t N, int64_t K,
                         const uint16_t *x, int64_t ldx, int32_t M, float *y, int64_t ldy,
                         void *ws, size_t ws_bytes, uint32_t *dev_status, q8_stream_t stream) {
    q8_linear_desc d;
    d.q = q;
    d.s = s;
    d.x = x;
    d.y = y;
    d.N = N;
    d.K = K;
    d.ldx = ldx;
    d.ldy = ldy;
    return q8_linear_batch_ex(&d, 1, M, Q8_VARIANT_AUTO, ws, ws_bytes, dev_status, stream);
}

extern "C++" {
namespace {

// q8_gemm_w8a8's launches: the full 32-row slices of x in groups of at most
// Q8_MAX_BATCH (one q8_linear_batch launch each, the slices as matrices that
// share the weights), then the remaining rows.
template <typename F>
q8_status for_w8a8_launches(const q8_linear_desc &d, int32_t M, F &&f) {
    q8_linear_desc descs[Q8_MAX_BATCH];
    const int32_t full = M / Q8_SKINNY_MAX_M;
    for (int32_t b = 0; b < full; b += Q8_MAX_BATCH) {
        const int32_t cnt = std::min<int32_t>(Q8_MAX_BATCH, full - b);
        for (int32_t j = 0; j < cnt; ++j) {
            descs[j] = d;
            descs[j].x = d.x + static_cast<int64_t>(b + j) * Q8_SKINNY_MAX_M * d.ldx;
            descs[j].y = d.y + static_cast<int64_t>(b + j) * Q8_SKINNY_MAX_M * d.ldy;
        }
        const q8_status st = f(descs, cnt, Q8_SKINNY_MAX_M);
        if (st != Q8_OK) return st;
    }
    const int32_t rem = M - full * Q8_SKINNY_MAX_M;
    if (rem > 0) {
        descs[0] = d;
        descs[0].x = d.x + static_cast<int64_t>(full) * Q8_SKINNY_MAX_M * d.ldx;
        descs[0].y = d.y + static_cast<int64_t>(full) * Q8_SKINNY_MAX_M * d.ldy;
        return f(descs, 1, rem);
    }
    return Q8_OK;
}

q8_linear_desc w8a8_desc(const int8_t *q, const uint16_t *s, int64_t N, int64_t K, const uint16_t *x, int64_t ldx,
                         float *y, int64_t ldy) {
    q8_linear_desc d;
    d.q = q;
    d.s = s;
    d.x = x;
    d.y = y;
    d.N = N;
    d.K = K;
    d.ldx = ldx;
    d.ldy = ldy;
    return d;
}

}  // namespace
}  // extern "C++"

size_t q8_gemm_w8a8_workspace_size(int64_t N, int64_t K, int32_t M) {
    if (N <= 0 || K <= 0 || K % 32 || M < 1) return 0;
    // placeholder addresses: only the slices' x must differ from one another
    const uintptr_t base = uintptr_t(1) << 40;
    const q8_linear_desc d = w8a8_desc(reinterpret_cast<const int8_t *>(base), reinterpret_cast<const uint16_t *>(base),
                                       N, K, reinterpret_cast<const uint16_t *>(base), K,
                                       reinterpret_cast<float *>(base), N);
    size_t need = 0;
    (void)for_w8a8_launches(d, M, [&](const q8_linear_desc *ds, int cnt, int m) {
        need = std::max(need, w8a8_workspace(ds, cnt, m));
        return Q8_OK;
    });
    return need;
}

q8_status q8_gemm_w8a8(const int8_t *q, const uint16_t *s, int64_t N, int64_t K, const uint16_t *x, int64_t ldx,
                       int32_t M, float *y, int64_t ldy, void *ws, size_t ws_bytes, uint32_t *dev_status,
                       q8_stream_t stream) {
    if (M < 0) return Q8_ERR_SHAPE;
    if (dev_status && !aligned(dev_status, 4)) return Q8_ERR_ALIGN;
    const q8_linear_desc d = w8a8_desc(q, s, N, K, x, ldx, y, ldy);
    q8_status st = check_desc(d, std::min<int32_t>(M, Q8_SKINNY_MAX_M));
    if (st != Q8_OK) return st;
    if (M > 1 && ldy < N) return Q8_ERR_SHAPE;
    if (M == 0 || N == 0) return Q8_OK;
    const size_t need = q8_gemm_w8a8_workspace_size(N, K, M);
    if (need > 0 && (ws == nullptr || ws_bytes < need)) return Q8_ERR_WORKSPACE;
    if (need > 0 && !aligned(ws, 256)) return Q8_ERR_ALIGN;
    const DeviceInfo *di;
    st = check_arch(&di);
    if (st != Q8_OK) return st;
    return for_w8a8_launches(d, M, [&](const q8_linear_desc *ds, int cnt, int m) {
        return launch_skinny(ds, cnt, m, Q8_VARIANT_W8A8, ws, ws_bytes, dev_status,
                             reinterpret_cast<cudaStream_t>(stream), false);
    });
}

q8_status q8_gemv(const int8_t *q, const uint16_t *s, int64_t N, int64_t K, const uint16_t *x, float *y,
                  void *ws, size_t ws_bytes, uint32_t *dev_status, q8_stream_t stream) {
    return q8_gemm_skinny(q, s, N, K, x, K + ((8 - K % 8) % 8), 1, y, N > 0 ? N : 1, ws, ws_bytes,
                          dev_status, stream);
}

q8_status q8_gemm(const int8_t *q, const uint16_t *s, int64_t N, int64_t K, const uint16_t *x, int64_t ldx,
                  int32_t M, uint16_t *y, int64_t ldy, uint32_t *dev_status, q8_stream_t stream) {
    return q8_gemm_ex(q, s, N, K, x, ldx, M, y, ldy, Q8_GEMM_TILE_AUTO, 0, dev_status, stream);
}

q8_status q8_gemm_ex(const int8_t *q, const uint16_t *s, int64_t N, int64_t K, const uint16_t *x, int64_t ldx,
                     int32_t M, uint16_t *y, int64_t ldy, int32_t tile, int32_t splits, uint32_t *dev_status,
                     q8_stream_t stream) {
    if (tile < Q8_GEMM_TILE_AUTO || tile > Q8_GEMM_TILE_64x128) return Q8_ERR_ARG;
    if (splits < 0 || splits > Q8_GEMM_MAX_SPLITS) return Q8_ERR_ARG;
    q8_status st = check_weights(q, s, N, K);
    if (st != Q8_OK) return st;
    if (M < 0) return Q8_ERR_SHAPE;
    if (N == 0 || M == 0) return Q8_OK;
    if (!x || !y) return Q8_ERR_ARG;
    if (ldx < K || ldy < N) return Q8_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(y, 16) || (ldx % 8) || (ldy % 8)) return Q8_ERR_ALIGN;
    if (dev_status && !aligned(dev_status, 4)) return Q8_ERR_ALIGN;
    const DeviceInfo *di;
    st = check_arch(&di);
    if (st != Q8_OK) return st;
    return launch_gemm_tc(q, s, N, K, x, ldx, M, y, ldy, tile, splits, dev_status,
                          reinterpret_cast<cudaStream_t>(stream));
}

q8_status q8_workspace_zero(void *ws, size_t bytes, q8_stream_t stream) {
    if (bytes == 0) return Q8_OK;
    if (!ws) return Q8_ERR_ARG;
    return cudaMemsetAsync(ws, 0, bytes, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? Q8_OK : Q8_ERR_CUDA;
}

// ---- decode step ---------------------------------------------------------------
static q8_status check_cache(const q8_kv_cache *c) {
    if (!c) return Q8_ERR_ARG;
    const int32_t ps = c->page_size;
    if (ps < 16 || ps > 1024 || (ps & (ps - 1)) != 0) return Q8_ERR_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return Q8_ERR_SHAPE;
    if (c->kv_heads < 1 || c->kv_heads > 1024 || c->pages < 1) return Q8_ERR_SHAPE;
    if (!c->kq || !c->ks || !c->vq || !c->vs) return Q8_ERR_ARG;
    if (!aligned(c->kq, 16) || !aligned(c->ks, 16) || !aligned(c->vq, 16) || !aligned(c->vs, 16)) return Q8_ERR_ALIGN;
    return Q8_OK;
}

static q8_status check_kv_rows(const q8_kv_cache *c, const void *k, const void *v, int64_t ldk, int64_t ldv,
                               int32_t dtype, const int64_t *slots, int64_t T, const uint32_t *dev_status) {
    q8_status st = check_cache(c);
    if (st != Q8_OK) return st;
    if (dtype != Q8_DTYPE_F32 && dtype != Q8_DTYPE_BF16) return Q8_ERR_ARG;
    const int64_t row = static_cast<int64_t>(c->kv_heads) * c->head_dim;
    if (T < 0 || T > INT32_MAX || ldk < row || ldv < row || ldk > INT32_MAX || ldv > INT32_MAX) return Q8_ERR_SHAPE;
    if (T == 0) return Q8_OK;
    if (!k || !v || !slots) return Q8_ERR_ARG;
    const int64_t mult = dtype == Q8_DTYPE_F32 ? 4 : 8;
    if (!aligned(k, 16) || !aligned(v, 16) || ldk % mult != 0 || ldv % mult != 0 || !aligned(slots, 8)) return Q8_ERR_ALIGN;
    if (dev_status && !aligned(dev_status, 4)) return Q8_ERR_ALIGN;
    return Q8_OK;
}

q8_status q8_kv_append(const q8_kv_cache *cache, const void *k, const void *v, int64_t ldk, int64_t ldv, int32_t dtype,
                       const int64_t *slots, int64_t T, uint32_t *dev_status, q8_stream_t stream) {
    q8_status st = check_kv_rows(cache, k, v, ldk, ldv, dtype, slots, T, dev_status);
    if (st != Q8_OK || T == 0) return st;
    const DeviceInfo *di;
    st = check_arch(&di);
    if (st != Q8_OK) return st;
    return launch_kv_append(*cache, k, v, ldk, ldv, dtype, slots, T, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

q8_status q8_kv_read(const q8_kv_cache *cache, const int64_t *slots, int64_t T, void *k, void *v, int64_t ldk,
                     int64_t ldv, int32_t dtype, uint32_t *dev_status, q8_stream_t stream) {
    q8_status st = check_kv_rows(cache, k, v, ldk, ldv, dtype, slots, T, dev_status);
    if (st != Q8_OK || T == 0) return st;
    const DeviceInfo *di;
    st = check_arch(&di);
    if (st != Q8_OK) return st;
    return launch_kv_read(*cache, slots, T, k, v, ldk, ldv, dtype, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

static q8_status check_heads(int32_t batch, int32_t q_heads, int32_t kv_heads) {
    if (batch < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || q_heads > 65536) return Q8_ERR_SHAPE;
    return Q8_OK;
}

size_t q8_attn_decode_workspace_size(int32_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    if (check_heads(batch, q_heads, kv_heads) != Q8_OK || batch == 0) return 0;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
    return attn_workspace(q_heads, kv_heads, head_dim);
}

q8_status q8_attn_decode(const q8_kv_cache *cache, const uint16_t *q, int64_t ldq, int32_t q_heads,
                         const int32_t *table, int32_t table_width, const int32_t *lens, int32_t batch, float scale,
                         float softcap, int32_t window, uint16_t *out, float *lse, void *ws, size_t ws_bytes,
                         uint32_t *dev_status, q8_stream_t stream) {
    q8_status st = check_cache(cache);
    if (st != Q8_OK) return st;
    st = check_heads(batch, q_heads, cache->kv_heads);
    if (st != Q8_OK) return st;
    if (table_width < 0 || static_cast<int64_t>(table_width) * cache->page_size > INT32_MAX - 4096) return Q8_ERR_SHAPE;
    if (window < 0 || !(softcap >= 0.0f) || !(scale - scale == 0.0f) || softcap - softcap != 0.0f) return Q8_ERR_ARG;
    if (ldq < static_cast<int64_t>(q_heads) * cache->head_dim) return Q8_ERR_SHAPE;
    if (batch == 0) return Q8_OK;
    if (!q || !lens || !out || (table_width > 0 && !table)) return Q8_ERR_ARG;
    if (!aligned(q, 16) || ldq % 8 != 0 || !aligned(out, 16) || !aligned(lens, 4) || !aligned(table, 4) ||
        !aligned(lse, 4) || !aligned(dev_status, 4))
        return Q8_ERR_ALIGN;
    const size_t need = attn_workspace(q_heads, cache->kv_heads, cache->head_dim);
    if (!ws || ws_bytes < need) return Q8_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return Q8_ERR_ALIGN;
    const DeviceInfo *di;
    st = check_arch(&di);
    if (st != Q8_OK) return st;
    AttnArgs a = {q, table, lens, out, lse, ldq, q_heads, table_width, batch, window, scale, softcap};
    return launch_attn(*cache, a, ws, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

static q8_status check_moe_shape(int32_t T, int32_t E, int64_t H, int64_t F, int32_t top_k) {
    if (T < 0 || T > Q8_SKINNY_MAX_M || E < 1 || E > Q8_MOE_MAX_EXPERTS) return Q8_ERR_SHAPE;
    if (H < 32 || F < 32 || H % 32 != 0 || F % 32 != 0 || H > Q8_MOE_MAX_HIDDEN || F > Q8_MOE_MAX_FFN) return Q8_ERR_SHAPE;
    if (top_k < 1 || top_k > E || top_k > Q8_MOE_MAX_TOP_K) return Q8_ERR_ARG;
    return Q8_OK;
}

size_t q8_moe_workspace_size(int32_t T, int32_t E, int64_t H, int64_t F, int32_t top_k) {
    if (check_moe_shape(T, E, H, F, top_k) != Q8_OK || T == 0) return 0;
    return moe_workspace(T, static_cast<int>(H), static_cast<int>(F), top_k);
}

q8_status q8_moe(const uint16_t *x, int64_t ldx, const float *logits, int64_t ldl, int32_t T, int32_t E, int32_t top_k,
                 int32_t renorm, const int8_t *q13, const uint16_t *s13, const int8_t *q2, const uint16_t *s2, int64_t H,
                 int64_t F, float *y, int64_t ldy, int32_t *ids, float *weights, void *ws, size_t ws_bytes,
                 uint32_t *dev_status, q8_stream_t stream) {
    q8_status st = check_moe_shape(T, E, H, F, top_k);
    if (st != Q8_OK) return st;
    if (ldx < H || ldl < E || ldy < H) return Q8_ERR_SHAPE;
    if (T == 0) return Q8_OK;
    if (!x || !logits || !q13 || !s13 || !q2 || !s2 || !y) return Q8_ERR_ARG;
    if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(q13, 16) || !aligned(s13, 16) || !aligned(q2, 16) || !aligned(s2, 16) ||
        !aligned(logits, 4) || !aligned(y, 4) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(dev_status, 4))
        return Q8_ERR_ALIGN;
    const size_t need = moe_workspace(T, static_cast<int>(H), static_cast<int>(F), top_k);
    if (!ws || ws_bytes < need) return Q8_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return Q8_ERR_ALIGN;
    const DeviceInfo *di;
    st = check_arch(&di);
    if (st != Q8_OK) return st;
    MoeArgs a = {x, logits, q13, q2, s13, s2, y, ids, weights, ldx, ldl, ldy, T, E, static_cast<int32_t>(H),
                 static_cast<int32_t>(F), top_k, renorm};
    return launch_moe(a, ws, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

q8_status q8_sample(const void *logits, int32_t dtype, int64_t ld, int32_t rows, int64_t V, const float *temperature,
                    const int32_t *top_k, const float *top_p, const float *min_p, const float *u, int32_t *token,
                    float *logprob, int32_t *kept, uint32_t *dev_status, q8_stream_t stream) {
    if (dtype != Q8_DTYPE_F32 && dtype != Q8_DTYPE_BF16) return Q8_ERR_ARG;
    if (rows < 0 || rows > (1 << 24) || V < 1 || V > Q8_SAMPLE_MAX_V || ld < V) return Q8_ERR_SHAPE;
    if (rows == 0) return Q8_OK;
    if (!logits || !u || !token) return Q8_ERR_ARG;
    if (!aligned(logits, dtype == Q8_DTYPE_F32 ? 4 : 2) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
        !aligned(min_p, 4) || !aligned(u, 4) || !aligned(token, 4) || !aligned(logprob, 4) || !aligned(kept, 4) ||
        !aligned(dev_status, 4))
        return Q8_ERR_ALIGN;
    const DeviceInfo *di;
    const q8_status st = check_arch(&di);
    if (st != Q8_OK) return st;
    SampleArgs a = {logits, temperature, top_p, min_p, u, top_k, token, kept, logprob, ld, rows, static_cast<int32_t>(V),
                    dtype == Q8_DTYPE_BF16 ? 1 : 0};
    return launch_sample(a, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

// ---- prompt step ---------------------------------------------------------------
static bool dtype_ok(int32_t d) { return d == Q8_DTYPE_F32 || d == Q8_DTYPE_BF16; }
// elements that a row's stride is a multiple of
static int64_t row_step(int32_t d) { return d == Q8_DTYPE_F32 ? 4 : 8; }

q8_status q8_rms_norm(const void *x, int64_t ldx, int32_t x_dtype, const void *residual, int64_t ldr, int32_t residual_dtype,
                      void *residual_out, int64_t ldo, const float *weight, float offset, float eps, int64_t T, int64_t W,
                      uint16_t *y, int64_t ldy, int8_t *q, uint16_t *s, uint32_t *dev_status, q8_stream_t stream) {
    if (!dtype_ok(x_dtype) || !dtype_ok(residual_dtype)) return Q8_ERR_ARG;
    if (T < 0 || T > INT32_MAX || W < 32 || W % 32 != 0 || W > Q8_NORM_MAX_WIDTH) return Q8_ERR_SHAPE;
    if (!(eps >= 0.0f) || eps - eps != 0.0f || offset - offset != 0.0f) return Q8_ERR_ARG;
    if ((q == nullptr) != (s == nullptr) || (residual_out && !residual)) return Q8_ERR_ARG;
    if (ldx < W || (residual && ldr < W) || (residual_out && ldo < W) || (y && ldy < W)) return Q8_ERR_SHAPE;
    if (T == 0) return Q8_OK;
    if (!x || (!y && !q && !residual_out)) return Q8_ERR_ARG;
    const int64_t xs = row_step(x_dtype), rs = row_step(residual_dtype);
    if (!aligned(x, 16) || ldx % xs != 0 || !aligned(residual, 16) || (residual && ldr % rs != 0) || !aligned(residual_out, 16) ||
        (residual_out && ldo % rs != 0) || !aligned(weight, 16) || !aligned(y, 16) || (y && ldy % 8 != 0) || !aligned(q, 16) ||
        !aligned(s, 16) || !aligned(dev_status, 4))
        return Q8_ERR_ALIGN;
    const DeviceInfo *di;
    const q8_status st = check_arch(&di);
    if (st != Q8_OK) return st;
    const NormArgs a = {x, residual, residual_out, weight, y, q, s, ldx, ldr, ldo, ldy, T, static_cast<int32_t>(W), x_dtype,
                        residual_dtype, offset, eps};
    return launch_norm(a, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

q8_status q8_rope_turns(const double *inv_freq, int32_t n, uint64_t *turns) {
    if (n < 0) return Q8_ERR_SHAPE;
    if (n > 0 && (!inv_freq || !turns)) return Q8_ERR_ARG;
    for (int32_t i = 0; i < n; ++i)
        if (!(inv_freq[i] >= -Q8_ROPE_MAX_FREQ && inv_freq[i] <= Q8_ROPE_MAX_FREQ)) return Q8_ERR_ARG;
    rope_turns(inv_freq, n, turns);
    return Q8_OK;
}

static q8_status check_rope(int32_t dtype, int32_t heads, int32_t head_dim, int32_t rot, int32_t layout, float factor,
                            const uint64_t *turns, const int32_t *positions, int64_t T, const uint32_t *dev_status) {
    if (!dtype_ok(dtype) || (layout != Q8_ROPE_HALF && layout != Q8_ROPE_INTERLEAVED) || factor - factor != 0.0f) return Q8_ERR_ARG;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return Q8_ERR_SHAPE;
    if (T < 0 || T > INT32_MAX || heads < 1 || heads > 65536 || rot < 16 || rot % 16 != 0 || rot > head_dim) return Q8_ERR_SHAPE;
    if (T > 0 && (!turns || !positions)) return Q8_ERR_ARG;
    if (!aligned(turns, 8) || !aligned(positions, 4) || !aligned(dev_status, 4)) return Q8_ERR_ALIGN;
    return Q8_OK;
}

q8_status q8_rope(const void *x, int64_t ldx, int32_t dtype, uint16_t *y, int64_t ldy, int32_t heads, int32_t head_dim, int32_t rot,
                  int32_t layout, float factor, const uint64_t *turns, const int32_t *positions, int64_t T, q8_stream_t stream) {
    q8_status st = check_rope(dtype, heads, head_dim, rot, layout, factor, turns, positions, T, nullptr);
    if (st != Q8_OK) return st;
    const int64_t row = static_cast<int64_t>(heads) * head_dim;
    if (ldx < row || ldy < row) return Q8_ERR_SHAPE;
    if (T == 0) return Q8_OK;
    if (!x || !y) return Q8_ERR_ARG;
    if (!aligned(x, 16) || ldx % row_step(dtype) != 0 || !aligned(y, 16) || ldy % 8 != 0) return Q8_ERR_ALIGN;
    const DeviceInfo *di;
    st = check_arch(&di);
    if (st != Q8_OK) return st;
    RopeArgs a = {};
    a.x = x, a.y = y, a.turns = turns, a.positions = positions, a.ldx = ldx, a.ldy = ldy, a.T = T;
    a.heads = heads, a.head_dim = head_dim, a.rot = rot, a.layout = layout, a.dtype = dtype, a.factor = factor;
    return launch_rope(a, nullptr, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

q8_status q8_rope_append(const q8_kv_cache *cache, const void *q, int64_t ldq, int32_t q_heads, const void *k, const void *v,
                         int64_t ldk, int64_t ldv, int32_t dtype, int32_t rot, int32_t layout, float factor, const uint64_t *turns,
                         const int32_t *positions, const int64_t *slots, int64_t T, uint16_t *y, int64_t ldy, uint32_t *dev_status,
                         q8_stream_t stream) {
    q8_status st = check_kv_rows(cache, k, v, ldk, ldv, dtype, slots, T, dev_status);
    if (st != Q8_OK) return st;
    st = check_rope(dtype, q_heads, cache->head_dim, rot, layout, factor, turns, positions, T, dev_status);
    if (st != Q8_OK) return st;
    const int64_t row = static_cast<int64_t>(q_heads) * cache->head_dim;
    if (ldq < row || ldy < row) return Q8_ERR_SHAPE;
    if (T == 0) return Q8_OK;
    if (!q || !y) return Q8_ERR_ARG;
    if (!aligned(q, 16) || ldq % row_step(dtype) != 0 || !aligned(y, 16) || ldy % 8 != 0) return Q8_ERR_ALIGN;
    const DeviceInfo *di;
    st = check_arch(&di);
    if (st != Q8_OK) return st;
    const RopeArgs a = {q, k, v, y, turns, positions, slots, ldq, ldk, ldv, ldy, T, q_heads, cache->head_dim, rot, layout, dtype, factor};
    return launch_rope(a, cache, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

q8_status q8_kv_plan(int32_t *table, int32_t table_width, int32_t pages, int32_t page_size, const int32_t *lens,
                     const int32_t *new_tokens, int32_t batch, const int32_t *free_pages, int32_t free_capacity,
                     const int32_t *free_count, int32_t *free_left, int64_t T, int32_t *starts, int64_t *slots, int32_t *positions,
                     int32_t *lens_out, uint32_t *dev_status, q8_stream_t stream) {
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0 || pages < 1) return Q8_ERR_SHAPE;
    if (table_width < 0 || static_cast<int64_t>(table_width) * page_size > INT32_MAX - 4096) return Q8_ERR_SHAPE;
    if (batch < 0 || batch > Q8_PLAN_MAX_BATCH || T < 0 || T > INT32_MAX || free_capacity < 0) return Q8_ERR_SHAPE;
    if (!starts || (batch > 0 && (!lens || !new_tokens || !lens_out || (table_width > 0 && !table)))) return Q8_ERR_ARG;
    if ((T > 0 && (!slots || !positions)) || (free_pages && (!free_count || !free_left))) return Q8_ERR_ARG;
    if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(new_tokens, 4) || !aligned(free_pages, 4) || !aligned(free_count, 4) ||
        !aligned(free_left, 4) || !aligned(starts, 4) || !aligned(slots, 8) || !aligned(positions, 4) || !aligned(lens_out, 4) ||
        !aligned(dev_status, 4))
        return Q8_ERR_ALIGN;
    const DeviceInfo *di;
    const q8_status st = check_arch(&di);
    if (st != Q8_OK) return st;
    const PlanArgs a = {table, lens, new_tokens, free_pages, free_count, starts, positions, lens_out, free_left, slots, T, batch,
                        table_width, page_size, pages, free_capacity};
    return launch_plan(a, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

size_t q8_attn_chunk_workspace_size(int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    if (check_heads(1, q_heads, kv_heads) != Q8_OK) return 0;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
    return chunk_workspace(q_heads, kv_heads, head_dim);
}

q8_status q8_attn_chunk(const q8_kv_cache *cache, const uint16_t *q, int64_t ldq, int32_t q_heads, int64_t T, const int32_t *table,
                        int32_t table_width, const int32_t *lens, const int32_t *starts, int32_t batch, float scale, float softcap,
                        int32_t window, uint16_t *out, float *lse, void *ws, size_t ws_bytes, uint32_t *dev_status,
                        q8_stream_t stream) {
    q8_status st = check_cache(cache);
    if (st != Q8_OK) return st;
    st = check_heads(batch, q_heads, cache->kv_heads);
    if (st != Q8_OK) return st;
    if (table_width < 0 || static_cast<int64_t>(table_width) * cache->page_size > INT32_MAX - 4096) return Q8_ERR_SHAPE;
    if (T < 0 || T * (q_heads / cache->kv_heads) > INT32_MAX - 4096 || T > INT32_MAX) return Q8_ERR_SHAPE;
    if (window < 0 || !(softcap >= 0.0f) || !(scale - scale == 0.0f) || softcap - softcap != 0.0f) return Q8_ERR_ARG;
    if (ldq < static_cast<int64_t>(q_heads) * cache->head_dim) return Q8_ERR_SHAPE;
    if (batch == 0 || T == 0) return Q8_OK;
    if (!q || !lens || !starts || !out || (table_width > 0 && !table)) return Q8_ERR_ARG;
    if (!aligned(q, 16) || ldq % 8 != 0 || !aligned(out, 16) || !aligned(lens, 4) || !aligned(starts, 4) || !aligned(table, 4) ||
        !aligned(lse, 4) || !aligned(dev_status, 4))
        return Q8_ERR_ALIGN;
    const size_t need = chunk_workspace(q_heads, cache->kv_heads, cache->head_dim);
    if (need > 0 && (!ws || ws_bytes < need)) return Q8_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return Q8_ERR_ALIGN;
    const DeviceInfo *di;
    st = check_arch(&di);
    if (st != Q8_OK) return st;
    const ChunkArgs a = {q, table, lens, starts, out, lse, ldq, T, q_heads, table_width, batch, window, scale, softcap};
    return launch_chunk(*cache, a, ws, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
