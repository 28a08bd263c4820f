// C ABI entry points: argument validation, workspace sizing, launch sequencing.
#include <atomic>
#include <mutex>
#include <vector>

#include "common.cuh"
#include "fp8.cuh"

namespace gptq {

static std::atomic<unsigned long long> g_launches{0};
void count_launch(unsigned n) { g_launches.fetch_add(n, std::memory_order_relaxed); }
unsigned long long launches_so_far() { return g_launches.load(); }

namespace {
struct AttrEntry {
  const void *func;
  int dev;
  int bytes;
};
std::mutex g_attr_mu;
std::vector<AttrEntry> g_attrs;            // (kernel, device) pairs already set
constexpr int kMaxSmDevices = 128;
std::atomic<int> g_sm_count[kMaxSmDevices];  // 0 = not yet queried
}  // namespace

gptq_status ensure_smem_attr(const void *func, int bytes) {
  int dev = -1;
  GPTQ_CUDA_CHECK(cudaGetDevice(&dev));
  std::lock_guard<std::mutex> lock(g_attr_mu);
  for (const AttrEntry &e : g_attrs)
    if (e.func == func && e.dev == dev && e.bytes >= bytes) return GPTQ_OK;
  GPTQ_CUDA_CHECK(cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  g_attrs.push_back(AttrEntry{func, dev, bytes});
  return GPTQ_OK;
}

gptq_status device_sm_count(int *out) {
  int dev = -1;
  GPTQ_CUDA_CHECK(cudaGetDevice(&dev));
  if (dev < 0 || dev >= kMaxSmDevices) return GPTQ_ERR_UNSUPPORTED;
  int n = g_sm_count[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    GPTQ_CUDA_CHECK(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev));
    g_sm_count[dev].store(n, std::memory_order_relaxed);
  }
  *out = n;
  return GPTQ_OK;
}

static bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

static size_t elem_size(int dt) {
  switch (dt) {
    case GPTQ_F16:
    case GPTQ_BF16: return 2;
    case GPTQ_F32: return 4;
    default: return 0;
  }
}


gptq_status quantize_layer_checked(const void *W, int wdtype, int64_t d_out,
                                         int64_t d_in, int64_t ldw, const float *U,
                                         const uint8_t *dead_mask, int bits, int block,
                                         uint32_t *qpacked, float *scale, int32_t *zero,
                                         float *W_hat, void *ws, size_t ws_bytes,
                                         gptq_stream_t stream, bool allow_overlap) {
  const size_t es = elem_size(wdtype);
  if (es == 0 || !W || !U || !qpacked || !scale || !zero) return GPTQ_ERR_INVALID_ARG;
  if (d_out < 1 || d_in < 1 || ldw < d_in) return GPTQ_ERR_INVALID_ARG;
  if (!(bits == 2 || bits == 3 || bits == 4 || bits == 8)) return GPTQ_ERR_INVALID_ARG;
  if (block < 1 || block > 128) return GPTQ_ERR_INVALID_ARG;
  if (!aligned(W, es) || !aligned(U, 16) || !aligned(qpacked, 4) || !aligned(scale, 4) ||
      !aligned(zero, 4) || (W_hat && !aligned(W_hat, 4)))
    return GPTQ_ERR_INVALID_ARG;
  if (d_in > (int64_t)1 << 17 || d_out > (int64_t)1 << 24) return GPTQ_ERR_UNSUPPORTED;
  if (!ws || !aligned(ws, 256) || ws_bytes < quantize_ws_bytes(d_out, d_in, bits, block))
    return GPTQ_ERR_WORKSPACE;
  return launch_quantize(W, wdtype, d_out, d_in, ldw, U, dead_mask, bits, block, qpacked,
                         scale, zero, W_hat, ws, (cudaStream_t)stream, allow_overlap);
}

}  // namespace gptq

using namespace gptq;

extern "C" {

const char *gptq_status_str(int status) {
  switch (status) {
    case GPTQ_OK: return "GPTQ_OK";
    case GPTQ_ERR_INVALID_ARG: return "GPTQ_ERR_INVALID_ARG";
    case GPTQ_ERR_NOT_PD: return "GPTQ_ERR_NOT_PD";
    case GPTQ_ERR_NONFINITE: return "GPTQ_ERR_NONFINITE";
    case GPTQ_ERR_TIMEOUT: return "GPTQ_ERR_TIMEOUT";
    case GPTQ_ERR_CUDA: return "GPTQ_ERR_CUDA";
    case GPTQ_ERR_UNSUPPORTED: return "GPTQ_ERR_UNSUPPORTED";
    case GPTQ_ERR_WORKSPACE: return "GPTQ_ERR_WORKSPACE";
    default: return "GPTQ_ERR_UNKNOWN";
  }
}

int gptq_abi_version(void) { return GPTQ_ABI_VERSION; }

unsigned long long gptq_kernel_launches(void) { return g_launches.load(); }

gptq_status gptq_hessian_accumulate(const void *X, int xdtype, int64_t n_tok, int64_t d_in,
                                    int64_t ldx, float *H, int accumulate,
                                    gptq_stream_t stream) {
  const size_t es = elem_size(xdtype);
  if (es == 0 || n_tok < 0 || d_in < 1 || ldx < d_in || !H) return GPTQ_ERR_INVALID_ARG;
  if (n_tok > 0 && (!X || !aligned(X, 16) || (ldx * (int64_t)es) % 16 != 0))
    return GPTQ_ERR_INVALID_ARG;
  if (!aligned(H, 16)) return GPTQ_ERR_INVALID_ARG;
  if (d_in > (int64_t)1 << 20) return GPTQ_ERR_UNSUPPORTED;
  return launch_hessian(X, xdtype, n_tok, d_in, ldx, H, accumulate ? 1 : 0, nullptr,
                        (cudaStream_t)stream);
}

size_t gptq_hessian_host_workspace_bytes(int xdtype, int64_t d_in, int64_t chunk_tok) {
  const size_t es = elem_size(xdtype);
  if (es == 0 || d_in < 1 || chunk_tok < 0) return 0;
  return hessian_host_ws_bytes(d_in, es, chunk_tok);
}

gptq_status gptq_hessian_accumulate_host(const void *X_host, int xdtype, int64_t n_tok,
                                         int64_t d_in, int64_t ldx, float *H, int accumulate,
                                         int64_t chunk_tok, void *ws, size_t ws_bytes,
                                         gptq_stream_t stream) {
  const size_t es = elem_size(xdtype);
  if (es == 0 || n_tok < 0 || d_in < 1 || ldx < d_in || chunk_tok < 0 || !H)
    return GPTQ_ERR_INVALID_ARG;
  if (n_tok > 0 && !X_host) return GPTQ_ERR_INVALID_ARG;
  if (!aligned(H, 16) || (d_in * (int64_t)es) % 16 != 0) return GPTQ_ERR_INVALID_ARG;
  if (d_in > (int64_t)1 << 20) return GPTQ_ERR_UNSUPPORTED;
  if (!ws || !aligned(ws, 256) || ws_bytes < hessian_host_ws_bytes(d_in, es, chunk_tok))
    return GPTQ_ERR_WORKSPACE;
  return launch_hessian_host(X_host, xdtype, es, n_tok, d_in, ldx, H, accumulate ? 1 : 0,
                             chunk_tok, ws, (cudaStream_t)stream);
}

size_t gptq_prepare_workspace_bytes(int64_t d_in) {
  if (d_in < 1) return 0;
  return prepare_ws_bytes(d_in);
}

gptq_status gptq_prepare(float *H, int64_t d_in, float damp, float *U, uint8_t *dead_mask,
                         int32_t *n_dead, void *ws, size_t ws_bytes, gptq_stream_t stream) {
  if (!H || !U || d_in < 1 || !(damp >= 0.0f) || !aligned(H, 16) || !aligned(U, 16))
    return GPTQ_ERR_INVALID_ARG;
  if (d_in > (int64_t)1 << 17) return GPTQ_ERR_UNSUPPORTED;
  if (!ws || !aligned(ws, 256) || ws_bytes < prepare_ws_bytes(d_in)) return GPTQ_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  GPTQ_TRY(launch_prepare(H, d_in, damp, U, dead_mask, ws, s));
  DevStatus st;
  GPTQ_CUDA_CHECK(cudaMemcpyAsync(&st, ws, sizeof(DevStatus), cudaMemcpyDeviceToHost, s));
  GPTQ_CUDA_CHECK(cudaStreamSynchronize(s));
  if (n_dead) *n_dead = st.n_dead;
  return (gptq_status)st.status;
}

size_t gptq_quantize_workspace_bytes(int64_t d_out, int64_t d_in, int bits, int block) {
  if (d_out < 1 || d_in < 1) return 0;
  return quantize_ws_bytes(d_out, d_in, bits, block);
}


size_t gptq_quantize_shared_workspace_bytes(int n_layers, const int64_t *d_out, int64_t d_in,
                                            int bits, int block) {
  if (n_layers < 1 || n_layers > GPTQ_MAX_SHARED_LAYERS || !d_out || d_in < 1) return 0;
  for (int i = 0; i < n_layers; ++i)
    if (d_out[i] < 1) return 0;
  return quantize_layers_ws_bytes(d_out, n_layers, d_in, bits, block);
}

gptq_status gptq_quantize_layers_shared(int n_layers, const void *const *W, const int *wdtype,
                                        const int64_t *d_out, const int64_t *ldw, int64_t d_in,
                                        const float *U, const uint8_t *dead_mask, int bits,
                                        int block, uint32_t *const *qpacked,
                                        float *const *scale, int32_t *const *zero,
                                        float *const *W_hat, void *ws, size_t ws_bytes,
                                        gptq_stream_t stream) {
  if (n_layers < 1 || n_layers > GPTQ_MAX_SHARED_LAYERS) return GPTQ_ERR_INVALID_ARG;
  if (!W || !wdtype || !d_out || !ldw || !qpacked || !scale || !zero || !U || d_in < 1)
    return GPTQ_ERR_INVALID_ARG;
  if (!(bits == 2 || bits == 3 || bits == 4 || bits == 8)) return GPTQ_ERR_INVALID_ARG;
  if (block < 1 || block > 128 || !aligned(U, 16)) return GPTQ_ERR_INVALID_ARG;
  QLayer L[GPTQ_MAX_SHARED_LAYERS];
  int64_t rows = 0;
  for (int i = 0; i < n_layers; ++i) {
    const size_t es = elem_size(wdtype[i]);
    float *wh = W_hat ? W_hat[i] : nullptr;
    if (es == 0 || !W[i] || !qpacked[i] || !scale[i] || !zero[i]) return GPTQ_ERR_INVALID_ARG;
    if (d_out[i] < 1 || ldw[i] < d_in) return GPTQ_ERR_INVALID_ARG;
    if (!aligned(W[i], es) || !aligned(qpacked[i], 4) || !aligned(scale[i], 4) ||
        !aligned(zero[i], 4) || (wh && !aligned(wh, 4)))
      return GPTQ_ERR_INVALID_ARG;
    rows += d_out[i];
    L[i] = QLayer{W[i], wdtype[i], d_out[i], ldw[i], qpacked[i], scale[i], zero[i], wh};
  }
  if (d_in > (int64_t)1 << 17 || rows > (int64_t)1 << 24) return GPTQ_ERR_UNSUPPORTED;
  if (!ws || !aligned(ws, 256) ||
      ws_bytes < quantize_layers_ws_bytes(d_out, n_layers, d_in, bits, block))
    return GPTQ_ERR_WORKSPACE;
  return launch_quantize_layers(L, n_layers, d_in, U, dead_mask, bits, block, ws,
                                (cudaStream_t)stream, true);
}

size_t gptq_recon_error_workspace_bytes(int xdtype, int64_t d_out, int64_t d_in,
                                        int64_t n_tok) {
  if (elem_size(xdtype) == 0 || d_out < 1 || d_in < 1 || n_tok < 0) return 0;
  return recon_ws_bytes(xdtype, d_out, d_in, n_tok);
}

gptq_status gptq_recon_error(const void *X, int xdtype, int64_t n_tok, int64_t d_in,
                             int64_t ldx, const void *W, int wdtype, int64_t d_out, int64_t ldw,
                             const uint32_t *qpacked, int bits, const float *scale,
                             const int32_t *zero, float *err, void *ws, size_t ws_bytes,
                             gptq_stream_t stream) {
  const size_t xes = elem_size(xdtype), wes = elem_size(wdtype);
  if (xes == 0 || wes == 0 || n_tok < 0 || d_in < 1 || d_out < 1 || ldx < d_in ||
      ldw < d_in || !W || !qpacked || !scale || !zero || !err)
    return GPTQ_ERR_INVALID_ARG;
  if (!(bits == 2 || bits == 3 || bits == 4 || bits == 8)) return GPTQ_ERR_INVALID_ARG;
  if (n_tok > 0 && (!X || !aligned(X, 16) || (ldx * (int64_t)xes) % 16 != 0))
    return GPTQ_ERR_INVALID_ARG;
  if (!aligned(W, wes) || !aligned(qpacked, 4) || !aligned(scale, 4) || !aligned(zero, 4) ||
      !aligned(err, 4))
    return GPTQ_ERR_INVALID_ARG;
  if (d_in > (int64_t)1 << 20 || d_out > (int64_t)1 << 24 || n_tok > (int64_t)1 << 31)
    return GPTQ_ERR_UNSUPPORTED;
  if (!ws || !aligned(ws, 256) || ws_bytes < recon_ws_bytes(xdtype, d_out, d_in, n_tok))
    return GPTQ_ERR_WORKSPACE;
  return launch_recon(X, xdtype, n_tok, d_in, ldx, W, wdtype, d_out, ldw, qpacked, bits, scale,
                      zero, err, ws, (cudaStream_t)stream);
}

size_t gptq_quantize_obq_workspace_bytes(int64_t d_out, int64_t d_in) {
  if (d_out < 1 || d_in < 1) return 0;
  return quantize_obq_ws_bytes(d_out, d_in);
}

gptq_status gptq_quantize_obq(const void *W, int wdtype, int64_t d_out, int64_t d_in,
                              int64_t ldw, const float *U, const uint8_t *dead_mask, int bits,
                              uint32_t *qpacked, float *scale, int32_t *zero, float *W_hat,
                              int32_t *order, void *ws, size_t ws_bytes, gptq_stream_t stream) {
  const size_t es = elem_size(wdtype);
  if (es == 0 || !W || !U || !qpacked || !scale || !zero) return GPTQ_ERR_INVALID_ARG;
  if (d_out < 1 || d_in < 1 || ldw < d_in) return GPTQ_ERR_INVALID_ARG;
  if (!(bits == 2 || bits == 3 || bits == 4 || bits == 8)) return GPTQ_ERR_INVALID_ARG;
  if (!aligned(W, es) || !aligned(U, 4) || !aligned(qpacked, 4) || !aligned(scale, 4) ||
      !aligned(zero, 4) || (W_hat && !aligned(W_hat, 4)) || (order && !aligned(order, 4)))
    return GPTQ_ERR_INVALID_ARG;
  if (d_in > GPTQ_OBQ_MAX_D_IN || d_out > (int64_t)1 << 24) return GPTQ_ERR_UNSUPPORTED;
  if (!ws || !aligned(ws, 256) || ws_bytes < quantize_obq_ws_bytes(d_out, d_in))
    return GPTQ_ERR_WORKSPACE;
  return launch_quantize_obq(W, wdtype, d_out, d_in, ldw, U, dead_mask, bits, qpacked, scale,
                             zero, W_hat, order, ws, (cudaStream_t)stream);
}

gptq_status gptq_quantize_layer(const void *W, int wdtype, int64_t d_out, int64_t d_in,
                                int64_t ldw, const float *U, const uint8_t *dead_mask,
                                int bits, int block, uint32_t *qpacked, float *scale,
                                int32_t *zero, float *W_hat, void *ws, size_t ws_bytes,
                                gptq_stream_t stream) {
  return gptq::quantize_layer_checked(W, wdtype, d_out, d_in, ldw, U, dead_mask, bits, block,
                                      qpacked, scale, zero, W_hat, ws, ws_bytes, stream, true);
}

gptq_status gptq_debug_hessian_lost_stage(const void *X, int xdtype, int64_t n_tok,
                                          int64_t d_in, int64_t ldx, float *H,
                                          int64_t lost_stage, uint64_t wait_ns, void *status_ws,
                                          gptq_stream_t stream) {
  const size_t es = elem_size(xdtype);
  if (es == 0 || n_tok < 1 || d_in < 1 || ldx < d_in || !X || !H || !status_ws)
    return GPTQ_ERR_INVALID_ARG;
  if (!aligned(X, 16) || (ldx * (int64_t)es) % 16 != 0 || !aligned(H, 16))
    return GPTQ_ERR_INVALID_ARG;
  if (!aligned(status_ws, 256)) return GPTQ_ERR_WORKSPACE;
  if (wait_ns < 1000 || wait_ns > 10000000000ull) return GPTQ_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  GPTQ_CUDA_CHECK(cudaMemsetAsync(status_ws, 0, sizeof(DevStatus), s));
  GPTQ_TRY(launch_hessian_lost_stage(X, xdtype, n_tok, d_in, ldx, H, lost_stage, wait_ns,
                                     (DevStatus *)status_ws, s));
  DevStatus st;
  GPTQ_CUDA_CHECK(cudaMemcpyAsync(&st, status_ws, sizeof(DevStatus), cudaMemcpyDeviceToHost, s));
  GPTQ_CUDA_CHECK(cudaStreamSynchronize(s));
  return (gptq_status)st.status;
}

gptq_status gptq_workspace_status(const void *ws, gptq_stream_t stream) {
  if (!ws || !aligned(ws, 256)) return GPTQ_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  DevStatus st;
  GPTQ_CUDA_CHECK(cudaMemcpyAsync(&st, ws, sizeof(DevStatus), cudaMemcpyDeviceToHost, s));
  GPTQ_CUDA_CHECK(cudaStreamSynchronize(s));
  return (gptq_status)st.status;
}

// A matrix of codes: base and pitch alignment, pitch >= d.
static bool fp8_codes_ok(const uint8_t *codes, int64_t ldc, int64_t d) {
  return codes && aligned(codes, 16) && ldc >= d && ldc % 16 == 0;
}
static bool fp8_exps_ok(const uint8_t *exps, int64_t lde, int64_t d) {
  return exps && aligned(exps, 4) && lde >= ceil_div(d, 128) && lde % 4 == 0;
}
constexpr int64_t kFp8MaxWidth = (int64_t)1 << 20, kFp8MaxRows = (int64_t)1 << 22;

gptq_status gptq_rmsnorm_fp8(const void *X, int xdtype, int64_t rows, int64_t d, int64_t ldx,
                             const void *R, int64_t ldr, const void *weight, int wdtype,
                             float eps, void *H, int64_t ldh, uint8_t *codes, int64_t ldc,
                             uint8_t *exps, int64_t lde, float *rstd, gptq_stream_t stream) {
  const size_t es = elem_size(xdtype);
  if (es == 0 || (wdtype != xdtype && wdtype != GPTQ_F32)) return GPTQ_ERR_INVALID_ARG;
  if (rows < 0 || d < 1 || ldx < d || (R && ldr < d) || (H && ldh < d) || !(eps >= 0.0f))
    return GPTQ_ERR_INVALID_ARG;
  if (!weight || !aligned(weight, elem_size(wdtype))) return GPTQ_ERR_INVALID_ARG;
  if (rows > 0 && (!X || !rstd || !fp8_codes_ok(codes, ldc, d) || !fp8_exps_ok(exps, lde, d)))
    return GPTQ_ERR_INVALID_ARG;
  if (!aligned(X, es) || (R && !aligned(R, es)) || (H && !aligned(H, es)) || !aligned(rstd, 4))
    return GPTQ_ERR_INVALID_ARG;
  if (d > kFp8MaxWidth || rows > kFp8MaxRows) return GPTQ_ERR_UNSUPPORTED;
  return launch_rmsnorm_fp8(X, xdtype, rows, d, ldx, R, ldr, weight, wdtype, eps, H, ldh, codes,
                            ldc, exps, lde, rstd, (cudaStream_t)stream);
}

gptq_status gptq_fp8_quantize(const void *X, int xdtype, int64_t rows, int64_t d, int64_t ldx,
                              int row_block, uint8_t *codes, int64_t ldc, uint8_t *exps,
                              int64_t lde, gptq_stream_t stream) {
  const size_t es = elem_size(xdtype);
  if (es == 0 || rows < 0 || d < 1 || ldx < d || (row_block != 1 && row_block != fp8::kBlock))
    return GPTQ_ERR_INVALID_ARG;
  if (rows > 0 && (!X || !aligned(X, es) || !fp8_codes_ok(codes, ldc, d) ||
                   !fp8_exps_ok(exps, lde, d)))
    return GPTQ_ERR_INVALID_ARG;
  if (d > kFp8MaxWidth || rows > kFp8MaxRows) return GPTQ_ERR_UNSUPPORTED;
  return launch_fp8_quantize(X, xdtype, rows, d, ldx, row_block, codes, ldc, exps, lde,
                             (cudaStream_t)stream);
}

gptq_status gptq_fp8_from_codes(const uint32_t *qpacked, int bits, const int32_t *zero,
                                int64_t d_out, int64_t d_in, uint8_t *codes, int64_t ldc,
                                uint8_t *exps, int64_t lde, gptq_stream_t stream) {
  if (!(bits == 2 || bits == 3 || bits == 4 || bits == 8)) return GPTQ_ERR_INVALID_ARG;
  if (d_out < 1 || d_in < 1 || !qpacked || !aligned(qpacked, 4) || !zero || !aligned(zero, 4))
    return GPTQ_ERR_INVALID_ARG;
  if (!fp8_codes_ok(codes, ldc, d_in) || !fp8_exps_ok(exps, lde, d_in))
    return GPTQ_ERR_INVALID_ARG;
  if (bits == 8 || d_in > kFp8MaxWidth || d_out > kFp8MaxRows) return GPTQ_ERR_UNSUPPORTED;
  return launch_fp8_from_codes(qpacked, bits, zero, d_out, d_in, codes, ldc, exps, lde,
                               (cudaStream_t)stream);
}

size_t gptq_fp8_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n < 1 || k < 1) return 0;
  return fp8_matmul_ws_bytes(m, n, k);
}

static gptq_status fp8_matmul_checked(const Fp8MatmulArgs &g, void *ws, size_t ws_bytes,
                                      gptq_stream_t stream) {
  if (g.M < 0 || g.N < 1 || g.K < 1 || (g.odtype != GPTQ_F16 && g.odtype != GPTQ_BF16) || g.ldo < g.N)
    return GPTQ_ERR_INVALID_ARG;
  if (!fp8_codes_ok(g.w, g.ldw, g.K) || !fp8_exps_ok(g.we, g.ldwe, g.K) || !aligned(g.rw, 4))
    return GPTQ_ERR_INVALID_ARG;
  if (g.M > 0 && (!fp8_codes_ok(g.a, g.lda, g.K) || !fp8_exps_ok(g.ae, g.ldae, g.K) ||
                  !aligned(g.ra, 4) || !g.out || !aligned(g.out, 2)))
    return GPTQ_ERR_INVALID_ARG;
  if (g.K > kFp8MaxWidth || g.M > kFp8MaxRows || g.N > kFp8MaxRows) return GPTQ_ERR_UNSUPPORTED;
  if (!ws || !aligned(ws, 256) || ws_bytes < fp8_matmul_ws_bytes(g.M, g.N, g.K))
    return GPTQ_ERR_WORKSPACE;
  return launch_fp8_matmul(g, ws, (cudaStream_t)stream);
}

gptq_status gptq_fp8_matmul(const uint8_t *a, int64_t lda, const uint8_t *a_exps, int64_t ldae,
                            const float *a_scale, const uint8_t *w, int64_t ldw,
                            const uint8_t *w_exps, int64_t ldwe, const float *w_scale, int64_t m,
                            int64_t n, int64_t k, void *out, int odtype, int64_t ldo, void *ws,
                            size_t ws_bytes, gptq_stream_t stream) {
  return fp8_matmul_checked({a, lda, a_exps, ldae, a_scale, w, ldw, w_exps, ldwe, w_scale, m, n, k,
                             out, odtype, ldo}, ws, ws_bytes, stream);
}

// A test hook's copy that is left out, and budget of the waits.
static bool lost_ok(int64_t lost, uint64_t wait_ns) {
  return lost >= 0 && lost <= INT32_MAX && wait_ns >= 1000 && wait_ns <= 10000000000ull;
}

gptq_status gptq_debug_fp8_matmul_lost_copy(const uint8_t *a, int64_t lda, const uint8_t *a_exps,
                                            int64_t ldae, const uint8_t *w, int64_t ldw,
                                            const uint8_t *w_exps, int64_t ldwe, int64_t m,
                                            int64_t n, int64_t k, void *out, int odtype,
                                            int64_t ldo, int64_t lost_copy, uint64_t wait_ns,
                                            void *ws, size_t ws_bytes, gptq_stream_t stream) {
  if (!lost_ok(lost_copy, wait_ns) || m < 1) return GPTQ_ERR_INVALID_ARG;
  Fp8MatmulArgs g{a, lda, a_exps, ldae, nullptr, w, ldw, w_exps, ldwe, nullptr, m, n, k,
                  out, odtype, ldo};
  g.wait_ns = wait_ns;
  g.lost = lost_copy;
  GPTQ_TRY(fp8_matmul_checked(g, ws, ws_bytes, stream));
  return gptq_workspace_status(ws, stream);
}

gptq_status gptq_serving_status(gptq_stream_t stream) {
  int product = 0, attention = 0;
  GPTQ_TRY(fp8_matmul_take_timeout(&product, (cudaStream_t)stream));
  GPTQ_TRY(kv8_attention_take_timeout(&attention, (cudaStream_t)stream));
  return (gptq_status)(product != 0 ? product : attention);
}

// What the two cache calls share; `ok` = valid, UNSUPPORTED for sizes outside the limits.
static gptq_status kv8_cache_check(int64_t n_seq, int64_t n_new, int n_kv, int dim,
                                   const uint8_t *k, const uint8_t *v, const uint8_t *k_exps,
                                   const uint8_t *v_exps, int64_t n_blocks, const int32_t *table,
                                   int64_t ld_table, int64_t max_blocks) {
  if (n_seq < 0 || n_new < 0 || n_kv < 1 || dim < 1 || n_blocks < 0 || max_blocks < 0 ||
      ld_table < max_blocks)
    return GPTQ_ERR_INVALID_ARG;
  if (n_blocks > 0 && (!k || !v || !k_exps || !v_exps || !aligned(k, 16) || !aligned(v, 16)))
    return GPTQ_ERR_INVALID_ARG;
  if (max_blocks > 0 && n_seq > 0 && (!table || !aligned(table, 4))) return GPTQ_ERR_INVALID_ARG;
  if ((dim != 64 && dim != 128) || n_kv > 4096 || n_seq > 65535 || n_new > (1 << 20) ||
      max_blocks > (1 << 20) || n_blocks > INT32_MAX / n_kv)
    return GPTQ_ERR_UNSUPPORTED;
  return GPTQ_OK;
}
static bool strides_ok(const int64_t *st) {
  return st && st[0] >= 0 && st[1] >= 0 && st[2] >= 0;
}
static int strided_alignment(const void *p, const int64_t *st, size_t es) {
  return fp8::alignment(p, st[0] * (int64_t)es, st[1] * (int64_t)es, st[2] * (int64_t)es);
}

gptq_status gptq_kv8_append(const void *new_k, const int64_t *k_strides, const void *new_v,
                            const int64_t *v_strides, int dtype, int64_t n_seq, int64_t n_new,
                            int n_kv, int dim, uint8_t *k, uint8_t *v, uint8_t *k_exps,
                            uint8_t *v_exps, int64_t n_blocks, const int32_t *table,
                            int64_t ld_table, int64_t max_blocks, const int32_t *start,
                            gptq_stream_t stream) {
  const size_t es = elem_size(dtype);
  if (es == 0 || !strides_ok(k_strides) || !strides_ok(v_strides)) return GPTQ_ERR_INVALID_ARG;
  GPTQ_TRY(kv8_cache_check(n_seq, n_new, n_kv, dim, k, v, k_exps, v_exps, n_blocks, table,
                           ld_table, max_blocks));
  if (n_seq == 0 || n_new == 0 || n_blocks == 0 || max_blocks == 0) return GPTQ_OK;
  if (!new_k || !new_v || !aligned(new_k, es) || !aligned(new_v, es) || !start ||
      !aligned(start, 4))
    return GPTQ_ERR_INVALID_ARG;
  Kv8AppendArgs g{};
  g.new_k = new_k; g.new_v = new_v; g.dtype = dtype;
  for (int i = 0; i < 3; ++i) {
    g.k_stride[i] = k_strides[i];
    g.v_stride[i] = v_strides[i];
  }
  g.align_k = strided_alignment(new_k, k_strides, es);
  g.align_v = strided_alignment(new_v, v_strides, es);
  g.n_seq = (int)n_seq; g.n_new = n_new; g.n_kv = n_kv; g.dim = dim;
  g.k = k; g.v = v; g.k_exps = k_exps; g.v_exps = v_exps; g.n_blocks = n_blocks;
  g.table = table; g.ld_table = ld_table; g.max_blocks = (int)max_blocks;
  g.start = start;
  return launch_kv8_append(g, (cudaStream_t)stream);
}

size_t gptq_kv8_attention_workspace_bytes(int64_t n_seq, int64_t n_new, int n_heads, int n_kv,
                                          int dim, int64_t max_blocks) {
  if (n_seq < 0 || n_seq > 65535 || n_new < 0 || n_new > (1 << 20) || n_kv < 1 || n_kv > 4096 ||
      n_heads < 1 || n_heads % n_kv != 0 || (dim != 64 && dim != 128) || max_blocks < 0 ||
      max_blocks > (1 << 20))
    return 0;
  return kv8_attention_ws_bytes((int)n_seq, n_new, n_heads, n_kv, dim, (int)max_blocks);
}

static gptq_status kv8_attention_checked(
    const void *q, const int64_t *q_strides, int dtype, int64_t n_seq, int64_t n_new, int n_heads,
    int n_kv, int dim, const uint8_t *k, const uint8_t *v, const uint8_t *k_exps,
    const uint8_t *v_exps, int64_t n_blocks, const int32_t *table, int64_t ld_table,
    int64_t max_blocks, const int32_t *lengths, int causal, float scale, void *out,
    const int64_t *o_strides, int64_t lost, uint64_t wait_ns, void *ws, size_t ws_bytes,
    gptq_stream_t stream) {
  if ((dtype != GPTQ_F16 && dtype != GPTQ_BF16) || !strides_ok(q_strides) || !strides_ok(o_strides))
    return GPTQ_ERR_INVALID_ARG;
  if (n_heads < 1 || n_kv < 1 || n_heads % n_kv != 0 || !(scale - scale == 0.0f))
    return GPTQ_ERR_INVALID_ARG;
  GPTQ_TRY(kv8_cache_check(n_seq, n_new, n_kv, dim, k, v, k_exps, v_exps, n_blocks, table,
                           ld_table, max_blocks));
  if (n_heads > 65535) return GPTQ_ERR_UNSUPPORTED;
  if (n_seq > 0 && n_new > 0 && (!q || !out || !aligned(q, 2) || !aligned(out, 2) || !lengths ||
                                 !aligned(lengths, 4)))
    return GPTQ_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256) ||
      ws_bytes < kv8_attention_ws_bytes((int)n_seq, n_new, n_heads, n_kv, dim, (int)max_blocks))
    return GPTQ_ERR_WORKSPACE;
  Kv8AttentionArgs g{};
  g.q = q; g.out = out; g.dtype = dtype;
  for (int i = 0; i < 3; ++i) {
    g.q_stride[i] = q_strides[i];
    g.o_stride[i] = o_strides[i];
  }
  g.n_seq = (int)n_seq; g.n_new = n_new; g.n_heads = n_heads; g.n_kv = n_kv; g.dim = dim;
  g.k = k; g.v = v; g.k_exps = k_exps; g.v_exps = v_exps; g.n_blocks = n_blocks;
  g.table = table; g.ld_table = ld_table; g.max_blocks = (int)max_blocks;
  g.lengths = lengths; g.causal = causal ? 1 : 0; g.scale = scale;
  g.vec_q = strided_alignment(q, q_strides, 2) == 16;
  g.vec_o = strided_alignment(out, o_strides, 2) == 16;
  g.lost = lost; g.wait_ns = wait_ns;
  return launch_kv8_attention(g, ws, (cudaStream_t)stream);
}

gptq_status gptq_kv8_attention(const void *q, const int64_t *q_strides, int dtype, int64_t n_seq,
                               int64_t n_new, int n_heads, int n_kv, int dim, const uint8_t *k,
                               const uint8_t *v, const uint8_t *k_exps, const uint8_t *v_exps,
                               int64_t n_blocks, const int32_t *table, int64_t ld_table,
                               int64_t max_blocks, const int32_t *lengths, int causal,
                               float scale, void *out, const int64_t *o_strides, void *ws,
                               size_t ws_bytes, gptq_stream_t stream) {
  return kv8_attention_checked(q, q_strides, dtype, n_seq, n_new, n_heads, n_kv, dim, k, v, k_exps,
                               v_exps, n_blocks, table, ld_table, max_blocks, lengths, causal,
                               scale, out, o_strides, -1, tc::kWaitNs, ws, ws_bytes, stream);
}

gptq_status gptq_debug_kv8_attention_lost_copy(
    const void *q, const int64_t *q_strides, int dtype, int64_t n_seq, int64_t n_new, int n_heads,
    int n_kv, int dim, const uint8_t *k, const uint8_t *v, const uint8_t *k_exps,
    const uint8_t *v_exps, int64_t n_blocks, const int32_t *table, int64_t ld_table,
    int64_t max_blocks, const int32_t *lengths, int causal, float scale, void *out,
    const int64_t *o_strides, int64_t lost_copy, uint64_t wait_ns, void *ws, size_t ws_bytes,
    gptq_stream_t stream) {
  if (!lost_ok(lost_copy, wait_ns)) return GPTQ_ERR_INVALID_ARG;
  GPTQ_TRY(kv8_attention_checked(q, q_strides, dtype, n_seq, n_new, n_heads, n_kv, dim, k, v, k_exps,
                                 v_exps, n_blocks, table, ld_table, max_blocks, lengths, causal,
                                 scale, out, o_strides, lost_copy, wait_ns, ws, ws_bytes, stream));
  return gptq_workspace_status(ws, stream);
}

}  // extern "C"
