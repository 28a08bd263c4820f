// Block-scaled e4m3 products with an epilogue, of one weight matrix or of one for each expert:
//   out = act(ra rw (A W^T) + bias) + residual                       (16 bits)
//   v = act(G) * U, G and U two such products of one A               (e4m3 codes by 1 x 128 blocks)
// Plain kernel: a CTA takes one position and 128 columns, a thread one column.
#include <math.h>

#include <type_traits>

#include "fp8.cuh"

namespace gptq {

namespace {

constexpr int BM = 128;

__device__ int g_gave_up;  // a wait ran out since it was last asked for

__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {
    case GPTQ_ACT_RELU: return x < 0.0f ? 0.0f : x;
    case GPTQ_ACT_SILU: return x / (1.0f + expf(-x));
    case GPTQ_ACT_GELU: return 0.5f * x * (1.0f + erff(x * 0.70710678f));
    default: return x;
  }
}

// Where expert e's positions end, limited and increasing.
__device__ __forceinline__ int64_t ends(const Fp8LinearArgs &g, int e) {
  int64_t most = 0;
  for (int i = 0; i <= e; ++i) most = max(most, (int64_t)g.offsets[i + 1]);
  return min(most, g.M);
}

template <typename TO>
__global__ void __launch_bounds__(BM) plain_kernel(Fp8LinearArgs g) {
  __shared__ float part[BM / 32];
  const int64_t n_w = ceil_div(g.N, (int64_t)BM), pos = blockIdx.x / n_w, nb = blockIdx.x % n_w;
  const int64_t n = nb * BM + threadIdx.x;
  int64_t e = 0, row = pos, out_row = pos;
  if (g.n_experts > 0) {
    for (e = 0; e < g.n_experts && pos >= ends(g, (int)e); ++e) {}
    if (e == g.n_experts || pos < min(max(g.offsets[0], 0), (int)g.M)) return;
    const int64_t o = g.order[pos];
    if (g.gated) row = o < 0 ? -1 : o / g.top_k;
    else out_row = o;
    if (row >= g.a_rows) row = -1;
    if (out_row < 0 || out_row >= g.M) return;
  }
  float acc[2] = {0.0f, 0.0f};
  if (n < g.N && row >= 0) {
    for (int j = 0; j < (g.gated ? 2 : 1); ++j) {
      const uint8_t *w = g.w[j].codes + e * g.w[j].next_codes + n * g.w[j].ld;
      const uint8_t *we = g.w[j].exps + e * g.w[j].next_exps + nb * g.w[j].ld_exps;
      for (int64_t kb = 0; kb * BM < g.K; ++kb) {
        float s = 0.0f;
        for (int64_t k = kb * BM; k < min(g.K, (kb + 1) * BM); ++k)
          s = fmaf(fp8::unpack1(g.a[row * g.lda + k]), fp8::unpack1(w[k]), s);
        acc[j] = fmaf(s, fp8::exp_value(g.ae[row * g.ldae + kb]) * fp8::exp_value(we[kb]), acc[j]);
      }
    }
  }
  const float ra = g.ra && row >= 0 ? g.ra[row] : 1.0f;
  float v[2];
  for (int j = 0; j < (g.gated ? 2 : 1); ++j) {
    const int64_t at = e * g.N + n;
    v[j] = acc[j] * (g.w[j].scale && n < g.N ? g.w[j].scale[at] : 1.0f) * ra;
    if (g.w[j].bias && n < g.N) v[j] += g.w[j].bias[at];
  }
  float x = activate(v[0], g.act);
  if (!g.gated) {
    if (n >= g.N) return;
    if (g.residual) x += to_f32(((const TO *)g.residual)[out_row * g.ldr + n]);
    ((TO *)g.out)[out_row * g.ldo + n] = fp8::from_f32<TO>(x);
    return;
  }
  x = n < g.N ? x * v[1] : 0.0f;
  float most = fp8::finite_abs(x);
  for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = most;
  __syncthreads();
  for (int i = 0; i < BM / 32; ++i) most = fmaxf(most, part[i]);
  const int ex = fp8::block_exponent(most);
  if (n < g.N) ((uint8_t *)g.out)[pos * g.ldo + n] = (uint8_t)fp8::pack2(fp8::inf_to_nan(x) * fp8::pow2(-ex), 0.0f);
  if (threadIdx.x == 0) g.oe[pos * g.ldoe + nb] = (uint8_t)(ex + fp8::kBias);
}

}  // namespace

size_t fp8_linear_ws_bytes(int64_t, int64_t, int64_t) { return 256; }

gptq_status fp8_linear_take_timeout(int *out, cudaStream_t s) { return take_flag(g_gave_up, out, s); }

gptq_status launch_fp8_linear(const Fp8LinearArgs &g, void *ws, cudaStream_t s) {
  GPTQ_CUDA_CHECK(cudaMemsetAsync(ws, 0, sizeof(DevStatus), s));
  if (g.M == 0) return GPTQ_OK;
  const int64_t ctas = g.M * ceil_div(g.N, (int64_t)BM);
  if (ctas > INT32_MAX) return GPTQ_ERR_UNSUPPORTED;
  return !g.gated && g.odtype == GPTQ_F16
             ? launch_kernel(plain_kernel<__half>, dim3((unsigned)ctas), dim3(BM), 0, s, g)
             : launch_kernel(plain_kernel<__nv_bfloat16>, dim3((unsigned)ctas), dim3(BM), 0, s, g);
}

}  // namespace gptq
