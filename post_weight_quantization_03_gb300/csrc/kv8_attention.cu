// Attention over the 8-bit cache.
#include <type_traits>

#include "fp8.cuh"

namespace gptq {

namespace {

constexpr int kTok = GPTQ_KV8_BLOCK;

template <typename T>
__device__ __forceinline__ T from_f32(float x) {
  if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// One warp per (sequence, new token, head): 32 tokens at a time, a lane per token for the
// scores and D / 32 channels per lane for the output.
template <typename T, int D>
__global__ void __launch_bounds__(128) attention_rows_kernel(Kv8AttentionArgs g) {
  __shared__ float sq[4][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t r = (int64_t)blockIdx.x * 4 + warp;
  if (r >= (int64_t)g.n_seq * g.n_new * g.n_heads) return;
  const int head = (int)(r % g.n_heads);
  const int64_t t = r / g.n_heads % g.n_new, seq = r / g.n_heads / g.n_new;
  const int kvh = head / (g.n_heads / g.n_kv);
  const T *q = (const T *)g.q + seq * g.q_stride[0] + t * g.q_stride[1] + head * g.q_stride[2];
  T *o = (T *)g.out + seq * g.o_stride[0] + t * g.o_stride[1] + head * g.o_stride[2];
  for (int d = lane; d < D; d += 32) sq[warp][d] = to_f32(q[d]) * g.scale;
  __syncwarp();
  int64_t len = g.lengths[seq];
  const int64_t cap = (int64_t)g.max_blocks * kTok;
  len = len < 0 ? 0 : (len > cap ? cap : len);
  int64_t end = g.causal ? len - g.n_new + t + 1 : len;
  float m = -INFINITY, l = 0.f, acc[D / 32] = {};
  for (int64_t j0 = 0; j0 < end; j0 += 32) {
    const int64_t page = g.table[seq * g.ld_table + j0 / kTok];
    if (page < 0 || page >= g.n_blocks) continue;
    const int64_t ph = page * g.n_kv + kvh;
    const uint8_t *kc = g.k + ph * (kTok * D), *vc = g.v + ph * (kTok * D);
    const float ks = fp8::exp_value(g.k_exps[ph]), vs = fp8::exp_value(g.v_exps[ph]);
    const int slot = (int)(j0 % kTok) + lane;
    const bool seen = j0 + lane < end;
    float s = -INFINITY;
    if (seen) {
      s = 0.f;
      for (int d = 0; d < D; ++d) s = fmaf(sq[warp][d], fp8::unpack1(kc[slot * D + d]), s);
      s *= ks;
    }
    float mx = s;
    for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    const float mn = fmaxf(m, mx), f = __expf(m - mn);
    const float pr = seen ? __expf(s - mn) : 0.f;
    m = mn;
    l = l * f + pr;
    for (int i = 0; i < D / 32; ++i) {
      float a = 0.f;
      for (int w = 0; w < 32; ++w) {
        const float pw = __shfl_sync(0xffffffffu, pr, w);
        if (j0 + w < end) a = fmaf(pw, fp8::unpack1(vc[(lane + 32 * i) * kTok + slot - lane + w]), a);
      }
      acc[i] = acc[i] * f + a * vs;
    }
  }
  for (int w = 16; w; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  for (int i = 0; i < D / 32; ++i)
    o[lane + 32 * i] = from_f32<T>(m == -INFINITY && l == 0.f ? 0.f : acc[i] / l);
}

}  // namespace

size_t kv8_attention_ws_bytes(int, int64_t, int, int, int, int) { return 256; }

gptq_status launch_kv8_attention(const Kv8AttentionArgs &g, void *ws, cudaStream_t s) {
  GPTQ_CUDA_CHECK(cudaMemsetAsync(ws, 0, sizeof(DevStatus), s));
  const int64_t rows = (int64_t)g.n_seq * g.n_new * g.n_heads;
  if (rows == 0) return GPTQ_OK;
  const dim3 grid((unsigned)ceil_div(rows, 4));
  if (g.dtype == GPTQ_F16)
    return g.dim == 64 ? launch_kernel(attention_rows_kernel<__half, 64>, grid, dim3(128), 0, s, g)
                       : launch_kernel(attention_rows_kernel<__half, 128>, grid, dim3(128), 0, s, g);
  return g.dim == 64
             ? launch_kernel(attention_rows_kernel<__nv_bfloat16, 64>, grid, dim3(128), 0, s, g)
             : launch_kernel(attention_rows_kernel<__nv_bfloat16, 128>, grid, dim3(128), 0, s, g);
}

}  // namespace gptq
