// The block-scaled e4m3 product
//   out[m, n] = ra_m rw_n sum_kb 2^(EA[m, kb] - 127) 2^(EW[n / 128, kb] - 127) sum_{k in kb} a w.
#include <type_traits>

#include "fp8.cuh"

namespace gptq {

namespace {

template <typename TO>
__device__ __forceinline__ TO out_f32(float x) {
  if constexpr (std::is_same<TO, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// CUDA cores: 64 x 64 outputs per CTA, 4 x 4 per thread, 16 elements of K at a time.
template <typename TO>
__global__ void __launch_bounds__(256)
matmul_simt_kernel(const uint8_t *__restrict__ a, int64_t lda, const uint8_t *__restrict__ ae,
                   int64_t ldae, const float *__restrict__ ra, const uint8_t *__restrict__ w,
                   int64_t ldw, const uint8_t *__restrict__ we, int64_t ldwe,
                   const float *__restrict__ rw, int64_t M, int64_t N, int64_t K,
                   TO *__restrict__ out, int64_t ldo) {
  __shared__ float As[16][64 + 4], Ws[16][64 + 4];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += 16) {
    const int64_t kb = k0 / fp8::kBlock;
    for (int e = threadIdx.x; e < 16 * 64; e += 256) {
      const int kk = e % 16, rr = e / 16;
      const int64_t m = m0 + rr, n = n0 + rr, k = k0 + kk;
      As[kk][rr] = (m < M && k < K)
                       ? fp8::unpack1(a[m * lda + k]) * fp8::exp_value(ae[m * ldae + kb]) : 0.f;
      Ws[kk][rr] = (n < N && k < K) ? fp8::unpack1(w[n * ldw + k]) *
                                          fp8::exp_value(we[n / fp8::kBlock * ldwe + kb]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = fmaf(As[kk][4 * ty + i], Ws[kk][4 * tx + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + 4 * ty + i, n = n0 + 4 * tx + j;
      if (m < M && n < N)
        out[m * ldo + n] = out_f32<TO>(acc[i][j] * (ra ? ra[m] : 1.f) * (rw ? rw[n] : 1.f));
    }
}

}  // namespace

size_t fp8_matmul_ws_bytes(int64_t, int64_t, int64_t) { return 256; }

gptq_status launch_fp8_matmul(const Fp8MatmulArgs &g, void *ws, cudaStream_t s) {
  GPTQ_CUDA_CHECK(cudaMemsetAsync(ws, 0, sizeof(DevStatus), s));
  if (g.M == 0) return GPTQ_OK;
  const dim3 grid((unsigned)ceil_div(g.N, 64), (unsigned)ceil_div(g.M, 64));
  if (g.odtype == GPTQ_F16)
    return launch_kernel(matmul_simt_kernel<__half>, grid, dim3(256), 0, s, g.a, g.lda, g.ae,
                         g.ldae, g.ra, g.w, g.ldw, g.we, g.ldwe, g.rw, g.M, g.N, g.K,
                         (__half *)g.out, g.ldo);
  return launch_kernel(matmul_simt_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, g.a, g.lda, g.ae,
                       g.ldae, g.ra, g.w, g.ldw, g.we, g.ldwe, g.rw, g.M, g.N, g.K,
                       (__nv_bfloat16 *)g.out, g.ldo);
}

}  // namespace gptq
