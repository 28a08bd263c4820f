// Making e4m3 operands: the RMS norm with the residual's addition and an 8-bit output, the
// plain quantizer of activations (1 x 128 blocks) and weights (128 x 128 blocks), and GPTQ's
// packed codes as exact e4m3 integers.
//
// Norm: h = x + r, u = h * w, rstd = (mean(h^2) + eps)^-1/2, y = rstd * u.  rstd is one factor
// per row and e4m3 is a floating format, so quantizing u and keeping rstd as the row's scale
// (which the product's epilogue applies) loses nothing against quantizing y, and the codes do
// not wait for the row's sum: the kernel reads x and r once, writes h and the codes in the same
// pass, and only the 4-byte rstd needs the whole row.  HBM-bound: 7 bytes an element for 16-bit
// x with a residual.
#include <type_traits>

#include "fp8.cuh"

namespace gptq {

namespace {

constexpr int kVec = 8;               // elements per lane: 16 lanes cover one 128-element block
constexpr int kMaxRowThreads = 512;

// Eight elements at p (the first `n` exist; the others give 0).  `vec`: p is 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T *__restrict__ p, int64_t n, bool vec, float (&v)[8]) {
  if (vec && n >= kVec) {
    if constexpr (sizeof(T) == 4) {
      const float4 a = reinterpret_cast<const float4 *>(p)[0];
      const float4 b = reinterpret_cast<const float4 *>(p)[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 q = *reinterpret_cast<const uint4 *>(p);
      const T *e = reinterpret_cast<const T *>(&q);
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = to_f32(e[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = i < n ? to_f32(p[i]) : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ T from_f32(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

template <typename T>
__device__ __forceinline__ void store8(T *__restrict__ p, int64_t n, bool vec, const float (&v)[8]) {
  if (vec && n >= kVec) {
    alignas(16) T e[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) e[i] = from_f32<T>(v[i]);
#pragma unroll
    for (int i = 0; i < (int)sizeof(e) / 16; ++i)
      reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(e)[i];
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

// Codes of eight elements scaled by `inv`; rows of codes are 16-byte aligned.
__device__ __forceinline__ void store_codes8(uint8_t *__restrict__ p, int64_t n,
                                             const float (&u)[8], float inv) {
  float c[8];
#pragma unroll
  for (int i = 0; i < kVec; ++i) c[i] = fp8::inf_to_nan(u[i]) * inv;
  const uint2 w = make_uint2(fp8::pack4(c[0], c[1], c[2], c[3]), fp8::pack4(c[4], c[5], c[6], c[7]));
  if (n >= kVec) {
    *reinterpret_cast<uint2 *>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i < n) p[i] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
}

struct RowsParams {
  const void *x; int64_t ldx;
  const void *r; int64_t ldr;      // residual or null
  const void *w;                   // norm weight or null (plain quantizer)
  void *h; int64_t ldh;            // x + r out, or null
  uint8_t *codes; int64_t ldc;
  uint8_t *exps; int64_t lde;
  float *rstd;                     // null: plain quantizer
  int64_t rows, d;
  float eps;
  int vx, vr, vw, vh;              // 16-byte alignment of each pointer's rows
};

// One CTA per row; half-warps take its 128-element blocks in turn.
template <typename T, typename TW>
__global__ void __launch_bounds__(kMaxRowThreads) rows_kernel(RowsParams p) {
  __shared__ float part[kMaxRowThreads / 32];
  const int64_t row = blockIdx.x;
  const T *x = (const T *)p.x + row * p.ldx;
  const T *r = p.r ? (const T *)p.r + row * p.ldr : nullptr;
  T *h = p.h ? (T *)p.h + row * p.ldh : nullptr;
  const TW *w = (const TW *)p.w;
  uint8_t *codes = p.codes + row * p.ldc;
  uint8_t *exps = p.exps + row * p.lde;
  const int lane = threadIdx.x % 32;
  float sq = 0.0f;
  // whole warps iterate together: the half-warp past the row's end computes on zeros
  for (int64_t base = (int64_t)(threadIdx.x - lane) * kVec; base < p.d;
       base += (int64_t)blockDim.x * kVec) {
    const int64_t c = base + lane * kVec, n = p.d - c;
    float v[8], u[8];
    load8(x + c, n, p.vx, v);
    if (r) {
      load8(r + c, n, p.vr, u);
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] += u[i];
    }
    if (h && n > 0) store8(h + c, n, p.vh, v);
    if (w) {
      load8(w + c, n, p.vw, u);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        sq = fmaf(v[i], v[i], sq);
        u[i] *= v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) u[i] = v[i];
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) amax = fmaxf(amax, fp8::finite_abs(u[i]));
#pragma unroll
    for (int o = 8; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int e = fp8::block_exponent(amax);
    if (n > 0) {
      store_codes8(codes + c, n, u, fp8::pow2(-e));
      if ((lane & 15) == 0) exps[c / fp8::kBlock] = (uint8_t)(e + fp8::kBias);
    }
  }
  if (!p.rstd) return;
#pragma unroll
  for (int o = 16; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  if (lane == 0) part[threadIdx.x / 32] = sq;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) s += part[i];
    p.rstd[row] = 1.0f / sqrtf(s / (float)p.d + p.eps);
  }
}

// Weights: one CTA per 128 x 128 block, its values held in registers between the maximum and
// the conversion (64 per thread: 16 lanes x 8 columns, 16 rows at a time).
template <typename T>
__global__ void __launch_bounds__(256)
tiles_kernel(const T *__restrict__ x, int64_t ldx, int vx, int64_t rows, int64_t d,
             uint8_t *__restrict__ codes, int64_t ldc, uint8_t *__restrict__ exps, int64_t lde) {
  __shared__ float part[8];
  const int64_t r0 = (int64_t)blockIdx.y * fp8::kBlock + threadIdx.x / 16;
  const int64_t c = (int64_t)blockIdx.x * fp8::kBlock + (threadIdx.x % 16) * kVec, n = d - c;
  float v[8][8];
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t row = r0 + 16 * j;
    load8(x + row * ldx + c, row < rows ? n : 0, vx, v[j]);
#pragma unroll
    for (int i = 0; i < kVec; ++i) amax = fmaxf(amax, fp8::finite_abs(v[j][i]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, part[i]);
  const int e = fp8::block_exponent(amax);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t row = r0 + 16 * j;
    if (row < rows && n > 0) store_codes8(codes + row * ldc + c, n, v[j], fp8::pow2(-e));
  }
  if (threadIdx.x == 0) exps[blockIdx.y * lde + blockIdx.x] = (uint8_t)(e + fp8::kBias);
}

// GPTQ's packed codes: code - zero is an integer in [-15, 15] at up to 4 bits, exact in e4m3.
// One thread per eight columns; exponents are all 2^0.
__global__ void __launch_bounds__(256)
from_codes_kernel(const uint32_t *__restrict__ qp, int64_t words, int bits,
                  const int32_t *__restrict__ zero, int64_t m, int64_t d,
                  uint8_t *__restrict__ codes, int64_t ldc, uint8_t *__restrict__ exps,
                  int64_t lde) {
  const int64_t groups = ceil_div(d, (int64_t)kVec), total = m * groups;
  for (int64_t t = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; t < total;
       t += (int64_t)gridDim.x * blockDim.x) {
    const int64_t i = t / groups, c = t % groups * kVec;
    const uint32_t *row = qp + i * words;
    const int z = zero[i];
    float v[8];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      v[j] = 0.0f;
      if (c + j < d) {
        const int64_t bit = (c + j) * bits;
        uint64_t two = row[bit >> 5];
        if (((bit & 31) + bits) > 32) two |= (uint64_t)row[(bit >> 5) + 1] << 32;
        v[j] = (float)((int)((uint32_t)(two >> (bit & 31)) & ((1u << bits) - 1u)) - z);
      }
    }
    store_codes8(codes + i * ldc + c, d - c, v, 1.0f);
    if (i % fp8::kBlock == 0 && c % fp8::kBlock == 0)
      exps[i / fp8::kBlock * lde + c / fp8::kBlock] = (uint8_t)fp8::kBias;
  }
}

bool rows_aligned(const void *p, int64_t ld, size_t es) {
  return ((uintptr_t)p % 16) == 0 && (ld * (int64_t)es) % 16 == 0;
}

gptq_status run_rows(RowsParams p, int xdtype, int wdtype, cudaStream_t s) {
  if (p.rows == 0) return GPTQ_OK;
  const size_t es = xdtype == GPTQ_F32 ? 4 : 2, wes = wdtype == GPTQ_F32 ? 4 : 2;
  p.vx = rows_aligned(p.x, p.ldx, es);
  p.vr = p.r && rows_aligned(p.r, p.ldr, es);
  p.vh = p.h && rows_aligned(p.h, p.ldh, es);
  p.vw = p.w && rows_aligned(p.w, 0, wes);
  int64_t threads = ceil_div(ceil_div(p.d, kVec), 32) * 32;
  if (threads > kMaxRowThreads) threads = kMaxRowThreads;
  const dim3 grid((unsigned)p.rows), block((unsigned)threads);
  switch (xdtype) {
    case GPTQ_F32: return launch_kernel(rows_kernel<float, float>, grid, block, 0, s, p);
    case GPTQ_F16:
      return wdtype == GPTQ_F32
                 ? launch_kernel(rows_kernel<__half, float>, grid, block, 0, s, p)
                 : launch_kernel(rows_kernel<__half, __half>, grid, block, 0, s, p);
    default:
      return wdtype == GPTQ_F32
                 ? launch_kernel(rows_kernel<__nv_bfloat16, float>, grid, block, 0, s, p)
                 : launch_kernel(rows_kernel<__nv_bfloat16, __nv_bfloat16>, grid, block, 0, s, p);
  }
}

}  // namespace

gptq_status launch_rmsnorm_fp8(const void *X, int xdtype, int64_t rows, int64_t d, int64_t ldx,
                               const void *R, int64_t ldr, const void *weight, int wdtype,
                               float eps, void *H, int64_t ldh, uint8_t *codes, int64_t ldc,
                               uint8_t *exps, int64_t lde, float *rstd, cudaStream_t s) {
  RowsParams p{};
  p.x = X; p.ldx = ldx;
  p.r = R; p.ldr = ldr;
  p.w = weight;
  p.h = H; p.ldh = ldh;
  p.codes = codes; p.ldc = ldc;
  p.exps = exps; p.lde = lde;
  p.rstd = rstd;
  p.rows = rows; p.d = d; p.eps = eps;
  return run_rows(p, xdtype, wdtype, s);
}

gptq_status launch_fp8_quantize(const void *X, int xdtype, int64_t rows, int64_t d, int64_t ldx,
                                int row_block, uint8_t *codes, int64_t ldc, uint8_t *exps,
                                int64_t lde, cudaStream_t s) {
  if (rows == 0) return GPTQ_OK;
  if (row_block == 1) {
    RowsParams p{};
    p.x = X; p.ldx = ldx;
    p.codes = codes; p.ldc = ldc;
    p.exps = exps; p.lde = lde;
    p.rows = rows; p.d = d;
    return run_rows(p, xdtype, xdtype, s);
  }
  const int vx = rows_aligned(X, ldx, xdtype == GPTQ_F32 ? 4 : 2);
  const dim3 grid((unsigned)ceil_div(d, fp8::kBlock), (unsigned)ceil_div(rows, fp8::kBlock));
  switch (xdtype) {
    case GPTQ_F32:
      return launch_kernel(tiles_kernel<float>, grid, dim3(256), 0, s, (const float *)X, ldx, vx,
                           rows, d, codes, ldc, exps, lde);
    case GPTQ_F16:
      return launch_kernel(tiles_kernel<__half>, grid, dim3(256), 0, s, (const __half *)X, ldx,
                           vx, rows, d, codes, ldc, exps, lde);
    default:
      return launch_kernel(tiles_kernel<__nv_bfloat16>, grid, dim3(256), 0, s,
                           (const __nv_bfloat16 *)X, ldx, vx, rows, d, codes, ldc, exps, lde);
  }
}

gptq_status launch_fp8_from_codes(const uint32_t *qpacked, int bits, const int32_t *zero,
                                  int64_t m, int64_t d, uint8_t *codes, int64_t ldc,
                                  uint8_t *exps, int64_t lde, cudaStream_t s) {
  const int64_t blocks = ceil_div(m * ceil_div(d, kVec), 256);
  return launch_kernel(from_codes_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)),
                       dim3(256), 0, s, qpacked, ceil_div(d, 32) * bits, bits, zero, m, d, codes,
                       ldc, exps, lde);
}

}  // namespace gptq
