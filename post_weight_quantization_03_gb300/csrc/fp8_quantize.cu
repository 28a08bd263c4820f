// Making e4m3 operands: the RMS norm with the residual's addition and an 8-bit output, the
// plain quantizer of activations (1 x 128 blocks) and weights (128 x 128 blocks), and GPTQ's
// packed codes as exact e4m3 integers.
//
// Norm: h = x + r, u = h * w, rstd = (mean(h^2) + eps)^-1/2, y = rstd * u.  rstd is one factor
// per row and e4m3 is a floating format, so quantizing u and keeping rstd as the row's scale
// (which the product's epilogue applies) loses nothing against quantizing y, and the codes do
// not wait for the row's sum: the kernel reads x and r once, writes h and the codes in the same
// pass, and only the 4-byte rstd needs the whole row.  HBM-bound: 7 bytes an element for 16-bit
// x with a residual (8192 x 8192: 73 us, 6.4 TB/s; 1 x 4096: 2.3 us, a launch and two latencies).
// Without one, 3 bytes, the issue slots come first (73 % taken): 51 us, 3.9 TB/s.
#include <type_traits>

#include "fp8.cuh"

namespace gptq {

namespace {

using fp8::from_f32;
using fp8::kVec;   // elements per lane: 16 lanes cover one 128-element block
using fp8::Raw8;
constexpr int kMaxRowThreads = 512;

// The largest finite magnitude of a half-warp's 128 elements; infinities become NaN (they would
// saturate).  Whole warp.  Looking at each element's exponent takes as many instructions as the
// rest of the element's way, so only a block in which the plain maximum is infinite does it.
__device__ __forceinline__ float block_max(float (&v)[kVec]) {
  auto reduce = [](float a) {
#pragma unroll
    for (int o = 8; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
  };
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) amax = fmaxf(amax, fabsf(v[i]));
  amax = reduce(amax);
  if (__any_sync(0xffffffffu, amax == INFINITY)) {
    amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      amax = fmaxf(amax, fp8::finite_abs(v[i]));
      v[i] = fp8::inf_to_nan(v[i]);
    }
    amax = reduce(amax);
  }
  return amax;
}

// Codes of eight elements (none infinite) scaled by `inv`; rows of codes are 16-byte aligned.
__device__ __forceinline__ void store_codes8(uint8_t *__restrict__ p, int64_t n,
                                             const float (&u)[8], float inv) {
  float c[8];
#pragma unroll
  for (int i = 0; i < kVec; ++i) c[i] = u[i] * inv;
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
  int vx, vr, vw, vh;              // alignment of each pointer's rows
};

// Whole CTA: (mean square + eps)^-1/2 of its row, `sq` being a thread's sum of squares.  A row whose
// sum passes fp32's range is read again by one warp (as H, where H has replaced X or R) and its
// squares summed as multiples of 2^192; an infinity gives 0 still, a NaN has not come here.
template <typename T>
__device__ __forceinline__ void store_rstd(const RowsParams &p, int64_t row, float sq) {
  __shared__ float part[kMaxRowThreads / 32];
  const int lane = threadIdx.x % 32;
  auto reduce = [](float a) {
#pragma unroll
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
  };
  sq = reduce(sq);
  if (lane == 0) part[threadIdx.x / 32] = sq;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  sq = reduce(threadIdx.x < blockDim.x / 32 ? part[threadIdx.x] : 0.0f);
  float rstd = 1.0f / sqrtf(sq / (float)p.d + p.eps);
  if (sq == INFINITY) {
    const bool in_place = p.h && (p.h == p.x || p.h == p.r);
    const T *x = in_place ? (const T *)p.h + row * p.ldh : (const T *)p.x + row * p.ldx;
    const T *r = in_place || !p.r ? nullptr : (const T *)p.r + row * p.ldr;
    float big = 0.0f;
#pragma unroll 1
    for (int64_t c = lane; c < p.d; c += 32) {
      const float v = (r ? to_f32(x[c]) + to_f32(r[c]) : to_f32(x[c])) * 0x1p-96f;
      big = fmaf(v, v, big);
    }
    rstd = 0x1p-96f / sqrtf(reduce(big) / (float)p.d);
  }
  if (threadIdx.x == 0) p.rstd[row] = rstd;
}

// One CTA per row; half-warps take 128-element blocks, a thread VPT pieces of eight.  All of a
// thread's loads are asked for before its stores, which the compiler may not move them past.
// CTAS an SM at least (of 512 threads): two, or three where rows queue for long.  Three leave 40
// registers a thread, so a row's loads are not all in flight, but more rows' are: what the
// memory's latency is hidden by in a long queue, and a longer way for each row in a short one
// (bf16 with a residual: 8192 x 8192 85 us with two and 73 us, 6.4 TB/s, with three; 4000 x 4096
// 22.7 and 19.5; but 1336 x 1728 4.5 and 5.4, 907 x 6144 6.9 and 6.8).
template <typename T, typename TW, int VPT, int CTAS>
__global__ void __launch_bounds__(kMaxRowThreads, CTAS)
rows_kernel(RowsParams p) {
  wait_for_grids();
  launch_dependents();
  const int lane = threadIdx.x % 32;
  const int64_t row = blockIdx.x;
  Raw8<T> x[VPT], r[VPT];
  Raw8<TW> w[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int64_t c = ((int64_t)threadIdx.x + (int64_t)j * blockDim.x) * kVec, n = p.d - c;
    x[j].load((const T *)p.x + row * p.ldx + c, n, p.vx);
    if (p.r) r[j].load((const T *)p.r + row * p.ldr + c, n, p.vr);
    if (p.w) w[j].load((const TW *)p.w + c, n, p.vw);
  }
  float sq = 0.0f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int64_t c = ((int64_t)threadIdx.x + (int64_t)j * blockDim.x) * kVec, n = p.d - c;
    float v[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      v[i] = p.r ? x[j].get(i) + r[j].get(i) : x[j].get(i);
      sq = fmaf(v[i], v[i], sq);
    }
    if (p.h && n > 0) {
      Raw8<T> h;
      h.set(v);
      h.store((T *)p.h + row * p.ldh + c, n, p.vh);
    }
    if (p.w) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] *= w[j].get(i);
    }
    const int e = fp8::block_exponent(block_max(v));
    if (n > 0) {
      store_codes8(p.codes + row * p.ldc + c, n, v, fp8::pow2(-e));
      if ((lane & 15) == 0) p.exps[row * p.lde + c / fp8::kBlock] = (uint8_t)(e + fp8::kBias);
    }
  }
  if (p.rstd) store_rstd<T>(p, row, sq);
}

// Rows too wide for a thread's registers: one CTA per row, its pieces in a loop.
template <typename T, typename TW>
__global__ void __launch_bounds__(kMaxRowThreads) wide_rows_kernel(RowsParams p) {
  wait_for_grids();
  launch_dependents();
  const int64_t row = blockIdx.x;
  const T *x = (const T *)p.x + row * p.ldx;
  const T *r = p.r ? (const T *)p.r + row * p.ldr : nullptr;
  const int lane = threadIdx.x % 32;
  float sq = 0.0f;
  // whole warps iterate together: the half-warp past the row's end computes on zeros
  for (int64_t base = (int64_t)(threadIdx.x - lane) * kVec; base < p.d;
       base += (int64_t)blockDim.x * kVec) {
    const int64_t c = base + lane * kVec, n = p.d - c;
    Raw8<T> xq, rq;
    Raw8<TW> wq;
    xq.load(x + c, n, p.vx);
    if (r) rq.load(r + c, n, p.vr);
    if (p.w) wq.load((const TW *)p.w + c, n, p.vw);
    float v[8];
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = r ? xq.get(i) + rq.get(i) : xq.get(i);
    if (p.h && n > 0) {
      Raw8<T> h;
      h.set(v);
      h.store((T *)p.h + row * p.ldh + c, n, p.vh);
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      sq = fmaf(v[i], v[i], sq);
      if (p.w) v[i] *= wq.get(i);
    }
    const int e = fp8::block_exponent(block_max(v));
    if (n > 0) {
      store_codes8(p.codes + row * p.ldc + c, n, v, fp8::pow2(-e));
      if ((lane & 15) == 0) p.exps[row * p.lde + c / fp8::kBlock] = (uint8_t)(e + fp8::kBias);
    }
  }
  if (p.rstd) store_rstd<T>(p, row, sq);
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
    Raw8<T> q;
    q.load(x + row * ldx + c, row < rows ? n : 0, vx);
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[j][i] = q.get(i);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      amax = fmaxf(amax, fp8::finite_abs(v[j][i]));
      v[j][i] = fp8::inf_to_nan(v[j][i]);
    }
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

int rows_aligned(const void *p, int64_t ld, size_t es) { return fp8::alignment(p, ld * (int64_t)es); }

template <typename T, typename TW>
gptq_status run_rows_of(const RowsParams &p, cudaStream_t s) {
  int sms = 0;
  GPTQ_TRY(device_sm_count(&sms));
  const int64_t pieces = ceil_div(p.d, kVec);
  // pieces a thread: one while all rows run at once (latency), two where they queue (loads in
  // flight); what is wider than four pieces of 512 threads goes in a loop
  const int vpt = pieces > 2 * kMaxRowThreads ? 4 : (pieces > kMaxRowThreads || p.rows > 8 * sms ? 2 : 1);
  if (pieces > 4 * kMaxRowThreads)
    return launch_early(wide_rows_kernel<T, TW>, dim3((unsigned)p.rows), dim3(kMaxRowThreads), 0, 1,
                        s, p);
  const dim3 grid((unsigned)p.rows), block((unsigned)(ceil_div(ceil_div(pieces, vpt), 32) * 32));
  if constexpr (sizeof(T) + sizeof(TW) == 4)
    if (vpt == 2 && (double)p.rows * block.x > 4.0 * sms * 2 * kMaxRowThreads)
      return launch_early(rows_kernel<T, TW, 2, 3>, grid, block, 0, 1, s, p);
  switch (vpt) {
    case 1: return launch_early(rows_kernel<T, TW, 1, 2>, grid, block, 0, 1, s, p);
    case 2: return launch_early(rows_kernel<T, TW, 2, 2>, grid, block, 0, 1, s, p);
    default: return launch_early(rows_kernel<T, TW, 4, 2>, grid, block, 0, 1, s, p);
  }
}

gptq_status run_rows(RowsParams p, int xdtype, int wdtype, cudaStream_t s) {
  if (p.rows == 0) return GPTQ_OK;
  const size_t es = xdtype == GPTQ_F32 ? 4 : 2, wes = wdtype == GPTQ_F32 ? 4 : 2;
  p.vx = rows_aligned(p.x, p.ldx, es);
  p.vr = rows_aligned(p.r, p.ldr, es);
  p.vh = rows_aligned(p.h, p.ldh, es);
  p.vw = rows_aligned(p.w, 0, wes);
  switch (xdtype) {
    case GPTQ_F32: return run_rows_of<float, float>(p, s);
    case GPTQ_F16:
      return wdtype == GPTQ_F32 ? run_rows_of<__half, float>(p, s) : run_rows_of<__half, __half>(p, s);
    default:
      return wdtype == GPTQ_F32 ? run_rows_of<__nv_bfloat16, float>(p, s)
                                : run_rows_of<__nv_bfloat16, __nv_bfloat16>(p, s);
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
