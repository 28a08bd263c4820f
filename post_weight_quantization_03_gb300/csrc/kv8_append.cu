// Appending new keys and values to the 8-bit cache.
//
// The cache holds blocks of 64 tokens; block b of head h keeps K codes [64, D] (a token's
// elements together), V codes [D, 64] (a channel's tokens together: the order in which the
// product of probabilities and values reads them) and one exponent byte for each of the two.
// New tokens raise a block's exponent to what they need; the block's older codes are then
// re-rounded by that power of two (exact but for codes that become subnormal).
//
// A token whose value vector holds something that is not finite gets zero codes there and NaN
// codes in its key: whoever attends to it gets NaN (as it should), and whoever does not is
// untouched, since a masked score is replaced while a masked value is only multiplied by zero.
#include "fp8.cuh"

namespace gptq {

namespace {

constexpr int kTok = GPTQ_KV8_BLOCK;
constexpr int kAThreads = 256;

// One CTA per (touched block, head, sequence); D is the head's width (64 or 128).
template <typename T, int D>
__global__ void __launch_bounds__(kAThreads) append_kernel(Kv8AppendArgs g) {
  constexpr int kVecs = D / 8;                       // 8-element pieces of a token
  constexpr int kIter = kTok * kVecs / kAThreads;    // pieces per thread: 2 or 4
  __shared__ alignas(16) uint8_t sv[D * kTok];
  __shared__ float part[2][kAThreads / 32];
  __shared__ int bad[kTok];

  const int seq = blockIdx.z, head = blockIdx.y;
  const int64_t start = g.start[seq];
  if (start < 0) return;
  const int64_t blk = start / kTok + blockIdx.x;
  const int64_t t0 = blk * kTok;
  const int64_t lo64 = start > t0 ? start - t0 : 0;
  int64_t hi64 = start + g.n_new - t0;
  if (hi64 > kTok) hi64 = kTok;
  if (lo64 >= hi64 || blk >= g.max_blocks) return;
  const int lo = (int)lo64, hi = (int)hi64;
  const int64_t page = g.table[seq * g.ld_table + blk];
  if (page < 0 || page >= g.n_blocks) return;
  const int64_t ph = page * g.n_kv + head;
  uint8_t *kc = g.k + ph * (int64_t)(kTok * D), *vc = g.v + ph * (int64_t)(kTok * D);

  if (threadIdx.x < kTok) bad[threadIdx.x] = 0;
  __syncthreads();

  // the new tokens' pieces, in registers between the maximum and the conversion
  const T *ks = (const T *)g.new_k + seq * g.k_stride[0] + head * g.k_stride[2];
  const T *vs = (const T *)g.new_v + seq * g.v_stride[0] + head * g.v_stride[2];
  float kx[kIter][8], vx[kIter][8];
  float ka = 0.f, va = 0.f;
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    const int i = threadIdx.x + kAThreads * j, slot = i / kVecs, d = i % kVecs * 8;
    const bool fresh = slot >= lo && slot < hi;
    const int64_t tok = t0 + slot - start;
    const T *kp = ks + tok * g.k_stride[1] + d, *vp = vs + tok * g.v_stride[1] + d;
    if (fresh && g.vec_k) {
      alignas(16) T e[8];
#pragma unroll
      for (int q = 0; q < (int)sizeof(e) / 16; ++q)
        reinterpret_cast<uint4 *>(e)[q] = reinterpret_cast<const uint4 *>(kp)[q];
#pragma unroll
      for (int q = 0; q < 8; ++q) kx[j][q] = to_f32(e[q]);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) kx[j][q] = fresh ? to_f32(kp[q]) : 0.f;
    }
    if (fresh && g.vec_v) {
      alignas(16) T e[8];
#pragma unroll
      for (int q = 0; q < (int)sizeof(e) / 16; ++q)
        reinterpret_cast<uint4 *>(e)[q] = reinterpret_cast<const uint4 *>(vp)[q];
#pragma unroll
      for (int q = 0; q < 8; ++q) vx[j][q] = to_f32(e[q]);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) vx[j][q] = fresh ? to_f32(vp[q]) : 0.f;
    }
    bool b = false;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      ka = fmaxf(ka, fp8::finite_abs(kx[j][q]));
      va = fmaxf(va, fp8::finite_abs(vx[j][q]));
      b |= !fp8::finite(vx[j][q]);
      if (!fp8::finite(vx[j][q])) vx[j][q] = 0.f;
    }
    if (b) bad[slot] = 1;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    ka = fmaxf(ka, __shfl_xor_sync(0xffffffffu, ka, o));
    va = fmaxf(va, __shfl_xor_sync(0xffffffffu, va, o));
  }
  if (threadIdx.x % 32 == 0) {
    part[0][threadIdx.x / 32] = ka;
    part[1][threadIdx.x / 32] = va;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAThreads / 32; ++i) {
    ka = fmaxf(ka, part[0][i]);
    va = fmaxf(va, part[1][i]);
  }
  int ke = fp8::block_exponent(ka), ve = fp8::block_exponent(va);
  int kd = 0, vd = 0;  // how far the older codes' exponents are raised
  if (lo > 0) {
    const int k_was = (int)g.k_exps[ph] - fp8::kBias, v_was = (int)g.v_exps[ph] - fp8::kBias;
    if (k_was >= ke) ke = k_was; else kd = ke - k_was;
    if (v_was >= ve) ve = v_was; else vd = ve - v_was;
  }
  const float ki = fp8::pow2(-ke), vi = fp8::pow2(-ve);
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    const int i = threadIdx.x + kAThreads * j, slot = i / kVecs, d = i % kVecs * 8;
    if (slot < lo || slot >= hi) continue;
    float c[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      c[q] = bad[slot] ? __uint_as_float(0x7FC00000u) : fp8::inf_to_nan(kx[j][q]) * ki;
    *reinterpret_cast<uint2 *>(kc + slot * D + d) =
        make_uint2(fp8::pack4(c[0], c[1], c[2], c[3]), fp8::pack4(c[4], c[5], c[6], c[7]));
#pragma unroll
    for (int q = 0; q < 8; q += 2) {
      const uint32_t two = fp8::pack2(vx[j][q] * vi, vx[j][q + 1] * vi);
      sv[(d + q) * kTok + slot] = (uint8_t)two;
      sv[(d + q + 1) * kTok + slot] = (uint8_t)(two >> 8);
    }
  }
  // older codes under a raised exponent (a difference past 126 leaves only zeros)
  if (kd > 0) {
    const float f = kd > 126 ? 0.f : fp8::pow2(-kd);
    for (int i = threadIdx.x; i < lo * D / 2; i += kAThreads) {
      uint16_t *p = reinterpret_cast<uint16_t *>(kc) + i;
      const float2 c = fp8::unpack2(*p);
      *p = (uint16_t)fp8::pack2(c.x * f, c.y * f);
    }
  }
  if (vd > 0) {
    const float f = vd > 126 ? 0.f : fp8::pow2(-vd);
    for (int i = threadIdx.x; i < lo * D; i += kAThreads) {
      const int at = i / lo * kTok + i % lo;
      sv[at] = (uint8_t)fp8::pack2(fp8::unpack1(vc[at]) * f, 0.f);
    }
  }
  __syncthreads();
  const int from = vd > 0 ? 0 : lo, width = hi - from;
  if (width == kTok) {
    for (int i = threadIdx.x; i < D * kTok / 16; i += kAThreads)
      reinterpret_cast<uint4 *>(vc)[i] = reinterpret_cast<const uint4 *>(sv)[i];
  } else {
    for (int i = threadIdx.x; i < D * width; i += kAThreads) {
      const int at = i / width * kTok + from + i % width;
      vc[at] = sv[at];
    }
  }
  if (threadIdx.x == 0) {
    g.k_exps[ph] = (uint8_t)(ke + fp8::kBias);
    g.v_exps[ph] = (uint8_t)(ve + fp8::kBias);
  }
}

template <typename T>
gptq_status launch_any(const Kv8AppendArgs &g, dim3 grid, cudaStream_t s) {
  if (g.dim == 64) return launch_kernel(append_kernel<T, 64>, grid, dim3(kAThreads), 0, s, g);
  return launch_kernel(append_kernel<T, 128>, grid, dim3(kAThreads), 0, s, g);
}

}  // namespace

gptq_status launch_kv8_append(const Kv8AppendArgs &g, cudaStream_t s) {
  if (g.n_seq == 0 || g.n_new == 0) return GPTQ_OK;
  const dim3 grid((unsigned)((g.n_new + 2 * (kTok - 1)) / kTok), (unsigned)g.n_kv,
                  (unsigned)g.n_seq);
  switch (g.dtype) {
    case GPTQ_F32: return launch_any<float>(g, grid, s);
    case GPTQ_F16: return launch_any<__half>(g, grid, s);
    default: return launch_any<__nv_bfloat16>(g, grid, s);
  }
}

}  // namespace gptq
