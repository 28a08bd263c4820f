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
//
// HBM-bound for prompts (a bf16 token read, half its bytes written): 4096 tokens of 8 heads of 128
// take 6.0 us, 4.2 TB/s.  For single tokens it is the chain of loads (start, table, token) and a
// launch: 3.1 us.
#include "fp8.cuh"

namespace gptq {

namespace {

using fp8::Raw8;

constexpr int kTok = GPTQ_KV8_BLOCK;
constexpr int kAThreads = 256;
constexpr int kFew = 4;        // up to so many new tokens take append_few_kernel

// Where a touched block of a sequence is, and which of its slots [lo, hi) are new.
struct Touched {
  int64_t ph;   // block and head; negative: nothing to write
  int lo, hi;
  int64_t tok;  // new token in slot 0 (negative where older tokens come first)
};
__device__ __forceinline__ Touched touched(const Kv8AppendArgs &g, int seq, int head, int nth) {
  Touched t{-1, 0, 0, 0};
  const int64_t start = g.start[seq];
  if (start < 0) return t;
  const int64_t blk = start / kTok + nth, t0 = blk * kTok;
  t.tok = t0 - start;
  const int64_t lo = t.tok < 0 ? -t.tok : 0, hi = g.n_new - t.tok < kTok ? g.n_new - t.tok : kTok;
  if (lo >= hi || blk >= g.max_blocks) return t;
  const int64_t page = g.table[seq * g.ld_table + blk];
  if (page < 0 || page >= g.n_blocks) return t;
  t.ph = page * g.n_kv + head;
  t.lo = (int)lo;
  t.hi = (int)hi;
  return t;
}

// The exponent of a block whose new tokens need `need`, and by how much its older codes' rises.
__device__ __forceinline__ int raised(int need, int lo, uint8_t was_byte, int &rise) {
  rise = 0;
  if (lo == 0) return need;
  const int was = (int)was_byte - fp8::kBias;
  if (was >= need) return was;
  rise = need - was;
  return need;
}
// 2^-rise; a rise past 126 leaves only zeros.
__device__ __forceinline__ float fall(int rise) { return rise > 126 ? 0.0f : fp8::pow2(-rise); }

// Older keys under a raised exponent: two codes at a time.
__device__ __forceinline__ void lower_keys(uint8_t *kc, int codes, int rise, int thread, int threads) {
  const float f = fall(rise);
  for (int i = thread; i < codes / 2; i += threads) {
    uint16_t *p = reinterpret_cast<uint16_t *>(kc) + i;
    const float2 c = fp8::unpack2(*p);
    *p = (uint16_t)fp8::pack2(c.x * f, c.y * f);
  }
}

// Prompts: one CTA per (touched block, head, sequence).  Keys: a thread takes pieces of eight
// elements of a token.  Values: eight channels of four tokens, so that the transposed codes go to
// shared memory as whole words in different banks and from there to the cache in rows.  Four CTAs
// an SM (64 registers): 4096 tokens are 520 CTAs, one round of four to an SM, but a full round
// and a short one of three (8.6 us against 6.0).
template <typename T, int D>
__global__ void __launch_bounds__(kAThreads, sizeof(T) == 4 ? 2 : 4) append_kernel(Kv8AppendArgs g) {
  constexpr int kVecs = D / 8;                       // pieces of a token
  constexpr int kIter = kTok * kVecs / kAThreads;    // keys: pieces per thread, 2 or 4
  __shared__ alignas(16) uint8_t sv[D * kTok];
  __shared__ uint32_t part[2][kAThreads / 32];
  __shared__ int bad[kTok];
  wait_for_grids();
  launch_dependents();
  const int seq = blockIdx.z, head = blockIdx.y, tid = threadIdx.x;
  const Touched b = touched(g, seq, head, blockIdx.x);
  if (b.ph < 0) return;
  const int lo = b.lo, hi = b.hi;
  uint8_t *kc = g.k + b.ph * (int64_t)(kTok * D), *vc = g.v + b.ph * (int64_t)(kTok * D);
  const uint8_t k_was = g.k_exps[b.ph], v_was = g.v_exps[b.ph];

  const T *ks = (const T *)g.new_k + seq * g.k_stride[0] + head * g.k_stride[2];
  const T *vs = (const T *)g.new_v + seq * g.v_stride[0] + head * g.v_stride[2];
  const int quad = tid % (kTok / 4) * 4, vd = tid / (kTok / 4) * 8;  // values: tokens, channels
  const bool has_v = vd < D;
  Raw8<T> kx[kIter], vx[4];
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    const int i = tid + kAThreads * j, slot = i / kVecs, d = i % kVecs * 8;
    kx[j].load(ks + (b.tok + slot) * g.k_stride[1] + d, slot >= lo && slot < hi ? 8 : 0, g.align_k);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int slot = quad + j;
    vx[j].load(vs + (b.tok + slot) * g.v_stride[1] + vd, has_v && slot >= lo && slot < hi ? 8 : 0,
               g.align_v);
  }
  uint32_t km = 0, vm = 0;  // largest magnitudes as fp32 bits
#pragma unroll
  for (int j = 0; j < kIter; ++j) km = kx[j].most(km);
#pragma unroll
  for (int j = 0; j < 4; ++j) vm = vx[j].most(vm);
  auto of_block = [&]() {
    km = __reduce_max_sync(0xffffffffu, km);
    vm = __reduce_max_sync(0xffffffffu, vm);
    if (tid % 32 == 0) {
      part[0][tid / 32] = km;
      part[1][tid / 32] = vm;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAThreads / 32; ++i) {
      km = max(km, part[0][i]);
      vm = max(vm, part[1][i]);
    }
  };
  km = Raw8<T>::most_bits(km);
  vm = Raw8<T>::most_bits(vm);
  of_block();
  if (max(km, vm) >= 0x7F800000u) {
    // Something is not finite (the whole CTA sees it): NaN in keys, and in all of the keys of a
    // token with such a value, zeros in values; the maxima are the others'.
    if (tid < kTok) bad[tid] = 0;
    __syncthreads();
    km = vm = 0;
    float e[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bool odd = false;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float x = vx[j].get(q);
        odd |= !fp8::finite(x);
        e[q] = fp8::finite(x) ? x : 0.0f;
        vm = max(vm, __float_as_uint(fabsf(e[q])));
      }
      vx[j].set(e);
      if (odd) bad[quad + j] = 1;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kIter; ++j) {
      const int slot = (tid + kAThreads * j) / kVecs;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float x = kx[j].get(q);
        km = max(km, __float_as_uint(fp8::finite_abs(x)));
        e[q] = bad[slot] ? __uint_as_float(0x7FC00000u) : fp8::inf_to_nan(x);
      }
      kx[j].set(e);
    }
    of_block();
  }
  const float ka = __uint_as_float(km), va = __uint_as_float(vm);
  int k_rise, v_rise;
  const int ke = raised(fp8::block_exponent(ka), lo, k_was, k_rise);
  const int ve = raised(fp8::block_exponent(va), lo, v_was, v_rise);
  const float ki = fp8::pow2(-ke), vi = fp8::pow2(-ve);
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    const int i = tid + kAThreads * j, slot = i / kVecs, d = i % kVecs * 8;
    if (slot < lo || slot >= hi) continue;
    float c[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      c[q] = kx[j].get(q) * ki;
    *reinterpret_cast<uint2 *>(kc + slot * D + d) =
        make_uint2(fp8::pack4(c[0], c[1], c[2], c[3]), fp8::pack4(c[4], c[5], c[6], c[7]));
  }
  if (has_v) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = vx[j].get(q) * vi;
      *reinterpret_cast<uint32_t *>(sv + (vd + q) * kTok + quad) = fp8::pack4(c[0], c[1], c[2], c[3]);
    }
  }
  if (k_rise > 0) lower_keys(kc, lo * D, k_rise, tid, kAThreads);
  __syncthreads();
  if (lo == 0 && hi == kTok) {
    for (int i = tid; i < D * kTok / 16; i += kAThreads)
      reinterpret_cast<uint4 *>(vc)[i] = reinterpret_cast<const uint4 *>(sv)[i];
  } else {
    const float f = fall(v_rise);
    const int from = v_rise > 0 ? 0 : lo, width = hi - from;
    for (int i = tid; i < D * width; i += kAThreads) {
      const int slot = from + i % width, at = i / width * kTok + slot;
      vc[at] = slot >= lo ? sv[at] : (uint8_t)fp8::pack2(fp8::unpack1(vc[at]) * f, 0.f);
    }
  }
  if (tid == 0) {
    g.k_exps[b.ph] = (uint8_t)(ke + fp8::kBias);
    g.v_exps[b.ph] = (uint8_t)(ve + fp8::kBias);
  }
}

// A few tokens (decoding): one warp per (touched block, head, sequence), a lane D / 32 channels.
template <typename T, int D>
__global__ void __launch_bounds__(128) append_few_kernel(Kv8AppendArgs g) {
  constexpr int C = D / 32;
  wait_for_grids();
  launch_dependents();
  const int lane = threadIdx.x % 32;
  const int64_t item = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
  if (item >= (int64_t)g.n_seq * g.n_kv * 2) return;
  const int head = (int)(item / 2 % g.n_kv), seq = (int)(item / 2 / g.n_kv);
  const Touched b = touched(g, seq, head, (int)(item % 2));
  if (b.ph < 0) return;
  const int lo = b.lo, n = b.hi - b.lo;
  uint8_t *kc = g.k + b.ph * (int64_t)(kTok * D), *vc = g.v + b.ph * (int64_t)(kTok * D);
  const uint8_t k_was = g.k_exps[b.ph], v_was = g.v_exps[b.ph];
  const T *ks = (const T *)g.new_k + seq * g.k_stride[0] + head * g.k_stride[2] +
                (b.tok + lo) * g.k_stride[1] + lane * C;
  const T *vs = (const T *)g.new_v + seq * g.v_stride[0] + head * g.v_stride[2] +
                (b.tok + lo) * g.v_stride[1] + lane * C;
  float kx[kFew][C], vx[kFew][C], ka = 0.f, va = 0.f;
#pragma unroll
  for (int j = 0; j < kFew; ++j)
#pragma unroll
    for (int q = 0; q < C; ++q) {
      kx[j][q] = j < n ? to_f32(ks[j * g.k_stride[1] + q]) : 0.0f;
      vx[j][q] = j < n ? to_f32(vs[j * g.v_stride[1] + q]) : 0.0f;
    }
  unsigned bad = 0;
#pragma unroll
  for (int j = 0; j < kFew; ++j)
#pragma unroll
    for (int q = 0; q < C; ++q) {
      ka = fmaxf(ka, fp8::finite_abs(kx[j][q]));
      va = fmaxf(va, fp8::finite_abs(vx[j][q]));
      bad |= fp8::finite(vx[j][q]) ? 0u : 1u << j;
    }
  bad = __reduce_or_sync(0xffffffffu, bad);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    ka = fmaxf(ka, __shfl_xor_sync(0xffffffffu, ka, o));
    va = fmaxf(va, __shfl_xor_sync(0xffffffffu, va, o));
  }
  int k_rise, v_rise;
  const int ke = raised(fp8::block_exponent(ka), lo, k_was, k_rise);
  const int ve = raised(fp8::block_exponent(va), lo, v_was, v_rise);
  const float ki = fp8::pow2(-ke), vi = fp8::pow2(-ve);
#pragma unroll
  for (int j = 0; j < kFew; ++j) {
    if (j >= n) break;
    float c[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < C; ++q) {
      c[q] = bad >> j & 1 ? __uint_as_float(0x7FC00000u) : fp8::inf_to_nan(kx[j][q]) * ki;
      v[q] = fp8::finite(vx[j][q]) ? vx[j][q] * vi : 0.0f;
    }
    const uint32_t kw = fp8::pack4(c[0], c[1], c[2], c[3]), vw = fp8::pack4(v[0], v[1], v[2], v[3]);
    uint8_t *kd = kc + (lo + j) * D + lane * C;
    if constexpr (C == 4) *reinterpret_cast<uint32_t *>(kd) = kw;
    else *reinterpret_cast<uint16_t *>(kd) = (uint16_t)kw;
#pragma unroll
    for (int q = 0; q < C; ++q) vc[(lane * C + q) * kTok + lo + j] = (uint8_t)(vw >> (8 * q));
  }
  if (k_rise > 0) lower_keys(kc, lo * D, k_rise, lane, 32);
  if (v_rise > 0) {
    const float f = fall(v_rise);
    for (int i = lane; i < D * lo; i += 32) {
      uint8_t *p = vc + i / lo * kTok + i % lo;
      *p = (uint8_t)fp8::pack2(fp8::unpack1(*p) * f, 0.f);
    }
  }
  if (lane == 0) {
    g.k_exps[b.ph] = (uint8_t)(ke + fp8::kBias);
    g.v_exps[b.ph] = (uint8_t)(ve + fp8::kBias);
  }
}

template <typename T, int D>
gptq_status launch_of(const Kv8AppendArgs &g, cudaStream_t s) {
  if (g.n_new <= kFew)
    return launch_early(append_few_kernel<T, D>,
                        dim3((unsigned)ceil_div((int64_t)g.n_seq * g.n_kv * 2, 4)), dim3(128), 0, 1,
                        s, g);
  const dim3 grid((unsigned)((g.n_new + 2 * (kTok - 1)) / kTok), (unsigned)g.n_kv,
                  (unsigned)g.n_seq);
  return launch_early(append_kernel<T, D>, grid, dim3(kAThreads), 0, 1, s, g);
}

template <typename T>
gptq_status launch_any(const Kv8AppendArgs &g, cudaStream_t s) {
  return g.dim == 64 ? launch_of<T, 64>(g, s) : launch_of<T, 128>(g, s);
}

}  // namespace

gptq_status launch_kv8_append(const Kv8AppendArgs &g, cudaStream_t s) {
  if (g.n_seq == 0 || g.n_new == 0) return GPTQ_OK;
  switch (g.dtype) {
    case GPTQ_F32: return launch_any<float>(g, s);
    case GPTQ_F16: return launch_any<__half>(g, s);
    default: return launch_any<__nv_bfloat16>(g, s);
  }
}

}  // namespace gptq
