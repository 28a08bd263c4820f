// What the two attention kernels over the 8-bit cache share.
#pragma once

#include <type_traits>

#include "fp8.cuh"
#include "tc.cuh"

namespace gptq {
namespace kv8 {

constexpr int kTok = GPTQ_KV8_BLOCK;
constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
__device__ __forceinline__ T from_f32(float x) {
  if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Cached tokens of a sequence, inside the table.
__device__ __forceinline__ int seq_length(const Kv8AttentionArgs &g, int seq) {
  const int len = g.lengths[seq], cap = g.max_blocks * kTok;
  return len < 0 ? 0 : (len > cap ? cap : len);
}

// Starts a kernel's dependents early, and waits for the kernels it depends on to complete.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_grids() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A finite power of two next to amax (1 for 0), for rows that are scaled into fp16's range.
__device__ __forceinline__ int row_exponent(float amax) {
  const int e = (int)(__float_as_uint(amax) >> 23) - 127;
  return amax == 0.0f ? 0 : (e < -120 ? -120 : (e > 120 ? 120 : e));
}

}  // namespace kv8
}  // namespace gptq
