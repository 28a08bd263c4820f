// What the block-scaled e4m3 products (tcgen05 kind::mxf8f6f4) share.
#pragma once

#include <type_traits>

#include "fp8.cuh"
#include "tc.cuh"

namespace gptq {
namespace mx {

constexpr int BM = 128;                     // weight rows of a tile
constexpr int BK = fp8::kBlock;             // 128 codes = 128 bytes = one swizzle row

template <typename TO>
__device__ __forceinline__ TO out_f32(float x) {
  if constexpr (std::is_same<TO, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// kind::mxf8f6f4 instruction descriptor: e4m3 operands, K-major, power-of-two scale bytes, 128 rows
// and tn columns.
__device__ __forceinline__ uint32_t instr_desc(int tn) {
  return (1u << 23) | ((uint32_t)(tn >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}

// D[tmem] (+)= (A * 2^sa)(B * 2^sb)^T, one thread; sa, sb: TMEM addresses of the scale columns;
// the operands' descriptors by their lower words (the upper one is the layout's).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8 rows on; version; swizzle
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                    uint32_t sa, uint32_t sb, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %7, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X "
      "[%0], a, b, %4, [%5], [%6], p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)accumulate)
      : "memory");
}

// 512 bytes of shared memory (32 rows of 16 bytes) to 32 lanes x 4 columns, repeated in each of
// the four lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  // no swizzle: 8 rows x 16 bytes contiguous, the next 8 rows 128 bytes on
  const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)8 << 16) |
                        ((uint64_t)8 << 32) | ((uint64_t)1 << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t caddr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(caddr)
               : "memory");
  return v;
}

}  // namespace mx
}  // namespace gptq
