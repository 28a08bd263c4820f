// The number format of the 8-bit serving operators: e4m3 codes with one exponent byte E per
// block, value = code * 2^(E - 127).
//
// A block whose largest finite magnitude is a has e = ceil(log2(a / 448)) limited to
// [kExpMin, kExpMax] (kExpMin for a block of zeros), E = e + 127.  The scale is a power of two
// because e4m3 is a floating format: any other scale moves the codes along the same 4-bit
// significands and gains nothing, while a power of two multiplies exactly and is what the
// tensor cores' block-scaled products take.  An element that is not finite becomes the NaN code.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace gptq {
namespace fp8 {

constexpr int kExpMin = -96, kExpMax = 120;
constexpr int kBias = 127;
constexpr int kBlock = 128;   // elements along K that share an exponent
constexpr uint8_t kNan = 0x7F;

// e for a block's largest magnitude (finite, >= 0).  448 = 1.75 * 2^8, so with
// amax = 1.f * 2^x the quotient's ceiling is x - 8 where 1.f <= 1.75 and x - 7 above.
__device__ __forceinline__ int block_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < kExpMin ? kExpMin : (e > kExpMax ? kExpMax : e);  // zero, subnormal: kExpMin
}

// 2^e as fp32, e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The value an exponent byte stands for; 0 and 255 do not occur in this format (they read as
// 0 and infinity).
__device__ __forceinline__ float exp_value(uint8_t E) { return __uint_as_float((uint32_t)E << 23); }

__device__ __forceinline__ bool finite(float x) {
  return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
}
__device__ __forceinline__ float finite_abs(float x) { return finite(x) ? fabsf(x) : 0.0f; }
// Infinity would saturate to 448: makes it NaN, which converts to the NaN code.
__device__ __forceinline__ float inf_to_nan(float x) {
  return finite(x) ? x : __uint_as_float(0x7FC00000u);
}

// Two codes, a in the low byte (round to nearest even).
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  return pack2(a, b) | (pack2(c, d) << 16);
}
__device__ __forceinline__ float2 unpack2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu),
                                                   __NV_E4M3);
  return __half22float2(__half2(h));
}
__device__ __forceinline__ float unpack1(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(__half(h));
}

}  // namespace fp8
}  // namespace gptq
