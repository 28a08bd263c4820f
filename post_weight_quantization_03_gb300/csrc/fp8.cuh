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

#include <type_traits>

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

constexpr int kVec = 8;

template <typename T>
__device__ __forceinline__ T from_f32(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// Eight elements as they are stored.  `align`: what the rows' addresses are a multiple of (16, 8,
// 4, else single elements); only the first n elements exist, the others read as 0.
template <typename T>
struct Raw8 {
  static constexpr int kWords = 2 * sizeof(T);
  uint32_t q[kWords];
  __device__ __forceinline__ void load(const T *__restrict__ p, int64_t n, int align) {
    if (n >= kVec && align >= 4) {
      if (align >= 16) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
          const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
          q[4 * i] = v.x; q[4 * i + 1] = v.y; q[4 * i + 2] = v.z; q[4 * i + 3] = v.w;
        }
      } else if (align >= 8) {
#pragma unroll
        for (int i = 0; i < kWords / 2; ++i) {
          const uint2 v = reinterpret_cast<const uint2 *>(p)[i];
          q[2 * i] = v.x; q[2 * i + 1] = v.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kWords; ++i) q[i] = reinterpret_cast<const uint32_t *>(p)[i];
      }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) q[i] = i < n ? __float_as_uint(p[i]) : 0u;
    } else {
      const uint16_t *e = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        q[i] = (2 * i < n ? (uint32_t)e[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)e[2 * i + 1] << 16 : 0u);
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(q[i]);
    } else if constexpr (std::is_same<T, __half>::value) {
      return __half2float(__ushort_as_half((unsigned short)(q[i / 2] >> (16 * (i % 2)))));
    } else {
      return __uint_as_float(i % 2 ? q[i / 2] & 0xFFFF0000u : q[i / 2] << 16);
    }
  }
  // The larger of `m` and the elements' magnitudes, as integers (of the even and the odd elements
  // where two share a word): infinities and NaN are above all numbers.
  __device__ __forceinline__ uint32_t most(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4) m = max(m, q[i] & 0x7FFFFFFFu);
      else m = __vmaxu2(m, q[i] & 0x7FFF7FFFu);
    }
    return m;
  }
  // That as the bits of an fp32 number.
  __device__ __forceinline__ static uint32_t most_bits(uint32_t m) {
    if constexpr (sizeof(T) == 4) return m;
    m = max(m & 0xFFFFu, m >> 16);
    if constexpr (std::is_same<T, __half>::value)
      return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
    return m << 16;
  }
  __device__ __forceinline__ void set(const float (&v)[kVec]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) q[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const T lo = from_f32<T>(v[2 * i]), hi = from_f32<T>(v[2 * i + 1]);
        q[i] = (uint32_t) * reinterpret_cast<const uint16_t *>(&lo) |
               (uint32_t) * reinterpret_cast<const uint16_t *>(&hi) << 16;
      }
    }
  }
  __device__ __forceinline__ void store(T *__restrict__ p, int64_t n, int align) const {
    if (n >= kVec && align >= 4) {
      if (align >= 16) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i)
          reinterpret_cast<uint4 *>(p)[i] = make_uint4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
      } else if (align >= 8) {
#pragma unroll
        for (int i = 0; i < kWords / 2; ++i)
          reinterpret_cast<uint2 *>(p)[i] = make_uint2(q[2 * i], q[2 * i + 1]);
      } else {
#pragma unroll
        for (int i = 0; i < kWords; ++i) reinterpret_cast<uint32_t *>(p)[i] = q[i];
      }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (i < n) p[i] = __uint_as_float(q[i]);
    } else {
      uint16_t *e = reinterpret_cast<uint16_t *>(p);
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (i < n) e[i] = (uint16_t)(q[i / 2] >> (16 * (i % 2)));
    }
  }
};

// What an address and all steps of `bytes` from it are a multiple of: 16, 8, 4 or less.
static inline int alignment(const void *p, int64_t bytes, int64_t bytes2 = 0, int64_t bytes3 = 0) {
  const uintptr_t bits = (uintptr_t)p | (uintptr_t)bytes | (uintptr_t)bytes2 | (uintptr_t)bytes3;
  return bits % 16 == 0 ? 16 : (bits % 8 == 0 ? 8 : (bits % 4 == 0 ? 4 : 1));
}

}  // namespace fp8
}  // namespace gptq
