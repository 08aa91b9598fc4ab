// cache.cuh -- the 8-bit cache format on the device: e4m3 values and one power-of-two scale a
// row, held as a byte b that stands for 2^(b - 127).
//
// The scale of a row is the least power of two 2^e (e >= -126) with amax <= 448 * 2^e, 448
// being e4m3's largest value.  A power of two costs a floating format at most one binade of
// range over the exact ratio amax / 448 and nothing in relative precision, and it makes both
// directions exact but for the one rounding to e4m3: x * 2^-e has no rounding of its own, so
// no value next to a border depends on how a division was done, and value * 2^e is exact in
// bf16 on the way to the tensor cores.
#pragma once

#include <cuda_fp8.h>

#include "sm103.cuh"

namespace fa {

template <typename T>
__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi);
template <>
__device__ __forceinline__ void unpack2<__nv_bfloat16>(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}
template <>
__device__ __forceinline__ void unpack2<__half>(uint32_t w, float& lo, float& hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  lo = f.x;
  hi = f.y;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  return pack_f16x2(lo, hi);
}

// |x|, or 0 for an infinity or a NaN.
__device__ __forceinline__ float finite_abs(float x) {
  const float y = fabsf(x);
  return y < INFINITY ? y : 0.f;
}

// The least e in [-126, 120] with amax <= 448 * 2^e, from amax's bits: with amax = m 2^k and
// 448 = 1.75 * 2^8, e = k - 8 if m <= 1.75, else k - 7.  (A subnormal amax has k < -126.)
__device__ __forceinline__ int row_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int k = static_cast<int>(bits >> 23) - 127;
  const int e = k - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
}

// Four values times 2^-e, rounded to e4m3 (nearest even).
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * inv, d * inv), __NV_SATFINITE, __NV_E4M3);
  return (lo & 0xffffu) | (hi << 16);
}

// 2^(b - 127); b = 0 stands for 2^-127, a subnormal.
__device__ __forceinline__ float scale_of_byte(uint32_t b) {
  return __uint_as_float(b > 0 ? b << 23 : 0x00400000u);
}

__device__ __forceinline__ void dequant4(uint32_t q, float s, float& a, float& b, float& c, float& d) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(q & 0xffffu), __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(q >> 16), __NV_E4M3);
  const float2 f = __half22float2(__half2(lo)), g = __half22float2(__half2(hi));
  a = f.x * s;
  b = f.y * s;
  c = g.x * s;
  d = g.y * s;
}

}  // namespace fa
