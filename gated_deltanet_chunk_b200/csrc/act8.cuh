// act8.cuh -- activations kept in 8 bits: e4m3 codes, and a power of two for every 32 values.
//
// A group of 32 consecutive values is kept as 32 e4m3 codes and one byte e + 127,
// where 2^e is the least power of two (e >= -126) with max |x| <= 448 2^e over the
// group's finite values.  Both steps are exact but for the one rounding to e4m3
// (half a step: 2^-4 of a value of at least 2^(e-6), 2^(e-10) below), and a value
// read back, code * 2^e, has four significant bits, so bf16 holds it too.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "train_common.cuh"

namespace gdn {
namespace act8 {

constexpr int kGroup = 32;

// e + 127 of the group whose largest finite magnitude is `top`.
__device__ __forceinline__ uint32_t scale_byte(float top) {
  const uint32_t b = __float_as_uint(top);
  // top = m 2^x with m in [1, 2): 448 = 1.75 2^8, so e = x - 8, or x - 7 where m > 1.75
  const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 1);
}
__device__ __forceinline__ float factor(uint32_t byte) { return __uint_as_float(byte << 23); }             // 2^e
__device__ __forceinline__ float inv_factor(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }  // 2^-e

// Four codes, low byte first, as the values they stand for.
__device__ __forceinline__ void decode4(uint32_t w, float f, float* x) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
  const float2 p = __half22float2(__half2(a)), q = __half22float2(__half2(b));
  x[0] = p.x * f;
  x[1] = p.y * f;
  x[2] = q.x * f;
  x[3] = q.y * f;
}

}  // namespace act8
}  // namespace gdn
