// act8.cu -- activation checkpoints in 8 bits: gdn_act_quantize and gdn_act_dequantize.
//
// The format is in act8.cuh.  A thread takes 16 consecutive values, so a group is
// two neighbouring lanes, the codes move as 16-byte vectors, and a warp's 16 scale
// bytes are contiguous.  Bound by HBM: a value is read once and its code written
// once (3.03 bytes per bf16 value each way).  All of a thread's loads are issued
// before any is used.  To quantize took as much issue time as traffic while every
// value was looked at for infinities (363 us for 537 million bf16 values), so a
// group's largest magnitude is found on the bits, two bf16 at a time, where
// infinities and NaN are the largest: only a group that has one, or that reaches
// fp32's last binade, takes the path that looks at each value: 239 us, and 238 to
// read back, 1.63 GB each way, which is the rate of a plain copy.
#include "act8.cuh"
#include "train_common.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace act8 {

constexpr int kThreads = 256;
constexpr int kPer = 16;  // values of a thread

template <typename IO> struct Words;  // 16 values as 32-bit words
template <> struct Words<float> {
  static constexpr int N = 16;
  __device__ static void unpack(const uint32_t* w, float* x) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(w[i]);
  }
  __device__ static void pack(const float* x, uint32_t* w) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(x[i]);
  }
  // The bits of the largest magnitude
  __device__ static uint32_t top(const uint32_t* w) {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) t = max(t, w[i] & 0x7fffffffu);
    return t;
  }
  // Values 2 i and 2 i + 1 times f
  __device__ static float2 scaled(const uint32_t* w, int i, float f) {
    return make_float2(__uint_as_float(w[2 * i]) * f, __uint_as_float(w[2 * i + 1]) * f);
  }
};
template <> struct Words<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void unpack(const uint32_t* w, float* x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static void pack(const float* x, uint32_t* w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  __device__ static uint32_t top(const uint32_t* w) {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = __vmaxu2(t, w[i] & 0x7fff7fffu);
    return max(t & 0xffff0000u, t << 16);
  }
  // f is a power of two, and what falls below bf16's normal numbers is zero in e4m3: the product is exact in bf16
  __device__ static float2 scaled(const uint32_t* w, int i, float f) {
    const __nv_bfloat162 h = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(w + i), __float2bfloat162_rn(f));
    return __bfloat1622float2(h);
  }
};

// `n16` = values / 16 (even: whole groups).
template <typename IO>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const IO* __restrict__ x, uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales, int64_t n16) {
  constexpr int NW = Words<IO>::N;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n16) return;  // n16 is even and a group's lanes are an even one and the next: they leave together
  const unsigned int both = 3u << (threadIdx.x & 30);
  uint32_t w[NW];
#pragma unroll
  for (int j = 0; j < NW / 4; ++j) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(x + i * kPer) + j);
    w[4 * j] = u.x; w[4 * j + 1] = u.y; w[4 * j + 2] = u.z; w[4 * j + 3] = u.w;
  }
  uint32_t top = Words<IO>::top(w), s, c[4];
  top = max(top, __shfl_xor_sync(both, top, 1));
  if (top < 0x7f000000u) {  // below 2^127
    s = scale_byte(__uint_as_float(top));
    const float f = inv_factor(s);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(Words<IO>::scaled(w, 2 * j, f), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(Words<IO>::scaled(w, 2 * j + 1, f), __NV_SATFINITE, __NV_E4M3);
      c[j] = lo | (hi << 16);
    }
  } else {
    float v[kPer], most = 0.f;
    Words<IO>::unpack(w, v);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float m = fabsf(v[j]);
      if (m < INFINITY) most = fmaxf(most, m); else v[j] = NAN;  // what is not finite reads back as NaN
    }
    most = fmaxf(most, __shfl_xor_sync(both, most, 1));
    s = scale_byte(most);
    const float f = inv_factor(s);
    // 2^128 would be beyond fp32: the last binade is cut to what can be read back
    const float lim = s >= 247u ? 240.f : 448.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t p[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float2 y = make_float2(v[4 * j + 2 * k] * f, v[4 * j + 2 * k + 1] * f);
        y.x = y.x > lim ? lim : (y.x < -lim ? -lim : y.x);  // a NaN stays one
        y.y = y.y > lim ? lim : (y.y < -lim ? -lim : y.y);
        p[k] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
      }
      c[j] = p[0] | (p[1] << 16);
    }
  }
  __stcs(reinterpret_cast<uint4*>(codes) + i, make_uint4(c[0], c[1], c[2], c[3]));
  if ((threadIdx.x & 1) == 0) scales[i >> 1] = (uint8_t)s;
}

template <typename IO>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, IO* __restrict__ y,
                                                              int64_t n16) {
  constexpr int NW = Words<IO>::N;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n16) return;
  const uint4 c = __ldcs(reinterpret_cast<const uint4*>(codes) + i);
  const float f = factor(scales[i >> 1]);
  float v[kPer];
  decode4(c.x, f, v);
  decode4(c.y, f, v + 4);
  decode4(c.z, f, v + 8);
  decode4(c.w, f, v + 12);
  uint32_t w[NW];
  Words<IO>::pack(v, w);
#pragma unroll
  for (int j = 0; j < NW / 4; ++j)
    __stcs(reinterpret_cast<uint4*>(y + i * kPer) + j, make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
}

}  // namespace act8

cudaError_t launch_act_quantize(const void* x, uint8_t* codes, uint8_t* scales, int64_t n, int io_bf16, cudaStream_t s) {
  using namespace act8;
  const int64_t n16 = n / kPer;
  const unsigned int grid = (unsigned int)((n16 + kThreads - 1) / kThreads);
  if (io_bf16)
    quantize_kernel<<<grid, kThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(x), codes, scales, n16);
  else
    quantize_kernel<<<grid, kThreads, 0, s>>>(static_cast<const float*>(x), codes, scales, n16);
  return cudaGetLastError();
}

cudaError_t launch_act_dequantize(const uint8_t* codes, const uint8_t* scales, void* y, int64_t n, int io_bf16, cudaStream_t s) {
  using namespace act8;
  const int64_t n16 = n / kPer;
  const unsigned int grid = (unsigned int)((n16 + kThreads - 1) / kThreads);
  if (io_bf16)
    dequantize_kernel<<<grid, kThreads, 0, s>>>(codes, scales, static_cast<__nv_bfloat16*>(y), n16);
  else
    dequantize_kernel<<<grid, kThreads, 0, s>>>(codes, scales, static_cast<float*>(y), n16);
  return cudaGetLastError();
}

}  // namespace gdn
