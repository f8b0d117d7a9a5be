// f32x2.cuh -- pairs of fp32 values for the packed arithmetic of sm_100
// (fma.rn.f32x2 and the like: two results per issue, each rounded as the scalar
// instruction rounds it), and SiLU's sigmoid and slope on them.
#pragma once

#include <stdint.h>

namespace gdn {

struct F2 {
  uint64_t v;
  __device__ __forceinline__ float x() const { return __uint_as_float((uint32_t)v); }
  __device__ __forceinline__ float y() const { return __uint_as_float((uint32_t)(v >> 32)); }
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// 1 / (1 + exp(-x)) to a few ulp; exp may overflow, and then gives 0
__device__ __forceinline__ F2 sigmoid2(F2 x) {
  const F2 t = mul2(x, f2(-1.44269504f, -1.44269504f));
  float e0, e1;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(t.x()));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(t.y()));
  const F2 d = add2(f2(e0, e1), f2(1.f, 1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(d.x()));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(d.y()));
  return f2(e0, e1);
}
// d silu(x) / dx = s (1 + x (1 - s)), s = sigmoid(x)
__device__ __forceinline__ F2 silu_slope(F2 x) {
  const F2 s = sigmoid2(x), one = f2(1.f, 1.f);
  return mul2(s, fma2(x, fma2(s, f2(-1.f, -1.f), one), one));
}
__device__ __forceinline__ float silu_slope(float x) { return silu_slope(f2(x, x)).x(); }

}  // namespace gdn
