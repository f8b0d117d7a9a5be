// gated_rmsnorm_bwd.cu -- gradients of the gated RMSNorm epilogue (gdn_gated_rmsnorm_bwd).
//
// Of y = n w s with n = o r, r = 1 / sqrt(mean(o^2) + eps), s = z sigma(z), per row:
//   do = r (dn - n mean(dn n)),  dn = dy w s
//   dz = dy n w sigma(z) (1 + z (1 - sigma(z)))
//   dw = sum over rows of dy n s
// r and s are formed again, so o and z are all that the forward pass has to keep,
// in io_dtype or in 8 bits (act8.cuh).  Bound by HBM: dy, o, z are read once, do and
// dz written once.  The layout is that of gated_rmsnorm.cu: a row spans the lanes of
// a group, and a thread's columns are the same in every row, so its part of dw
// stays in registers until the block's groups are joined in shared memory; a
// second kernel joins the blocks, in a fixed order.  Measured: 16,384 tokens x 8 heads of
// 128 in fp32, 0.34 GB, 55 us and 4 for the second kernel (87 % of the copy
// bandwidth); 65,536 x 32 in bf16 from 8 bits, 2.16 GB, 366 and 4 us (89 %).
#include "act8.cuh"
#include "f32x2.cuh"
#include "train_common.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace rmsbwd {

constexpr int kThreads = 256;
// 65,536 tokens x 32 heads of 128, o and z in 8 bits: 366 us; with 1 row in flight 413, with 2 or 4 blocks 412 and 496
constexpr int kUnroll = 2;                // rows of a lane group in flight
constexpr int kPerSm = 3;                 // blocks per SM
constexpr int kMaxBlocks = 148 * kPerSm;  // one wave

template <typename IO> struct Vec;  // 16 bytes of IO
template <> struct Vec<float> {
  static constexpr int N = 4;
  __device__ static void unpack(uint4 v, float* x) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
  __device__ static void store(void* p, const float* x) { __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3])); }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void unpack(uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static void store(void* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
};

// The E values at element `at` of a kept activation: io_dtype, or codes and the scale byte of their group.
template <typename IO, bool k8>
struct Kept {
  static constexpr int E = Vec<IO>::N;
  uint4 w;
  uint32_t s;
  __device__ void load(const void* x, const uint8_t* scales, size_t at) {
    if constexpr (!k8) {
      w = __ldcs(reinterpret_cast<const uint4*>(static_cast<const IO*>(x) + at));
    } else {
      const uint8_t* c = static_cast<const uint8_t*>(x) + at;
      if constexpr (E == 8) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(c));
        w.x = v.x;
        w.y = v.y;
      } else {
        w.x = __ldcs(reinterpret_cast<const unsigned int*>(c));
      }
      s = scales[at / act8::kGroup];
    }
  }
  __device__ void unpack(float* x) const {
    if constexpr (!k8) {
      Vec<IO>::unpack(w, x);
    } else {
      const float f = act8::factor(s);
      act8::decode4(w.x, f, x);
      if constexpr (E == 8) act8::decode4(w.y, f, x + 4);
    }
  }
};

template <typename IO, int DIM, bool kO8, bool kZ8>
__global__ void __launch_bounds__(kThreads, kPerSm) gated_rmsnorm_bwd_kernel(NormBwdArgs p, float* part) {
  let_next_begin();
  constexpr int E = Vec<IO>::N, L = DIM / E, G = kThreads / L;
  __shared__ float sum[G][DIM];
  const int lr = threadIdx.x % L, grp = threadIdx.x / L;
  constexpr int P = E / 2;
  F2 wv[P], dw[P];
#pragma unroll
  for (int e = 0; e < P; ++e) {
    wv[e] = f2(p.w[lr * E + 2 * e], p.w[lr * E + 2 * e + 1]);
    dw[e] = f2(0.f, 0.f);
  }
  const int64_t step = (int64_t)G * gridDim.x;
  uint4 dyw[kUnroll];
  Kept<IO, kO8> ow[kUnroll];
  Kept<IO, kZ8> zw[kUnroll];
  auto load = [&](int64_t b0, int u) {
    const int64_t r = b0 + u * step + grp;
    if (r < p.rows) {
      const size_t at = (size_t)r * DIM + lr * E;
      dyw[u] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const IO*>(p.dy) + at));
      ow[u].load(p.o, p.o_scales, at);
      zw[u].load(p.z, p.z_scales, at);
    }
  };
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) load((int64_t)blockIdx.x * G, u);
  // every lane of a warp takes the same number of passes (the shuffles need them all)
  for (int64_t b0 = (int64_t)blockIdx.x * G; b0 < p.rows; b0 += step * kUnroll) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t r = b0 + u * step + grp;
      const bool valid = r < p.rows;
      F2 dy[P], o[P], z[P];
      float x[E];
      Vec<IO>::unpack(dyw[u], x);
#pragma unroll
      for (int e = 0; e < P; ++e) dy[e] = f2(x[2 * e], x[2 * e + 1]);
      ow[u].unpack(x);
#pragma unroll
      for (int e = 0; e < P; ++e) o[e] = f2(x[2 * e], x[2 * e + 1]);
      zw[u].unpack(x);
#pragma unroll
      for (int e = 0; e < P; ++e) z[e] = f2(x[2 * e], x[2 * e + 1]);
      load(b0 + step * kUnroll, u);  // comes in while this row and the next are worked on
      F2 acc = f2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < P; ++e) acc = fma2(o[e], o[e], acc);
      float ss = acc.x() + acc.y();
#pragma unroll
      for (int m = L / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      const float inv = rsqrtf(ss * (1.f / DIM) + p.eps);
      const F2 inv2 = f2(inv, inv), one = f2(1.f, 1.f), neg = f2(-1.f, -1.f);
      F2 dn[P];
      acc = f2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const F2 n = mul2(o[e], inv2), sig = sigmoid2(z[e]), s = mul2(z[e], sig), g = mul2(dy[e], wv[e]);
        dn[e] = mul2(g, s);
        if (valid) dw[e] = fma2(mul2(dy[e], n), s, dw[e]);
        z[e] = mul2(mul2(g, n), fma2(s, fma2(sig, neg, one), sig));  // sig (1 + z (1 - sig))
        o[e] = n;
        acc = fma2(dn[e], n, acc);
      }
      float c = acc.x() + acc.y();
#pragma unroll
      for (int m = L / 2; m > 0; m >>= 1) c += __shfl_xor_sync(0xffffffffu, c, m);
      c *= -1.f / DIM;
      if (valid) {
        const size_t at = (size_t)r * DIM + lr * E;
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const F2 d = mul2(inv2, fma2(o[e], f2(c, c), dn[e]));
          x[2 * e] = d.x();
          x[2 * e + 1] = d.y();
        }
        Vec<IO>::store(static_cast<IO*>(p.d_o) + at, x);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          x[2 * e] = z[e].x();
          x[2 * e + 1] = z[e].y();
        }
        Vec<IO>::store(static_cast<IO*>(p.d_z) + at, x);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < P; ++e) {
    sum[grp][lr * E + 2 * e] = dw[e].x();
    sum[grp][lr * E + 2 * e + 1] = dw[e].y();
  }
  __syncthreads();
  if (threadIdx.x < DIM) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < G; ++i) s += sum[i][threadIdx.x];
    part[(size_t)blockIdx.x * DIM + threadIdx.x] = s;
  }
}

// out[c] = sum over blocks of part[block][c]; one warp a column
__global__ void __launch_bounds__(kThreads) weight_sums_kernel(const float* part, int blocks, int dim, float* out) {
  wait_for_previous();
  const int c = blockIdx.x * (kThreads / 32) + threadIdx.x / 32, lane = threadIdx.x & 31;
  float s = 0.f;
  for (int b = lane; b < blocks; b += 32) s += part[(size_t)b * dim + c];
  s = warp_sum(s);
  if (lane == 0) out[c] = s;
}

static int blocks_of(int64_t rows, int dim, int io_bf16) {
  const int64_t per = (int64_t)(kThreads / (dim / (io_bf16 ? 8 : 4))) * kUnroll;
  const int64_t need = (rows + per - 1) / per;
  return (int)(need < kMaxBlocks ? need : kMaxBlocks);
}

template <typename IO, int DIM>
static cudaError_t launch(const NormBwdArgs& p, float* part, cudaStream_t s) {
  const int blocks = blocks_of(p.rows, DIM, sizeof(IO) == 2);
  if (blocks > 0) {
    if (p.o_scales && p.z_scales)
      gated_rmsnorm_bwd_kernel<IO, DIM, true, true><<<blocks, kThreads, 0, s>>>(p, part);
    else if (p.o_scales)
      gated_rmsnorm_bwd_kernel<IO, DIM, true, false><<<blocks, kThreads, 0, s>>>(p, part);
    else if (p.z_scales)
      gated_rmsnorm_bwd_kernel<IO, DIM, false, true><<<blocks, kThreads, 0, s>>>(p, part);
    else
      gated_rmsnorm_bwd_kernel<IO, DIM, false, false><<<blocks, kThreads, 0, s>>>(p, part);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return launch_next(weight_sums_kernel, DIM / (kThreads / 32), kThreads, 0, s, part, blocks, DIM, p.dw);
}

}  // namespace rmsbwd

int64_t gated_rmsnorm_bwd_workspace(int64_t rows, int dim, int io_bf16) {
  return (int64_t)rmsbwd::blocks_of(rows, dim, io_bf16) * dim * (int64_t)sizeof(float);
}

cudaError_t launch_gated_rmsnorm_bwd(const NormBwdArgs& p, int dim, int io_bf16, float* part, cudaStream_t s) {
  using bf = __nv_bfloat16;
  if (dim == 64) return io_bf16 ? rmsbwd::launch<bf, 64>(p, part, s) : rmsbwd::launch<float, 64>(p, part, s);
  if (dim == 128) return io_bf16 ? rmsbwd::launch<bf, 128>(p, part, s) : rmsbwd::launch<float, 128>(p, part, s);
  return cudaErrorInvalidValue;
}

}  // namespace gdn
