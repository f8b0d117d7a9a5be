// gate_bwd.cu -- gradients of the layer's gate (gdn_gate_bwd).
//
// With u = a + dt_bias, g = -exp(A_log) softplus(u), beta = sigmoid(b):
//   da = -exp(A_log) sigmoid(u) dg,        db = beta (1 - beta) dbeta
//   dA_log[h] = sum_t dg g,                ddt_bias[h] = sum_t da
// One pass over the tokens.  A thread keeps to the same v-heads (four where Nv is a
// multiple of four: 16-byte loads, else one), so the two sums stay in its
// registers; a block's threads are joined in shared memory and the blocks by a
// second kernel, in a fixed order.  da is summed in fp32, before its rounding.
// 65,536 tokens x 32 heads, 34 MB, take 11.3 us and 2.3 for the second kernel (5.1 at
// the copy bandwidth): two waves of loads and the launches are what is left.  Fewer
// tokens are one block's, and one launch.
#include "train_common.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace gatebwd {

constexpr int kThreads = 256;
constexpr int kBlocks = 4 * 148;  // row blocks at most (8 * 148: the same)
constexpr int kUnroll = 4;        // rows in flight per thread (2: 15.8 us against 14.8 from a cold L2)
// Passes over its rows up to which one block takes all tokens.  A pass is about 2.5 us, and blocks of one pass with
// the second kernel are 8 us and another launch by the host: 1024 tokens x 8 heads, two passes, take 8.5 against 8.1 us
// on the GPU, 2500 tokens 15.4 against 7.9.
constexpr int kOneBlock = 2;

struct Shape {
  int vec;                // v-heads of a thread
  int cols, rows, tiles;  // a block's threads across and rows at a time; column tiles
  int blocks;             // row blocks
};
static Shape shape_of(int64_t tokens, int nv) {
  Shape s;
  s.vec = nv % 4 == 0 ? 4 : 1;
  const int across = nv / s.vec;
  s.cols = across < kThreads ? across : kThreads;
  s.rows = kThreads / s.cols;
  s.tiles = (across + s.cols - 1) / s.cols;
  const int64_t need = (tokens + (int64_t)s.rows * kUnroll - 1) / ((int64_t)s.rows * kUnroll);
  const int64_t most = kBlocks / s.tiles > 0 ? kBlocks / s.tiles : 1;
  s.blocks = need <= kOneBlock ? (need > 0) : (int)(need < most ? need : most);
  return s;
}

template <typename IO, int V> __device__ __forceinline__ void load(const IO* p, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = to_f32(*p);
  } else if constexpr (sizeof(IO) == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
}
template <typename IO, int V> __device__ __forceinline__ void store(IO* p, const float (&x)[V]) {
  if constexpr (V == 1) {
    *p = from_f32<IO>(x[0]);
  } else if constexpr (sizeof(IO) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

template <typename IO, int V>
__global__ void __launch_bounds__(kThreads) gate_bwd_kernel(GateBwdArgs p, Shape s, float* part) {
  let_next_begin();
  __shared__ float sum[2][V][kThreads];
  const int tid = threadIdx.x, cl = tid % s.cols, rl = tid / s.cols;
  const int h = (blockIdx.x * s.cols + cl) * V;
  const bool mine = rl < s.rows && h < p.nv;
  float sA[V] = {}, sdt[V] = {};
  if (mine) {
    float rate[V], dt[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      rate[e] = expf(p.A_log[h + e]);
      dt[e] = p.dt_bias[h + e];
    }
    const int64_t step = (int64_t)s.rows * s.blocks;
    for (int64_t t0 = (int64_t)blockIdx.y * s.rows + rl; t0 < p.tokens; t0 += step * kUnroll) {
      float a[kUnroll][V], b[kUnroll][V], dg[kUnroll][V], db[kUnroll][V];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int64_t t = t0 + i * step;
        const size_t at = (size_t)(t < p.tokens ? t : t0) * p.nv + h;
        load<float, V>(p.a + at, a[i]);
        load<float, V>(p.b + at, b[i]);
        load<IO, V>(static_cast<const IO*>(p.dg) + at, dg[i]);
        load<IO, V>(static_cast<const IO*>(p.dbeta) + at, db[i]);
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int64_t t = t0 + i * step;
        if (t >= p.tokens) break;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float u = a[i][e] + dt[e], x = expf(-fabsf(u)), sig = __fdividef(u >= 0.f ? 1.f : x, 1.f + x);
          a[i][e] = -dg[i][e] * rate[e] * sig;
          sA[e] = fmaf(dg[i][e], -rate[e] * (fmaxf(u, 0.f) + log1pf(x)), sA[e]);
          sdt[e] += a[i][e];
          // sigmoid(b) (1 - sigmoid(b)) without cancellation
          const float y = expf(-fabsf(b[i][e])), q = 1.f + y;
          b[i][e] = db[i][e] * __fdividef(y, q * q);
        }
        const size_t at = (size_t)t * p.nv + h;
        store<IO, V>(static_cast<IO*>(p.da) + at, a[i]);
        store<IO, V>(static_cast<IO*>(p.db) + at, b[i]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    sum[0][e][tid] = sA[e];
    sum[1][e][tid] = sdt[e];
  }
  // halving over the rows, in a fixed order
  for (int n = s.rows; n > 1;) {
    const int half = (n + 1) / 2;
    __syncthreads();
    if (rl < n - half) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        sum[0][e][tid] += sum[0][e][tid + half * s.cols];
        sum[1][e][tid] += sum[1][e][tid + half * s.cols];
      }
    }
    n = half;
  }
  if (rl == 0 && h < p.nv) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (s.blocks == 1) {
        p.dA_log[h + e] = sum[0][e][tid];
        p.ddt_bias[h + e] = sum[1][e][tid];
      } else {
        part[((size_t)blockIdx.y * 2) * p.nv + h + e] = sum[0][e][tid];
        part[((size_t)blockIdx.y * 2 + 1) * p.nv + h + e] = sum[1][e][tid];
      }
    }
  }
}

// One block per column of part [blocks][cols]: out[c] = its sum.
__global__ void __launch_bounds__(128) column_sums_kernel(const float* part, int blocks, int nv, float* dA, float* ddt) {
  wait_for_previous();
  __shared__ float sum[4];
  const int c = blockIdx.x;
  float s = 0.f;
  for (int b = threadIdx.x; b < blocks; b += 128) s += part[(size_t)b * 2 * nv + c];
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) sum[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x == 0) (c < nv ? dA : ddt)[c < nv ? c : c - nv] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

template <typename IO>
static cudaError_t launch(const GateBwdArgs& p, float* part, cudaStream_t stream) {
  const Shape s = shape_of(p.tokens, p.nv);
  if (s.blocks > 0) {
    if (s.vec == 4)
      gate_bwd_kernel<IO, 4><<<dim3(s.tiles, s.blocks), kThreads, 0, stream>>>(p, s, part);
    else
      gate_bwd_kernel<IO, 1><<<dim3(s.tiles, s.blocks), kThreads, 0, stream>>>(p, s, part);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || s.blocks == 1) return e;
  }
  return launch_next(column_sums_kernel, 2 * p.nv, 128, 0, stream, part, s.blocks, p.nv, p.dA_log, p.ddt_bias);
}

}  // namespace gatebwd

int64_t gate_bwd_workspace(int64_t tokens, int nv) {
  const gatebwd::Shape s = gatebwd::shape_of(tokens, nv);
  return s.blocks > 1 ? (int64_t)s.blocks * 2 * nv * (int64_t)sizeof(float) : 0;
}

cudaError_t launch_gate_bwd(const GateBwdArgs& p, int io_bf16, float* part, cudaStream_t s) {
  return io_bf16 ? gatebwd::launch<__nv_bfloat16>(p, part, s) : gatebwd::launch<float>(p, part, s);
}

}  // namespace gdn
