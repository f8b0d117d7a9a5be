// gate_bwd.cu -- gradients of the layer's gate (gdn_gate_bwd).
//
// With u = a + dt_bias, g = -exp(A_log) softplus(u), beta = sigmoid(b):
//   da = -exp(A_log) sigmoid(u) dg,        db = beta (1 - beta) dbeta
//   dA_log[h] = sum_t dg g,                ddt_bias[h] = sum_t da
// One pass over the tokens.  A thread keeps to one v-head, so the two sums stay in
// its registers; a block's threads are joined in shared memory and the blocks by a
// second kernel, in a fixed order.  da is summed in fp32, before its rounding.
#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace gatebwd {

constexpr int kThreads = 256;
constexpr int kBlocks = 4 * 148;  // row blocks at most: two to four waves of small blocks
constexpr int kUnroll = 4;        // rows in flight per thread

struct Shape {
  int cols, rows, tiles;  // a block's v-heads and rows at a time; column tiles
  int blocks;             // row blocks
};
static Shape shape_of(int64_t tokens, int nv) {
  Shape s;
  s.cols = nv < kThreads ? nv : kThreads;
  s.rows = kThreads / s.cols;
  s.tiles = (nv + s.cols - 1) / s.cols;
  const int64_t need = (tokens + (int64_t)s.rows * kUnroll - 1) / ((int64_t)s.rows * kUnroll);
  const int64_t most = kBlocks / s.tiles > 0 ? kBlocks / s.tiles : 1;
  s.blocks = (int)(need < most ? need : most);
  return s;
}

template <typename IO>
__global__ void __launch_bounds__(kThreads) gate_bwd_kernel(GateBwdArgs p, Shape s, float* part) {
  __shared__ float sum[2][kThreads];
  const int tid = threadIdx.x, cl = tid % s.cols, rl = tid / s.cols;
  const int h = blockIdx.x * s.cols + cl;
  float sA = 0.f, sdt = 0.f;
  if (rl < s.rows && h < p.nv) {
    const float rate = expf(p.A_log[h]), dt = p.dt_bias[h];
    const int64_t step = (int64_t)s.rows * s.blocks;
    for (int64_t t0 = (int64_t)blockIdx.y * s.rows + rl; t0 < p.tokens; t0 += step * kUnroll) {
      float a[kUnroll], b[kUnroll], dg[kUnroll], db[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int64_t t = t0 + i * step;
        const size_t at = (size_t)(t < p.tokens ? t : t0) * p.nv + h;
        a[i] = p.a[at];
        b[i] = p.b[at];
        dg[i] = to_f32(static_cast<const IO*>(p.dg)[at]);
        db[i] = to_f32(static_cast<const IO*>(p.dbeta)[at]);
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int64_t t = t0 + i * step;
        if (t >= p.tokens) break;
        const size_t at = (size_t)t * p.nv + h;
        const float u = a[i] + dt, x = expf(-fabsf(u)), sig = (u >= 0.f ? 1.f : x) / (1.f + x);
        const float da = -dg[i] * rate * sig;
        sA = fmaf(dg[i], -rate * (fmaxf(u, 0.f) + log1pf(x)), sA);
        sdt += da;
        // sigmoid(b) (1 - sigmoid(b)) without cancellation
        const float y = expf(-fabsf(b[i])), q = 1.f + y;
        static_cast<IO*>(p.da)[at] = from_f32<IO>(da);
        static_cast<IO*>(p.db)[at] = from_f32<IO>(db[i] * (y / (q * q)));
      }
    }
  }
  sum[0][tid] = sA;
  sum[1][tid] = sdt;
  __syncthreads();
  if (rl == 0 && h < p.nv) {
    for (int r = 1; r < s.rows; ++r) {
      sA += sum[0][r * s.cols + cl];
      sdt += sum[1][r * s.cols + cl];
    }
    if (s.blocks == 1) {
      p.dA_log[h] = sA;
      p.ddt_bias[h] = sdt;
    } else {
      part[((size_t)blockIdx.y * 2) * p.nv + h] = sA;
      part[((size_t)blockIdx.y * 2 + 1) * p.nv + h] = sdt;
    }
  }
}

// One warp per column of part [blocks][cols]: out[c] = its sum.
__global__ void __launch_bounds__(kThreads) column_sums_kernel(const float* __restrict__ part, int blocks, int nv, float* dA, float* ddt) {
  const int c = blockIdx.x * (kThreads / 32) + threadIdx.x / 32, lane = threadIdx.x & 31;
  if (c >= 2 * nv) return;
  float s = 0.f;
  for (int b = lane; b < blocks; b += 32) s += part[(size_t)b * 2 * nv + c];
  s = warp_sum(s);
  if (lane == 0) (c < nv ? dA : ddt)[c < nv ? c : c - nv] = s;
}

template <typename IO>
static cudaError_t launch(const GateBwdArgs& p, float* part, cudaStream_t stream) {
  const Shape s = shape_of(p.tokens, p.nv);
  if (s.blocks > 0) {
    gate_bwd_kernel<IO><<<dim3(s.tiles, s.blocks), kThreads, 0, stream>>>(p, s, part);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || s.blocks == 1) return e;
  }
  column_sums_kernel<<<(2 * p.nv + kThreads / 32 - 1) / (kThreads / 32), kThreads, 0, stream>>>(part, s.blocks, p.nv, p.dA_log, p.ddt_bias);
  return cudaGetLastError();
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
