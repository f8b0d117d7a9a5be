// causal_conv_bwd.cu -- gradients of the causal depthwise conv1d + SiLU (gdn_qkv_conv_bwd).
//
// With pre[t] = bias + sum_i w_i in(t - (K - 1) + i), y = pre sigma(pre) and in() as in
// causal_conv.cu (the sequence, before it the window conv_state):
//
//   dpre[t] = dy[t] sigma (1 + pre (1 - sigma))
//   din(p)  = sum_i w_i dpre[p + (K - 1) - i]      (tokens of the sequence only)
//   dw_i    = sum_t dpre[t] in(t - (K - 1) + i),   dbias = sum_t dpre[t]
//
// and the new conv_state holds the last K inputs, so its gradient, where there is
// one, is added to theirs.  dy is read from dq, dk and dv, as they are laid out.
// pre is formed again from x (in io_dtype, or in 8 bits, act8.cuh), so x is all
// that the forward pass has to keep.
//
// Bound by HBM: x and dy are read once, dx written once.  A thread owns 4 channels
// over a run of tokens, which may cross sequences.  Its rows come through a ring
// of cp.async copies that only it reads.  In registers it keeps the K - 1 inputs
// before the token, the K - 1 gradients that later tokens still add to (so a run
// also looks at the K - 1 tokens behind it), and its part of dw and dbias, which
// go to the workspace once per run and are added up by a second kernel in a fixed
// order.
#include "act8.cuh"
#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace convbwd {

constexpr int kThreads = 128;
constexpr int E = 4;                       // channels of a thread
constexpr int kMinRun = 32;                // tokens of a run at least
constexpr int kMaxBlocks = 148 * 6;

struct Shape {
  int tiles;    // channel blocks
  int run;      // tokens of a run
  int blocks;   // runs
};
static Shape shape_of(int64_t tokens, int channels) {
  Shape s;
  s.tiles = (channels + kThreads * E - 1) / (kThreads * E);
  const int64_t most = kMaxBlocks / s.tiles > 0 ? kMaxBlocks / s.tiles : 1;
  int64_t run = (tokens + most - 1) / most;
  if (run < kMinRun) run = kMinRun;
  s.run = (int)run;
  s.blocks = (int)((tokens + run - 1) / run);
  return s;
}

template <int B> __device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(dst), "l"(src), "n"(B) : "memory");
}

template <typename IO> __device__ __forceinline__ void unpack4(const void* p, float* x);
template <> __device__ __forceinline__ void unpack4<float>(const void* p, float* x) {
  const float4 v = *static_cast<const float4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
template <> __device__ __forceinline__ void unpack4<__nv_bfloat16>(const void* p, float* x) {
  const uint2 v = *static_cast<const uint2*>(p);
  x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
}
template <typename IO> __device__ __forceinline__ void store4(IO* p, const float* x);
template <> __device__ __forceinline__ void store4<float>(float* p, const float* x) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
}
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* p, const float* x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  __stcs(reinterpret_cast<uint2*>(p), make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b)));
}

// sigma(x) (1 + x (1 - sigma(x))); the exponent is clamped so that the divisor stays below the limit of __fdividef
__device__ __forceinline__ float silu_slope(float x) {
  const float s = __fdividef(1.f, 1.f + __expf(fminf(-x, 80.f)));
  return s * fmaf(x, 1.f - s, 1.f);
}

// Where the gradient of channel c0's output is: dq, dk or dv, and the elements between its rows.
template <typename IO>
__device__ __forceinline__ const IO* dy_of(const ConvBwdArgs& a, int c0, size_t& pitch) {
  const int qk = a.nqk * a.dk;
  pitch = c0 < 2 * qk ? (size_t)qk : (size_t)a.nv * a.dv;
  if (c0 < qk) return static_cast<const IO*>(a.dq) + c0;
  if (c0 < 2 * qk) return static_cast<const IO*>(a.dk_) + (c0 - qk);
  return static_cast<const IO*>(a.dv_) + (c0 - 2 * qk);
}

// Input x[t, c] of one channel.
template <typename IO, bool k8>
__device__ __forceinline__ float x_at(const ConvBwdArgs& a, int64_t t, int c) {
  const size_t at = (size_t)t * a.channels + c;
  if constexpr (k8) {
    float v[4];
    act8::decode4(static_cast<const uint8_t*>(a.x)[at], act8::factor(a.x_scales[at / act8::kGroup]), v);
    return v[0];
  } else {
    return to_f32(static_cast<const IO*>(a.x)[at]);
  }
}
template <typename IO>
__device__ __forceinline__ float window_at(const ConvBwdArgs& a, int n, int c, int j) {
  if (a.state_in == nullptr || j < 0 || j >= a.ksize) return 0.f;
  return to_f32(static_cast<const IO*>(a.state_in)[((size_t)n * a.channels + c) * a.ksize + j]);
}

__device__ __forceinline__ int seq_of(const int32_t* cu, int num_seqs, int64_t t) {
  int lo = 0, hi = num_seqs - 1;
  while (lo < hi) {  // the first n with cu[n + 1] > t
    const int mid = (lo + hi) >> 1;
    if ((int64_t)cu[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

template <typename IO, int K, bool k8>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(ConvBwdArgs a, Shape sh, float* part) {
  constexpr int kX = k8 ? E : E * (int)sizeof(IO), kY = E * (int)sizeof(IO);  // bytes of a row
  constexpr int kDepth = sizeof(IO) == 2 ? 16 : 8;
  constexpr int H = K - 1;                 // inputs before the token
  __shared__ __align__(16) uint8_t ring_y[kDepth][kThreads * kY];
  __shared__ __align__(16) uint8_t ring_x[kDepth][kThreads * kX];
  const int c0 = (blockIdx.x * kThreads + threadIdx.x) * E;
  if (c0 >= a.channels) return;
  const int64_t T = a.total_tokens, t0 = (int64_t)blockIdx.y * sh.run;
  const int64_t t1 = min(T, t0 + sh.run), te = min(T, t1 + H);  // dx of [t0, t1) needs dpre of [t0, te)
  size_t pitch;
  const IO* dy = dy_of<IO>(a, c0, pitch);
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + (size_t)c0 * (kX / E);
  const size_t xpitch = (size_t)a.channels * (kX / E);
  const uint8_t* xs = k8 ? a.x_scales + c0 / act8::kGroup : nullptr;
  const size_t spitch = (size_t)a.channels / act8::kGroup;
  const uint32_t by = (uint32_t)__cvta_generic_to_shared(&ring_y[0][threadIdx.x * kY]);
  const uint32_t bx = (uint32_t)__cvta_generic_to_shared(&ring_x[0][threadIdx.x * kX]);
  auto fetch = [&](int64_t t, int slot) {
    if (t < te) {
      cp_async<kY>(by + slot * (kThreads * kY), dy + (size_t)t * pitch);
      cp_async<kX>(bx + slot * (kThreads * kX), x + (size_t)t * xpitch);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
#pragma unroll
  for (int u = 0; u + 1 < kDepth; ++u) fetch(t0 + u, u);

  float w[K][E], b[E], dw[K][E], db[E], win[H > 0 ? H : 1][E], pend[H > 0 ? H : 1][E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    b[e] = a.bias ? a.bias[c0 + e] : 0.f;
    db[e] = 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      w[i][e] = a.weight[(size_t)(c0 + e) * K + i];
      dw[i][e] = 0.f;
    }
  }
  int n = a.cu ? seq_of(a.cu, a.num_seqs, t0) : (int)(t0 / a.uniform_len);
  int64_t s0, s1;
  seq_bounds(a, n, s0, s1);
  // win[j]: input at t - H + j; pend[j]: what is known of the gradient of the input at t - H + j
#pragma unroll
  for (int j = 0; j < H; ++j) {
    const int64_t p = t0 - H + j;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      win[j][e] = p >= s0 ? x_at<IO, k8>(a, p, c0 + e) : window_at<IO>(a, n, c0 + e, (int)(K + (p - s0)));
      pend[j][e] = 0.f;
    }
  }
  // dx of token t, which no later token adds to, if it is this run's and this sequence's
  auto emit = [&](int64_t t, float* g) {
    if (t < t0 || t >= t1 || t < s0 || t >= s1) return;
    if (a.dstate_out && t >= s1 - K) {
      const IO* d = static_cast<const IO*>(a.dstate_out) + ((size_t)n * a.channels + c0) * K + (t - (s1 - K));
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] += to_f32(d[e * K]);
    }
    store4<IO>(static_cast<IO*>(a.dx) + (size_t)t * a.channels + c0, g);
  };
  // the gradients still pending when the tokens of a sequence end before token t
  auto flush = [&](int64_t t) {
#pragma unroll
    for (int j = 0; j < H; ++j) emit(t - H + j, pend[j]);
  };
  uint32_t sc[4] = {0u, 0u, 0u, 0u};  // scale bytes of four rows, read four rows ahead
  auto scales = [&](int64_t t) {
    if constexpr (k8) {
#pragma unroll
      for (int u = 0; u < 4; ++u) sc[u] = t + u < te ? xs[(size_t)(t + u) * spitch] : 127u;
    }
  };
  scales(t0);
  const int rows = (int)(te - t0);
  bool open = true;  // the run's last sequence still adds to it
  for (int i0 = 0; i0 < rows && open; i0 += 4) {
    uint32_t cur[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) cur[u] = sc[u];
    scales(t0 + i0 + 4);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u;
      if (i >= rows) break;
      const int64_t t = t0 + i;
      fetch(t + kDepth - 1, (i + kDepth - 1) % kDepth);
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kDepth - 1) : "memory");
      if (t >= s1) {  // the next sequence that has tokens begins
        flush(t);
        if (t >= t1) {  // it is all behind the run
          open = false;
          break;
        }
        while (t >= s1 && n + 1 < a.num_seqs) {
          ++n;
          seq_bounds(a, n, s0, s1);
        }
#pragma unroll
        for (int j = 0; j < H; ++j)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            win[j][e] = window_at<IO>(a, n, c0 + e, j + 1);
            pend[j][e] = 0.f;
          }
      }
      const bool outside = t < s0 || t >= s1;  // only with inconsistent cu_seqlens, already reported
      float g[E], v[E], cur_g[E];
      unpack4<IO>(&ring_y[i % kDepth][threadIdx.x * kY], g);
      if constexpr (k8)
        act8::decode4(*reinterpret_cast<const uint32_t*>(&ring_x[i % kDepth][threadIdx.x * kX]), act8::factor(cur[u]), v);
      else
        unpack4<IO>(&ring_x[i % kDepth][threadIdx.x * kX], v);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float pre = b[e];
#pragma unroll
        for (int j = 0; j < H; ++j) pre = fmaf(w[j][e], win[j][e], pre);
        pre = fmaf(w[K - 1][e], v[e], pre);
        const float d = outside ? 0.f : g[e] * silu_slope(pre);
        if (t < t1) {
          db[e] += d;
#pragma unroll
          for (int j = 0; j < H; ++j) dw[j][e] = fmaf(d, win[j][e], dw[j][e]);
          dw[K - 1][e] = fmaf(d, v[e], dw[K - 1][e]);
        }
#pragma unroll
        for (int j = 0; j < H; ++j) pend[j][e] = fmaf(w[j][e], d, pend[j][e]);
        cur_g[e] = w[K - 1][e] * d;
      }
      if constexpr (H > 0) {
        emit(t - H, pend[0]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
#pragma unroll
          for (int j = 0; j + 1 < H; ++j) {
            win[j][e] = win[j + 1][e];
            pend[j][e] = pend[j + 1][e];
          }
          win[H - 1][e] = v[e];
          pend[H - 1][e] = cur_g[e];
        }
      } else {
        emit(t, cur_g);
      }
    }
  }
  if (open) flush(te);
  asm volatile("cp.async.wait_group 0;\n" ::: "memory");  // no copy outlives the block
  float* p = part + (size_t)blockIdx.y * (K + 1) * a.channels + c0;
#pragma unroll
  for (int i = 0; i < K; ++i)
    *reinterpret_cast<float4*>(p + (size_t)i * a.channels) = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
  *reinterpret_cast<float4*>(p + (size_t)K * a.channels) = make_float4(db[0], db[1], db[2], db[3]);
}

// dw[c, i] and dbias[c] from the runs' parts [run][K + 1][channels]: 32 columns by 8 shares of the runs
__global__ void __launch_bounds__(256) conv_weight_kernel(const float* __restrict__ part, int runs, int channels, int K, float* dw, float* db) {
  __shared__ float sum[8][32];
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, i = blockIdx.y;
  const size_t pitch = (size_t)(K + 1) * channels;
  float s = 0.f;
  if (c < channels)
    for (int r = share; r < runs; r += 8) s += part[(size_t)r * pitch + (size_t)i * channels + c];
  sum[share][lane] = s;
  __syncthreads();
  if (share != 0 || c >= channels) return;
#pragma unroll
  for (int j = 1; j < 8; ++j) s += sum[j][lane];
  if (i < K) dw[(size_t)c * K + i] = s; else if (db) db[c] = s;
}

// The gradient of the window before every sequence, one thread per sequence and channel.  Index j stands for
// position p = j - K: the taps i < j of the first tokens meet it, and the new conv_state still holds it where the
// sequence is shorter than K.
template <typename IO, int K, bool k8>
__global__ void __launch_bounds__(kThreads) conv_state_bwd_kernel(ConvBwdArgs a) {
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (idx >= (int64_t)a.num_seqs * a.channels) return;
  const int n = (int)(idx / a.channels), c = (int)(idx % a.channels);
  int64_t s0, s1;
  seq_bounds(a, n, s0, s1);
  const int64_t len = s1 - s0;
  float w[K], line[2 * K], g[K], dpre[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    w[i] = a.weight[(size_t)c * K + i];
    line[i] = window_at<IO>(a, n, c, i);                                 // positions -K ..
    line[K + i] = i < len ? x_at<IO, k8>(a, s0 + i, c) : 0.f;
    g[i] = 0.f;
  }
  size_t pitch;
  const IO* dy = dy_of<IO>(a, c, pitch);
  const float b = a.bias ? a.bias[c] : 0.f;
#pragma unroll
  for (int t = 0; t + 1 < K; ++t) {
    float pre = b;
#pragma unroll
    for (int i = 0; i < K; ++i) pre = fmaf(w[i], line[t + 1 + i], pre);
    dpre[t] = t < len ? to_f32(dy[(size_t)(s0 + t) * pitch]) * silu_slope(pre) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < K; ++j) {
#pragma unroll
    for (int i = 0; i < j; ++i) g[j] = fmaf(w[i], dpre[j - 1 - i], g[j]);
    if (a.dstate_out && j >= len) g[j] += to_f32(static_cast<const IO*>(a.dstate_out)[idx * K + (j - len)]);
    static_cast<IO*>(a.dstate_in)[idx * K + j] = from_f32<IO>(g[j]);
  }
}

template <typename IO, int K, bool k8>
static cudaError_t launch_k(const ConvBwdArgs& a, float* part, cudaStream_t s) {
  const Shape sh = shape_of(a.total_tokens, a.channels);
  cudaError_t e;
  if (sh.blocks > 0) {
    conv_bwd_kernel<IO, K, k8><<<dim3(sh.tiles, sh.blocks), kThreads, 0, s>>>(a, sh, part);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  conv_weight_kernel<<<dim3((a.channels + 31) / 32, K + 1), 256, 0, s>>>(part, sh.blocks, a.channels, K, a.dw, a.db);
  if ((e = cudaGetLastError()) != cudaSuccess || !a.dstate_in) return e;
  const int64_t threads = (int64_t)a.num_seqs * a.channels;
  conv_state_bwd_kernel<IO, K, k8><<<(unsigned int)((threads + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename IO, int K>
static cudaError_t launch_io(const ConvBwdArgs& a, float* part, cudaStream_t s) {
  return a.x_scales ? launch_k<IO, K, true>(a, part, s) : launch_k<IO, K, false>(a, part, s);
}
template <int K>
static cudaError_t launch_any(const ConvBwdArgs& a, int io_bf16, float* part, cudaStream_t s) {
  return io_bf16 ? launch_io<__nv_bfloat16, K>(a, part, s) : launch_io<float, K>(a, part, s);
}

}  // namespace convbwd

int64_t conv_bwd_workspace(int64_t tokens, int channels, int ksize) {
  return (int64_t)convbwd::shape_of(tokens, channels).blocks * (ksize + 1) * channels * (int64_t)sizeof(float);
}

cudaError_t launch_conv_bwd(const ConvBwdArgs& a, int io_bf16, float* part, cudaStream_t s) {
  switch (a.ksize) {
    case 1: return convbwd::launch_any<1>(a, io_bf16, part, s);
    case 2: return convbwd::launch_any<2>(a, io_bf16, part, s);
    case 3: return convbwd::launch_any<3>(a, io_bf16, part, s);
    case 4: return convbwd::launch_any<4>(a, io_bf16, part, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gdn
