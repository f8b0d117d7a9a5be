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
// Bound by HBM: x and dy are read once, dx written once.  A thread owns 16 bytes
// of channels (8 bf16 or 4 fp32) over a run of tokens, which may cross sequences.
// Its rows come through a ring of cp.async copies that only it reads.  In
// registers it keeps the K - 1 inputs before the token, the K - 1 gradients that
// later tokens still add to (so a run also looks at the K - 1 tokens behind it),
// and its part of dw and dbias, which go to the workspace once per run and are
// added up by a second kernel in a fixed order.  The arithmetic is about 13
// multiply-adds and two MUFU operations a value, more issue time than the traffic
// takes, so channels go in pairs through fma.rn.f32x2 and two rows side by side.
// Measured, 8192 channels, 4 taps, bf16: 15,866 packed tokens 151 us (0.79 GB, 79 % of
// the copy bandwidth), 65,536 tokens from 8 bits 639 us (2.70 GB, 64 %); the FMA pipes
// are half busy and a warp's own latencies are the rest, with two warps to a scheduler
// because a thread keeps 128 values.  Four channels to a thread instead of eight, with
// twice the warps, repeat the work of each row too often: 166 and 722 us.
#include <type_traits>

#include "act8.cuh"
#include "f32x2.cuh"
#include "train_common.cuh"
#include "gdn_launch.h"
#include "sm100_ptx.cuh"

namespace gdn {
namespace convbwd {

constexpr int kThreads = 64;
constexpr int kStateThreads = 128;
constexpr int kMinRun = 32;    // tokens of a run at least

template <typename IO> struct Io;
template <> struct Io<float> { static constexpr int E = 4, kPerSm = 8; };          // channels of a thread, blocks per SM
template <> struct Io<__nv_bfloat16> { static constexpr int E = 8, kPerSm = 4; };  // 6 blocks, and so fewer registers: 165 and 675 us

struct Shape {
  int tiles;    // channel blocks
  int run;      // tokens of a run
  int blocks;   // runs
};
// Runs as long as one wave of resident blocks allows.
static Shape shape_of(int64_t tokens, int channels, int io_bf16) {
  Shape s;
  const int per = kThreads * (io_bf16 ? Io<__nv_bfloat16>::E : Io<float>::E);
  const int wave = 148 * (io_bf16 ? Io<__nv_bfloat16>::kPerSm : Io<float>::kPerSm);
  s.tiles = (channels + per - 1) / per;
  const int64_t most = wave / s.tiles > 0 ? wave / s.tiles : 1;
  int64_t run = (tokens + most - 1) / most;
  if (run < kMinRun) run = kMinRun;
  s.run = (int)run;
  s.blocks = (int)((tokens + run - 1) / run);
  return s;
}

template <int B> __device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(dst), "l"(src), "n"(B) : "memory");
}

// 16 bytes of IO as pairs, and back
template <typename IO> __device__ __forceinline__ void unpack(const void* p, F2* x);
template <> __device__ __forceinline__ void unpack<float>(const void* p, F2* x) {
  const float4 v = *static_cast<const float4*>(p);
  x[0] = f2(v.x, v.y);
  x[1] = f2(v.z, v.w);
}
template <> __device__ __forceinline__ void unpack<__nv_bfloat16>(const void* p, F2* x) {
  const uint4 v = *static_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
template <typename IO> __device__ __forceinline__ void store(IO* p, const F2* x);
template <> __device__ __forceinline__ void store<float>(float* p, const F2* x) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(x[0].x(), x[0].y(), x[1].x(), x[1].y()));
}
template <> __device__ __forceinline__ void store<__nv_bfloat16>(__nv_bfloat16* p, const F2* x) {
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(ptx::pack_bf16x2(x[0].x(), x[0].y()), ptx::pack_bf16x2(x[1].x(), x[1].y()),
                                                 ptx::pack_bf16x2(x[2].x(), x[2].y()), ptx::pack_bf16x2(x[3].x(), x[3].y())));
}
// E codes as pairs
template <int E> __device__ __forceinline__ void decode(const uint8_t* p, float f, F2* x) {
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    float v[4];
    act8::decode4(reinterpret_cast<const uint32_t*>(p)[i], f, v);
    x[2 * i] = f2(v[0], v[1]);
    x[2 * i + 1] = f2(v[2], v[3]);
  }
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
__global__ void __launch_bounds__(kThreads, Io<IO>::kPerSm) conv_bwd_kernel(ConvBwdArgs a, Shape sh, float* part) {
  let_next_begin();
  constexpr int E = Io<IO>::E, P = E / 2;
  constexpr int kX = k8 ? E : 16;          // bytes of a row of x
  constexpr int kDepth = 8;                // rows of the ring; 4 or 16: within 2 %
  constexpr int H = K - 1;                 // inputs before the token
  constexpr int HA = H > 0 ? H : 1;
  __shared__ __align__(16) uint8_t ring_y[kDepth][kThreads * 16];
  __shared__ __align__(16) uint8_t ring_x[kDepth][kThreads * kX];
  // scale bytes of 32 rows for a warp's channels (32 E of them: E groups)
  __shared__ __align__(4) uint8_t sbuf[k8 ? kThreads / 32 : 1][32][E];
  const int c0 = (blockIdx.x * kThreads + threadIdx.x) * E;
  const unsigned int lanes = __ballot_sync(0xffffffffu, c0 < a.channels);
  if (c0 >= a.channels) return;
  // tokens are counted from the run's first one, t0; dx of [0, own) needs dpre of [0, rows)
  const int64_t T = a.total_tokens, t0 = (int64_t)blockIdx.y * sh.run;
  const int own = (int)min((int64_t)sh.run, T - t0), rows = (int)min((int64_t)own + H, T - t0);
  size_t pitch;
  const IO* dy = dy_of<IO>(a, c0, pitch);
  const uint8_t* py = reinterpret_cast<const uint8_t*>(dy + (size_t)t0 * pitch);
  const size_t ypitch = pitch * sizeof(IO), xpitch = (size_t)a.channels * (kX / E);
  const uint8_t* px = static_cast<const uint8_t*>(a.x) + (size_t)t0 * xpitch + (size_t)c0 * (kX / E);
  const size_t spitch = (size_t)a.channels / act8::kGroup;
  IO* pdx = static_cast<IO*>(a.dx) + (size_t)t0 * a.channels + c0;
  const uint32_t by = (uint32_t)__cvta_generic_to_shared(&ring_y[0][threadIdx.x * 16]);
  const uint32_t bx = (uint32_t)__cvta_generic_to_shared(&ring_x[0][threadIdx.x * kX]);
  int fetched = 0;
  auto fetch = [&](int slot) {
    if (fetched < rows) {
      cp_async<16>(by + slot * (kThreads * 16), py);
      cp_async<kX>(bx + slot * (kThreads * kX), px);
      py += ypitch;
      px += xpitch;
    }
    ++fetched;
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
#pragma unroll
  for (int u = 0; u + 2 < kDepth; ++u) fetch(u);

  F2 w[K][P], b[P], dw[K][P], db[P], win[HA][P], pend[HA][P];
  const F2 zero = f2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < P; ++e) {
    const int c = c0 + 2 * e;
    b[e] = a.bias ? f2(a.bias[c], a.bias[c + 1]) : zero;
    db[e] = zero;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      w[i][e] = f2(a.weight[(size_t)c * K + i], a.weight[(size_t)(c + 1) * K + i]);
      dw[i][e] = zero;
    }
  }
  int n = a.cu ? seq_of(a.cu, a.num_seqs, t0) : (int)(t0 / a.uniform_len);
  int64_t s0, s1;
  seq_bounds(a, n, s0, s1);
  // win[j]: input at the token - H + j; pend[j]: what is known of the gradient of the input at the token - H + j
#pragma unroll
  for (int j = 0; j < H; ++j) {
    const int64_t p = t0 - H + j;
#pragma unroll
    for (int e = 0; e < P; ++e) {
      float v[2];
#pragma unroll
      for (int m = 0; m < 2; ++m)
        v[m] = p >= s0 ? x_at<IO, k8>(a, p, c0 + 2 * e + m) : window_at<IO>(a, n, c0 + 2 * e + m, (int)(K + (p - s0)));
      win[j][e] = f2(v[0], v[1]);
      pend[j][e] = zero;
    }
  }
  // of the sequence: its tokens [lo, hi) in this run, where it ends, and from where d_conv_state_out adds to dx
  int lo, hi, stop, add;
  auto enter = [&]() {
    lo = (int)min((int64_t)rows, max((int64_t)0, s0 - t0));
    stop = (int)min((int64_t)rows, s1 - t0);
    hi = min(own, stop);
    add = a.dstate_out ? (int)min((int64_t)rows, s1 - K - t0) : rows;
  };
  enter();
  // dx of token i, which no later token adds to, if it is this run's and this sequence's
  auto emit = [&](int i, F2* g) {
    if (i < lo || i >= hi) return;
    if (i >= add) {
      const IO* d = static_cast<const IO*>(a.dstate_out) + ((size_t)n * a.channels + c0) * K + (t0 + i - (s1 - K));
#pragma unroll
      for (int e = 0; e < P; ++e) g[e] = add2(g[e], f2(to_f32(d[2 * e * K]), to_f32(d[(2 * e + 1) * K])));
    }
    store<IO>(pdx + (size_t)i * a.channels, g);
  };
  // before row i, a multiple of 32: the scale bytes of the 32 rows from it
  auto scales = [&](int i) {
    if constexpr (k8) {
      const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, m = __popc(lanes);
      const int first = (c0 - lane * E) / act8::kGroup;  // of the warp's groups; there are an even number of all
      __syncwarp(lanes);
      for (int r = lane; r < 32 && i + r < rows; r += m) {
        const uint8_t* src = a.x_scales + (size_t)(t0 + i + r) * spitch + first;
#pragma unroll
        for (int j = 0; j < E; j += 2)
          if (first + j < (int)spitch) *reinterpret_cast<uint16_t*>(&sbuf[warp][r][j]) = *reinterpret_cast<const uint16_t*>(src + j);
      }
      __syncwarp(lanes);
    }
  };
  auto scale_of = [&](int i) { return k8 ? (uint32_t)sbuf[threadIdx.x / 32][i & 31][(threadIdx.x & 31) * E / act8::kGroup] : 127u; };
  // Token i: its share of dw and dbias, of the pending gradients, and dx of token i - H.  kInside: the token is
  // this run's and its sequence's, and so is token i - H, which d_conv_state_out does not add to.
  auto load = [&](int i, uint32_t scale, F2* g, F2* v) {
    unpack<IO>(&ring_y[i % kDepth][threadIdx.x * 16], g);
    if constexpr (k8)
      decode<E>(&ring_x[i % kDepth][threadIdx.x * kX], act8::factor(scale), v);
    else
      unpack<IO>(&ring_x[i % kDepth][threadIdx.x * kX], v);
  };
  // two rows are in flight less than the ring holds: what comes in next replaces rows that are done with
  auto arrived = [&]() { asm volatile("cp.async.wait_group %0;\n" ::"n"(kDepth - 2) : "memory"); };
  auto row = [&](int i, F2* g, F2* v, auto inside) {
    constexpr bool kInside = decltype(inside)::value;
    F2 last[P];
    if (!kInside && (i < lo || i >= stop)) {  // of no sequence (inconsistent cu_seqlens, already reported)
#pragma unroll
      for (int e = 0; e < P; ++e) g[e] = zero;
    }
#pragma unroll
    for (int e = 0; e < P; ++e) {
      F2 pre = b[e];
#pragma unroll
      for (int j = 0; j < H; ++j) pre = fma2(w[j][e], win[j][e], pre);
      pre = fma2(w[K - 1][e], v[e], pre);
      g[e] = mul2(g[e], silu_slope(pre));
#pragma unroll
      for (int j = 0; j < H; ++j) pend[j][e] = fma2(w[j][e], g[e], pend[j][e]);
      last[e] = mul2(w[K - 1][e], g[e]);
    }
    if (kInside || i < own) {
#pragma unroll
      for (int e = 0; e < P; ++e) {
        db[e] = add2(db[e], g[e]);
#pragma unroll
        for (int j = 0; j < H; ++j) dw[j][e] = fma2(g[e], win[j][e], dw[j][e]);
        dw[K - 1][e] = fma2(g[e], v[e], dw[K - 1][e]);
      }
    }
    F2* out = H > 0 ? pend[0] : last;
    if constexpr (kInside)
      store<IO>(pdx + (size_t)(i - H) * a.channels, out);
    else
      emit(i - H, out);
    if constexpr (H > 0) {
#pragma unroll
      for (int e = 0; e < P; ++e) {
#pragma unroll
        for (int j = 0; j + 1 < H; ++j) {
          win[j][e] = win[j + 1][e];
          pend[j][e] = pend[j + 1][e];
        }
        win[HA - 1][e] = v[e];
        pend[HA - 1][e] = last[e];
      }
    }
  };
  int i = 0;
  while (i < rows) {
    for (const int to = min(hi - 4, add - 4 + H); i >= lo + H && i <= to; i += 4) {
      if ((i & 31) == 0) scales(i);
#pragma unroll
      for (int u = 0; u < 4; u += 2) {  // two rows' loads and slopes side by side: one at a time, 156 and 678 us
        F2 g[2][P], v[2][P];
        fetch((i + u + kDepth - 2) % kDepth);
        fetch((i + u + kDepth - 1) % kDepth);
        arrived();
        load(i + u, scale_of(i + u), g[0], v[0]);
        load(i + u + 1, scale_of(i + u + 1), g[1], v[1]);
        row(i + u, g[0], v[0], std::true_type{});
        row(i + u + 1, g[1], v[1], std::true_type{});
      }
    }
    if (i < rows && (i & 31) == 0) scales(i);
#pragma unroll 1
    for (int u = 0; u < 4 && i < rows; ++u, ++i) {
      if (i >= stop) {  // the next sequence that has tokens begins
#pragma unroll
        for (int j = 0; j < H; ++j) emit(i - H + j, pend[j]);
        if (i >= own) {  // it is all behind the run
          i = rows + 1;
          break;
        }
        while (t0 + i >= s1 && n + 1 < a.num_seqs) {
          ++n;
          seq_bounds(a, n, s0, s1);
        }
        if (t0 + i >= s1) {  // of no sequence, and neither is what follows (inconsistent cu_seqlens, already reported)
          i = rows + 1;
          break;
        }
        enter();
#pragma unroll
        for (int j = 0; j < H; ++j)
#pragma unroll
          for (int e = 0; e < P; ++e) {
            win[j][e] = f2(window_at<IO>(a, n, c0 + 2 * e, j + 1), window_at<IO>(a, n, c0 + 2 * e + 1, j + 1));
            pend[j][e] = zero;
          }
      }
      F2 g[P], v[P];
      fetch((i + kDepth - 2) % kDepth);
      arrived();
      load(i, scale_of(i), g, v);
      row(i, g, v, std::false_type{});
    }
    if (i == rows) {
#pragma unroll
      for (int j = 0; j < H; ++j) emit(rows - H + j, pend[j]);
    }
  }
  asm volatile("cp.async.wait_group 0;\n" ::: "memory");  // no copy outlives the block
  float* p = part + (size_t)blockIdx.y * (K + 1) * a.channels + c0;
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const F2 s = j < K ? dw[j < K ? j : 0][e] : db[e];
      *reinterpret_cast<float2*>(p + (size_t)j * a.channels + 2 * e) = make_float2(s.x(), s.y());
    }
}

// dw[c, i] and dbias[c] from the runs' parts [run][K + 1][channels]: 32 columns by 8 shares of the runs
__global__ void __launch_bounds__(256) conv_weight_kernel(const float* part, int runs, int channels, int K, float* dw, float* db) {
  let_next_begin();
  wait_for_previous();
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
__global__ void __launch_bounds__(kStateThreads) conv_state_bwd_kernel(ConvBwdArgs a) {
  wait_for_previous();
  const int64_t idx = (int64_t)blockIdx.x * kStateThreads + threadIdx.x;
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
  const Shape sh = shape_of(a.total_tokens, a.channels, sizeof(IO) == 2);
  cudaError_t e;
  if (sh.blocks > 0) {
    conv_bwd_kernel<IO, K, k8><<<dim3(sh.tiles, sh.blocks), kThreads, 0, s>>>(a, sh, part);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  e = launch_next(conv_weight_kernel, dim3((a.channels + 31) / 32, K + 1), 256, 0, s, part, sh.blocks, a.channels, K, a.dw, a.db);
  if (e != cudaSuccess || !a.dstate_in) return e;
  const int64_t threads = (int64_t)a.num_seqs * a.channels;
  return launch_next(conv_state_bwd_kernel<IO, K, k8>, (unsigned int)((threads + kStateThreads - 1) / kStateThreads), kStateThreads, 0, s, a);
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

int64_t conv_bwd_workspace(int64_t tokens, int channels, int ksize, int io_bf16) {
  return (int64_t)convbwd::shape_of(tokens, channels, io_bf16).blocks * (ksize + 1) * channels * (int64_t)sizeof(float);
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
