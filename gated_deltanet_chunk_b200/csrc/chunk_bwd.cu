// chunk_bwd.cu -- gradients of the chunked gated delta rule (gdn_chunk_bwd).
//
// Notation of chunk_simt.cu, per chunk of C = 64 tokens and v-head, with q_hat,
// k_hat the normalised rows (the scale s kept apart), gc the in-chunk inclusive
// cumsum of g, e_r = exp(gc_r), l_r = exp(gc_last - gc_r), b = beta,
// Gamma_ri = exp(gc_r - gc_i) for i <= r, S the state before the chunk:
//
//   Kd = strictLower(K K^T Gamma),  A = -diag(b) Kd,  T = (I - A)^-1
//   P  = s lower(Q K^T Gamma)
//   X  = diag(b) (V - diag(e) K S),  V' = T X = U - W S,
//        U = T diag(b) V,  W = T diag(b e) K
//   O  = s diag(e) Q S + P V',   S' = e_last S + (diag(l) K)^T V'
//
// Given dO and dS' (the gradient of the state behind the chunk), the chain rule
// through these lines, with V' = X + A V' differentiated implicitly, gives
//
//   dV' = P^T dO + diag(l) K dS',   dX = T^T dV'
//   dS  = e_last dS' + (s diag(e) Q)^T dO - W^T dV'
//   dA  = strictLower(dX V'^T),     dP = lower(dO V'^T)
//   dQ  = s diag(e) dO S^T + N K,               N = s dP Gamma
//   dK  = diag(l) V' dS'^T - diag(b e) dX S^T + N^T Q + (B + B^T) K,
//                                               B = -diag(b) dA Gamma
//   dV  = diag(b) dX
//   db_r  = dX_r . V_r - e_r k_r . (dX S^T)_r - sum_i (dA Kd)_ri
//   dgc_r = sum_i (P dP + A dA)_ri - sum_i (P dP + A dA)_ir
//           + e_r s q_r . (dO S^T)_r - b_r e_r k_r . (dX S^T)_r - l_r k_r . (V' dS'^T)_r
//   dgc_last += e_last <S, dS'> + sum_r l_r k_r . (V' dS'^T)_r
//   dg_t  = sum_{r >= t} dgc_r          (within the chunk)
//
// and the L2 norm's own gradient, dq = (dq_hat - q_hat (q_hat . dq_hat)) / |q|.
//
// Only S -> S' and dS' -> dS are sequential, and both are separable in the Dv
// columns.  So three kernels run one after another:
//   1. prepare (every chunk and v-head at once): T, U, W, Y = P^T dO.
//   2. states: one warp per 16 Dv columns walks its sequence, forwards for S
//      and V', backwards for dS' and dV'.  The state slice stays in the warp's
//      registers as S^T [16 x Dk] MMA accumulators, whose layout is that of
//      the next product's A operand, so a chunk is two (or three) chained
//      products without a shared-memory round trip.  The two directions need
//      nothing of each other and run in the same launch.
//   3. gradients (every chunk and qk-head at once): the rest.  One block takes
//      all the v-heads that share a qk-head, one after another, so dq and dk
//      are summed in registers, in a fixed order.
// What they pass on is fp32 in the caller's workspace, but for the states kernel's
// B operands.  Every operand is a pair hi + lo of lower precision: three MMAs, and
// each product within about 2^-22 of its value.  Prepare and gradients split into
// TF32 as they load; the states kernel, which is bound by what a single warp can
// do, takes fp16 pairs (under powers of two shared by a row or a tile) at twice
// TF32's rate, formed once by prepare and fetched as images.  With TF32 pairs split
// on the way its loop was 7,700 instructions long and ran out of the instruction
// cache: 2.26 ms against 0.64 for 4 x 4096 tokens, 4 / 8 heads of 128.  Partial sums
// of one MMA step (8 or 16 terms) are added in fp32: the MMA itself truncates, and
// over long sums that showed (3.8e-6 relative against 64 bits; now 3.2e-7).

#include "chunk_bwd.cuh"
#include "gdn_common.cuh"
#include "gdn_launch.h"
#include "sm100_ptx.cuh"

namespace gdn {
namespace bwd {

constexpr int kThreads = 256;   // prepare and gradients

// One record per (chunk slot, v-head) in the workspace, in floats.
template <int DK, int DV>
struct Rec {
  static constexpr size_t kT = 0;                 // [C][C] T
  static constexpr size_t kW = kT + C * C;        // images of W [C][DK]: hi, lo
  static constexpr size_t kU = kW + C * DK;       // U^T as accumulators, then V'^T [DV][C]
  static constexpr size_t kY = kU + C * DV;       // (P^T dO)^T as accumulators, then dV'^T [DV][C]
  static constexpr size_t kOq = kY + C * DV;      // (diag(qe) dO)^T as A fragments: hi, lo
  static constexpr size_t kS = kOq + C * DV;      // [DV][DK] S^T before the chunk
  static constexpr size_t kD = kS + DV * DK;      // [DV][DK] dS'^T behind the chunk
  static constexpr size_t kKw = kD + DV * DK;     // [C] l_r over the factor of row r of K16
  static constexpr size_t kOf = kKw + C;          // [DV] 1 / factor of the columns of Dv in Oq
  static constexpr size_t kScal = kOf + DV;       // e_last, 1 / factor of W (padded to C)
  static constexpr size_t kFloats = kScal + C;
};
// One record per (chunk slot, qk-head), in floats: images of k_hat and s e... q_hat under factors by row
template <int DK>
struct QkRec {
  static constexpr size_t kK = 0;                 // images [C][DK] of k_hat: hi, lo
  static constexpr size_t kQ = kK + C * DK;       // of q_hat
  static constexpr size_t kFloats = kQ + C * DK;
};
template <int DK, int DV>
__device__ __forceinline__ float* rec_at(const BwdArgs& a, int64_t slot, int h) {
  return a.ws + ((size_t)slot * a.nv + h) * Rec<DK, DV>::kFloats;
}
template <int DK, int DV>
__device__ __forceinline__ float* qk_at(const BwdArgs& a, int64_t slot, int hq) {
  const size_t slots = (size_t)(a.total_tokens / C + a.num_seqs);
  return a.ws + slots * a.nv * Rec<DK, DV>::kFloats + ((size_t)slot * a.nqk + hq) * QkRec<DK>::kFloats;
}

// x f as a pair of fp16, hi + lo, two values at a time
__device__ __forceinline__ void pair2(float x, float y, float f, uint32_t& hi, uint32_t& lo) {
  x *= f;
  y *= f;
  hi = pack2(x, y);
  const float2 h = unpack2(hi);
  lo = pack2(x - h.x, y - h.y);
}

// Rows [c0, c0 + C) of one head of a [T, heads, D] tensor into a tile of pitch P
// (rows from `end` on as zeros), and the L2-norm factor of every row into
// norm[] when it is not null, and the factor of two that brings the row's largest
// element to [2^7, 2^8) into fac[].  One warp per row, 8 rows in turn per warp.
template <int D, int P, typename IO>
__device__ __forceinline__ void load_rows(const IO* x, int64_t c0, int64_t end, int heads, int head, float* tile,
                                          float* norm, float* fac, bool l2, int warp, int lane) {
  constexpr int PER = D / 32;
#pragma unroll 4
  for (int r = warp; r < C; r += kThreads / 32) {
    const int64_t tk = c0 + r;
    const bool valid = tk < end;
    const IO* src = x + ((size_t)(valid ? tk : c0) * heads + head) * D;
    float v[PER], ss = 0.f, top = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      v[e] = valid ? to_f32(src[lane + 32 * e]) : 0.f;
      ss = fmaf(v[e], v[e], ss);
      top = fmaxf(top, fabsf(v[e]));
    }
    float f = 1.f;
    if (norm) {
      ss = warp_sum(ss);
      f = l2 ? 1.f / sqrtf(ss + kNormEps) : 1.f;
      if (lane == 0) norm[r] = f;
    }
    if (fac) {
      const float m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top * f)));
      float fr, inv;
      pow2_factor(m, fr, inv);
      if (lane == 0) fac[r] = fr;
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) tile[r * P + lane + 32 * e] = v[e] * f;
  }
}

// ------------------------------------------------------------------ 1. prepare

template <int DK, int DV>
struct PrepSmem {
  static constexpr int KP = DK + 4, VP = DV + 4;
  static constexpr int kK = 0;                 // [C][KP] k_hat
  static constexpr int kQ = kK + C * KP;       // [C][KP] q_hat
  static constexpr int kV = kQ + C * KP;       // [C][VP] V
  static constexpr int kO = kV + C * VP;       // [C][VP] dO
  static constexpr int kA = kO + C * VP;       // [C][TP] A, then T
  static constexpr int kP = kA + C * TP;       // [C][TP] the inverse's scratch, then P
  static constexpr int kGc = kP + C * TP;      // [C] gcum
  static constexpr int kBeta = kGc + C;
  static constexpr int kBe = kBeta + C;        // [2][C] beta e; e over the factor of row r of q_hat
  static constexpr int kNq = kBe + 2 * C;      // [C] 1 / |q|
  static constexpr int kNk = kNq + C;          // [C] 1 / |k|
  static constexpr int kFk = kNk + C;          // [C] factor of two of row r of k_hat
  static constexpr int kFq = kFk + C;          // of q_hat
  static constexpr int kTop = kFq + C;         // [8] largest |W| by warp
  static constexpr int kTotal = kTop + 8;
  static constexpr size_t kBytes = size_t(kTotal) * sizeof(float);
  static_assert(kBytes <= 232448, "shared memory budget");
};

template <int DK, int DV, typename IO>
__global__ void __launch_bounds__(kThreads, 1) prepare_kernel(BwdArgs a) {
  using L = PrepSmem<DK, DV>;
  using R = Rec<DK, DV>;
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
  const int h = blockIdx.y;
  const int64_t slot = blockIdx.x;
  int64_t c0, end;
  if (!chunk_at(a, slot, c0, end)) return;
  const int hq = h / (a.nv / a.nqk);
  float *K = sm + L::kK, *Q = sm + L::kQ, *V = sm + L::kV, *O = sm + L::kO, *A = sm + L::kA, *P = sm + L::kP;
  float *gc = sm + L::kGc, *bt = sm + L::kBeta, *be = sm + L::kBe, *nq = sm + L::kNq, *nk = sm + L::kNk;
  float *fk = sm + L::kFk, *fq = sm + L::kFq, *tops = sm + L::kTop;
  float* rec = rec_at<DK, DV>(a, slot, h);

  load_rows<DK, L::KP>(static_cast<const IO*>(a.k), c0, end, a.nqk, hq, K, nk, fk, a.qk_l2norm != 0, warp, lane);
  load_rows<DK, L::KP>(static_cast<const IO*>(a.q), c0, end, a.nqk, hq, Q, nq, fq, a.qk_l2norm != 0, warp, lane);
  load_rows<DV, L::VP>(static_cast<const IO*>(a.v), c0, end, a.nv, h, V, (float*)nullptr, (float*)nullptr, false, warp, lane);
  load_rows<DV, L::VP>(static_cast<const IO*>(a.dout), c0, end, a.nv, h, O, (float*)nullptr, (float*)nullptr, false, warp, lane);
  if (tid < C) {
    float gv = 0.f, bv = 0.f;
    if (c0 + tid < end) load_gate(a, (size_t)(c0 + tid) * a.nv + h, h, gv, bv);
    gc[tid] = gv;
    bt[tid] = bv;
  }
  __syncthreads();
  if (warp == 0) cumsum_chunk(gc, lane);
  __syncthreads();
  if (tid < C) {
    const float e = expf(gc[tid]);
    be[tid] = bt[tid] * e;
    be[C + tid] = e / fq[tid];
    rec[R::kKw + tid] = expf(gc[C - 1] - gc[tid]) / fk[tid];  // a power of two
    if (tid == C - 1) rec[R::kScal] = e;
  }
  if (h % (a.nv / a.nqk) == 0) {  // K16 and Q16, once for the qk-head
    uint8_t* qrec = reinterpret_cast<uint8_t*>(qk_at<DK, DV>(a, slot, hq));
    for (int i = tid; i < 2 * C * DK / 8; i += kThreads) {
      const int m = i / (C * DK / 8), r = i / (DK / 8) % C, c = 8 * (i % (DK / 8));
      const float* src = (m ? Q : K) + r * L::KP + c;
      const float f = (m ? fq : fk)[r];
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) pair2(src[2 * e], src[2 * e + 1], f, hi[e], lo[e]);
      uint8_t* dst = qrec + 4 * (m ? QkRec<DK>::kQ : QkRec<DK>::kK) + image<2 * DK>(r, c);
      *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(dst + 2 * C * DK) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  // warp: rows 16 wr .. + 15, columns by the half wc
  const int wr = 16 * (warp & 3), wc = warp >> 2;
  // A, and later P: entries above the diagonal are zero; whole 8-column tiles above it are not formed
  auto pairs = [&](const float* X, float (&acc)[4][4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
    if (32 * wc < wr + 16)
      warp_gemm<4>(acc, 0, DK, [&](int m, int k) { return X[(wr + m) * L::KP + k]; },
                   [&](int k, int n) { return K[(32 * wc + n) * L::KP + k]; }, g8, t4);
  };
  float acc[4][4], accp[4][4];
  pairs(K, acc);
  pairs(Q, accp);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = wr + g8 + 8 * (e >> 1), i = 32 * wc + 8 * j + 2 * t4 + (e & 1);
      const float gamma = i <= r ? expf(gc[r] - gc[i]) : 0.f;  // masked before exp
      A[r * TP + i] = i < r ? -bt[r] * (acc[j][e] * gamma) : 0.f;
      accp[j][e] = i <= r ? a.scale * accp[j][e] * gamma : 0.f;
    }
  __syncthreads();
  invert_chunk<true>(A, P, warp, lane);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = wr + g8 + 8 * (e >> 1), i = 32 * wc + 8 * j + 2 * t4 + (e & 1);
      P[r * TP + i] = accp[j][e];
      rec[R::kT + r * C + i] = A[r * TP + i];
    }
  __syncthreads();
  {  // W = T diag(b e) K, as pairs under one factor for the tile
    constexpr int NT = DK / 16;
    float x[NT][4] = {}, top = 0.f, f, inv;
    const int n0 = 8 * NT * wc;
    warp_gemm<NT>(x, 0, wr + 16, [&](int m, int k) { return A[(wr + m) * TP + k]; },
                  [&](int k, int n) { return be[k] * K[k * L::KP + n0 + n]; }, g8, t4);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(x[j][e]));
    const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    if (lane == 0) tops[warp] = __uint_as_float(w);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, tops[i]);
    pow2_factor(top, f, inv);
    if (tid == 0) rec[R::kScal + 1] = inv;
    uint8_t* img = reinterpret_cast<uint8_t*>(rec + R::kW);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int at = image<2 * DK>(wr + g8 + 4 * e, n0 + 8 * j + 2 * t4);
        uint32_t hi, lo;
        pair2(x[j][e], x[j][e + 1], f, hi, lo);
        *reinterpret_cast<uint32_t*>(img + at) = hi;
        *reinterpret_cast<uint32_t*>(img + 2 * C * DK + at) = lo;
      }
  }
  // U^T = V^T (T diag(b))^T and Y^T = dO^T P, 16 columns of Dv a unit
  for (int u = warp; u < DV / 8; u += kThreads / 32) {
    const bool isY = u >= DV / 16;
    const int m0 = 16 * (u % (DV / 16));
    float x[8][4] = {};
    if (isY)
      warp_gemm<8>(x, 0, C, [&](int m, int k) { return O[k * L::VP + m0 + m]; }, [&](int k, int n) { return P[k * TP + n]; }, g8, t4);
    else
      warp_gemm<8>(x, 0, C, [&](int m, int k) { return V[k * L::VP + m0 + m]; }, [&](int k, int n) { return A[n * TP + k] * bt[k]; }, g8, t4);
    float4* dst = reinterpret_cast<float4*>(rec + (isY ? R::kY : R::kU)) + (m0 / 16) * 256 + lane;
#pragma unroll
    for (int j = 0; j < 8; ++j) dst[32 * j] = make_float4(x[j][0], x[j][1], x[j][2], x[j][3]);
  }
  // (diag(s e) dO)^T over q_hat's factors, as fragments: rows m0 + g, + 8 (columns of Dv), pairs of tokens
  for (int u = warp; u < DV / 16; u += kThreads / 32) {
    const int c = 16 * u + g8;
    float x[8][4], top[2] = {0.f, 0.f}, f[2], inv[2];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 8 * j + 2 * t4 + (e & 1);
        x[j][e] = O[r * L::VP + c + 8 * (e >> 1)] * (a.scale * be[C + r]);
        top[e >> 1] = fmaxf(top[e >> 1], fabsf(x[j][e]));
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
      pow2_factor(top[e], f[e], inv[e]);
      if (t4 == 0) rec[R::kOf + c + 8 * e] = inv[e];
    }
    uint4* dst = reinterpret_cast<uint4*>(rec + R::kOq) + u * 128 + lane;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) pair2(x[2 * k + (e >> 1)][2 * (e & 1)], x[2 * k + (e >> 1)][2 * (e & 1) + 1], f[e & 1], hi[e], lo[e]);
      dst[32 * k] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      dst[DV * 8 + 32 * k] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
}

// ------------------------------------------------------------------ 2. states
// One block per (sequence, v-head, direction, 64 columns of Dv), one warp per 16 columns.

constexpr int kStateWarps = 4;
constexpr int kStateThreads = 32 * kStateWarps;

template <int DK>
struct StateSmem {
  static constexpr size_t kTile = 2 * C * DK;            // one image; W, K16 and (backwards) Q16 as hi and lo
  static constexpr size_t kStage = 6 * kTile + 4 * C;    // and kw
  static constexpr size_t kBar = 2 * kStage;
  static constexpr size_t kBytes = kBar + 16;
  static_assert(kStage % 128 == 0 && kBytes <= 232448, "shared memory budget");
};

// Rows g and g + 8 of two 16 x 8 tiles, times f0 and f1, as A fragments hi and lo
__device__ __forceinline__ void pair_frag(const float* lo8, const float* hi8, float f0, float f1, uint32_t* hi, uint32_t* lo) {
  pair2(lo8[0], lo8[1], f0, hi[0], lo[0]);
  pair2(lo8[2], lo8[3], f1, hi[1], lo[1]);
  pair2(hi8[0], hi8[1], f0, hi[2], lo[2]);
  pair2(hi8[2], hi8[3], f1, hi[3], lo[3]);
}
// The factors of two of rows g and g + 8 of accumulators, from this thread's largest of each
__device__ __forceinline__ void row_factors(float (&top)[2], float (&f)[2], float (&inv)[2]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
    top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
    pow2_factor(top[e], f[e], inv[e]);
  }
}
// x[8] (64 columns from n0) += (hi + lo) B[16 k .. + 15], B an image pair [n][k] (kT: [k][n]) whose lo stands `tile` behind
template <int RB, bool kT>
__device__ __forceinline__ void mma_pairs(float (&x)[8][4], const uint32_t* hi, const uint32_t* lo, uint32_t img, uint32_t tile,
                                          int n0, int k, const Lane& ln) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t bh[4], bl[4];
    if (kT) {
      img_b_t<RB>(bh, img, n0 + 16 * j, 16 * k, ln);
      img_b_t<RB>(bl, img + tile, n0 + 16 * j, 16 * k, ln);
    } else {
      img_b<RB>(bh, img, n0 + 16 * j, 16 * k, ln);
      img_b<RB>(bl, img + tile, n0 + 16 * j, 16 * k, ln);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float d[4] = {};
      mma_f16(d, lo, bh + 2 * m);
      mma_f16(d, hi, bl + 2 * m);
      mma_f16(d, hi, bh + 2 * m);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[2 * j + m][e] += d[e];
    }
  }
}

template <int DK, int DV, bool kBackward>
__device__ __forceinline__ void walk(const BwdArgs& a, uint8_t* sm, int n, int h, int col0) {
  using L = StateSmem<DK>;
  using R = Rec<DK, DV>;
  using QR = QkRec<DK>;
  constexpr int ND = DK / 8, RB = 2 * DK;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int slice = col0 / 16 + warp, c = 16 * slice + g;  // this thread's columns of Dv: c and c + 8
  const int hq = h / (a.nv / a.nqk);
  Lane ln(lane);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::kBar);
  int64_t start, end;
  seq_bounds(a, n, start, end);
  const int64_t chunks = (end - start + C - 1) / C, slot0 = start / C + n;

  float s[ND][4];  // S^T or dS^T: rows c, c + 8, columns d = 8 j + 2 t, + 1
  const float* init = kBackward ? a.ds_final : a.s0;
  const size_t state_off = ((size_t)n * a.nv + h) * (size_t)DK * DV;
#pragma unroll
  for (int j = 0; j < ND; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s[j][e] = init ? init[state_off + (size_t)(8 * j + 2 * t + (e & 1)) * DV + c + 8 * (e >> 1)] : 0.f;

  auto slot_of = [&](int64_t i) { return slot0 + (kBackward ? chunks - 1 - i : i); };
  auto fetch = [&](int64_t i) {  // by one thread
    if (i >= chunks) return;
    uint8_t* st = sm + (i & 1) * L::kStage;
    const float* rec = rec_at<DK, DV>(a, slot_of(i), h);
    constexpr uint32_t tiles = (kBackward ? 4 : 2) * L::kTile;
    ptx::mbar_arrive_expect_tx(bar + (i & 1), (uint32_t)(2 * L::kTile + tiles + 4 * C));
    bulk_copy(st, rec + R::kW, 2 * L::kTile, bar + (i & 1));
    bulk_copy(st + 2 * L::kTile, qk_at<DK, DV>(a, slot_of(i), hq) + QR::kK, tiles, bar + (i & 1));  // Q16 stands behind K16
    bulk_copy(st + 6 * L::kTile, rec + R::kKw, 4 * C, bar + (i & 1));
  };
  if (tid == 0) {
    ptx::mbar_init(bar, 1);
    ptx::mbar_init(bar + 1, 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();
  if (tid == 0) {
    fetch(0);
    fetch(1);
  }
  for (int64_t i = 0; i < chunks; ++i) {
    float* rec = rec_at<DK, DV>(a, slot_of(i), h);
    const float gl = rec[R::kScal], winv = rec[R::kScal + 1];
    // the state as this chunk meets it, for the gradients
    float* sv = rec + (kBackward ? R::kD : R::kS) + (size_t)c * DK + 2 * t;
    float top[2] = {0.f, 0.f}, sf[2], sinv[2];
#pragma unroll
    for (int j = 0; j < ND; ++j) {
      *reinterpret_cast<float2*>(sv + 8 * j) = make_float2(s[j][0], s[j][1]);
      *reinterpret_cast<float2*>(sv + 8 * DK + 8 * j) = make_float2(s[j][2], s[j][3]);
      top[0] = fmaxf(top[0], fmaxf(fabsf(s[j][0]), fabsf(s[j][1])));
      top[1] = fmaxf(top[1], fmaxf(fabsf(s[j][2]), fabsf(s[j][3])));
    }
    row_factors(top, sf, sinv);
    const bool ok = ptx::mbar_wait_bounded(bar + (i & 1), (uint32_t)((i >> 1) & 1), kWaitLimitNs);
    const uint8_t* st = sm + (i & 1) * L::kStage;
    const uint32_t W = ptx::smem_u32(st), K = W + 2 * (uint32_t)L::kTile, Q = W + 4 * (uint32_t)L::kTile;
    const float* kw = reinterpret_cast<const float*>(st + 6 * L::kTile);
    // x = S^T W^T (forwards) or dS'^T K^T (backwards), [16 x C]
    float x[8][4] = {};
#pragma unroll
    for (int k = 0; k < ND / 2; ++k) {
      uint32_t hi[4], lo[4];
      pair_frag(s[2 * k], s[2 * k + 1], sf[0], sf[1], hi, lo);
      mma_pairs<RB, false>(x, hi, lo, kBackward ? K : W, (uint32_t)L::kTile, 0, k, ln);
    }
    // forwards V'^T = U^T - x, backwards dV'^T = Y^T + x diag(kw); stored over U^T, Y^T (this warp's 4 KB)
    const float4* uw = reinterpret_cast<const float4*>(rec + (kBackward ? R::kY : R::kU)) + slice * 256 + lane;
    float4 u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = uw[32 * j];
    __syncwarp();
    float* vv = rec + (kBackward ? R::kY : R::kU) + (size_t)c * C + 2 * t;
    top[0] = top[1] = 0.f;
    float vf[2], vinv[2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 w = *reinterpret_cast<const float2*>(kw + 8 * j + 2 * t);
      const float2 f = kBackward ? w : make_float2(-winv, -winv);
      x[j][0] = fmaf(x[j][0] * sinv[0], f.x, u[j].x);
      x[j][1] = fmaf(x[j][1] * sinv[0], f.y, u[j].y);
      x[j][2] = fmaf(x[j][2] * sinv[1], f.x, u[j].z);
      x[j][3] = fmaf(x[j][3] * sinv[1], f.y, u[j].w);
      *reinterpret_cast<float2*>(vv + 8 * j) = make_float2(x[j][0], x[j][1]);
      *reinterpret_cast<float2*>(vv + 8 * C + 8 * j) = make_float2(x[j][2], x[j][3]);
      if (!kBackward) {
        x[j][0] *= w.x;
        x[j][1] *= w.y;
        x[j][2] *= w.x;
        x[j][3] *= w.y;
      }
      top[0] = fmaxf(top[0], fmaxf(fabsf(x[j][0]), fabsf(x[j][1])));
      top[1] = fmaxf(top[1], fmaxf(fabsf(x[j][2]), fabsf(x[j][3])));
    }
    row_factors(top, vf, vinv);
    // forwards S^T = e_last S^T + (V' diag(kw))^T K, backwards dS^T = e_last dS'^T + (s diag(e) dO)^T Q - dV'^T W
    const float f0 = kBackward ? -vinv[0] * winv : vinv[0], f1 = kBackward ? -vinv[1] * winv : vinv[1];
#pragma unroll
    for (int m = 0; m < ND; m += 8) {  // 64 columns of Dk at a time
      float y[8][4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t hi[4], lo[4];
        pair_frag(x[2 * k], x[2 * k + 1], vf[0], vf[1], hi, lo);
        mma_pairs<RB, true>(y, hi, lo, kBackward ? W : K, (uint32_t)L::kTile, 8 * m, k, ln);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[m + j][e] = fmaf(e < 2 ? f0 : f1, y[j][e], gl * s[m + j][e]);
    }
    if (kBackward) {
      const uint4* ow = reinterpret_cast<const uint4*>(rec + R::kOq) + slice * 128 + lane;
      const float o0 = rec[R::kOf + c], o1 = rec[R::kOf + c + 8];
#pragma unroll
      for (int m = 0; m < ND; m += 8) {
        float y[8][4] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 h4 = ow[32 * k], l4 = ow[DV * 8 + 32 * k];
          const uint32_t hi[4] = {h4.x, h4.y, h4.z, h4.w}, lo[4] = {l4.x, l4.y, l4.z, l4.w};
          mma_pairs<RB, true>(y, hi, lo, Q, (uint32_t)L::kTile, 8 * m, k, ln);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[m + j][e] = fmaf(e < 2 ? o0 : o1, y[j][e], s[m + j][e]);
      }
    }
    if (__syncthreads_or(!ok)) {  // a copy never came: report it, wait once more for what is in flight, and leave
      if (tid == 0) {
        report_status(a.status, kStatusTimeout);
        ptx::mbar_wait_bounded(bar + (i & 1), (uint32_t)((i >> 1) & 1), kWaitLimitNs);
        if (i + 1 < chunks) ptx::mbar_wait_bounded(bar + ((i + 1) & 1), (uint32_t)(((i + 1) >> 1) & 1), kWaitLimitNs);
      }
      return;
    }
    if (tid == 0) fetch(i + 2);  // the stage is free
  }
  if (kBackward && a.ds0) {
#pragma unroll
    for (int j = 0; j < ND; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        a.ds0[state_off + (size_t)(8 * j + 2 * t + (e & 1)) * DV + c + 8 * (e >> 1)] = s[j][e];
  }
}

// blockIdx.x: direction and 64-column slice, y: v-head, z: sequence
template <int DK, int DV>
__global__ void __launch_bounds__(kStateThreads) states_kernel(BwdArgs a) {
  extern __shared__ __align__(128) uint8_t smb[];
  const int col0 = 16 * kStateWarps * (blockIdx.x >> 1);
  if (blockIdx.x & 1)
    walk<DK, DV, true>(a, smb, blockIdx.z, blockIdx.y, col0);
  else
    walk<DK, DV, false>(a, smb, blockIdx.z, blockIdx.y, col0);
}

// ------------------------------------------------------------------ 3. gradients

template <int DK>
struct GradSmem {
  static constexpr int KP = DK + 4, SP = DK + 8;
  static constexpr int kK = 0;                  // [C][KP] k_hat
  static constexpr int kQ = kK + C * KP;        // [C][KP] q_hat
  static constexpr int kKK = kQ + C * KP;       // [C][TP] k_r . k_i
  static constexpr int kQK = kKK + C * TP;      // [C][TP] q_r . k_i
  static constexpr int kT = kQK + C * TP;       // [C][TP] T
  static constexpr int kS = kT + C * TP;        // [64][SP] 64 rows of S^T, then of dS'^T
  static constexpr int kVn = kS + 64 * SP;      // [64][TP] V'^T rows, then N
  static constexpr int kO = kVn + C * TP;       // [C][TP] dO columns, then B
  static constexpr int kX = kO + C * TP;        // [64][TP] dV'^T rows, then dX^T
  static constexpr int kGc = kX + C * TP;       // [C] gcum
  static constexpr int kBeta = kGc + C;
  static constexpr int kEg = kBeta + C;         // [C] e
  static constexpr int kEl = kEg + C;           // [C] l
  static constexpr int kNq = kEl + C;           // [C] 1 / |q|
  static constexpr int kNk = kNq + C;           // [C] 1 / |k|
  static constexpr int kRed = kNk + C;          // [2][3][C] row sums by column half; [2][2][C] at the end
  static constexpr int kCol = kRed + 6 * C;     // [4][C] column sums by row block
  static constexpr int kDot = kCol + 4 * C;     // [8] <S, dS'> by warp
  static constexpr int kTotal = kDot + 8;
  static constexpr size_t kBytes = size_t(kTotal) * sizeof(float);
  static_assert(kS % 4 == 0 && kBytes <= 232448, "shared memory budget");
};

// x = D[C x 64] (kDT: kept as its transpose) S[64 x Dk] (rows wr .., column half wc): sum += f x by rows, dot = x . Y by rows (this thread's part).
template <int NK, int KP, int SP, bool kDT>
__device__ __forceinline__ void with_state(const float* D, const float* S, const float* Y, int wr, int wc, const float (&f)[2],
                                           float (&sum)[NK][4], float (&dot)[2], int g, int t) {
  float x[NK][4] = {};
  const int n0 = 8 * NK * wc;
  warp_gemm<NK>(x, 0, 64, [&](int m, int k) { return kDT ? D[k * TP + wr + m] : D[(wr + m) * TP + k]; },
                [&](int k, int n) { return S[k * SP + n0 + n]; }, g, t);
#pragma unroll
  for (int e2 = 0; e2 < 2; ++e2) {
    const float* y = Y + (wr + g + 8 * e2) * KP + n0 + 2 * t;
    dot[e2] = 0.f;
#pragma unroll
    for (int j = 0; j < NK; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        dot[e2] = fmaf(x[j][2 * e2 + e], y[8 * j + e], dot[e2]);
        sum[j][2 * e2 + e] = fmaf(f[e2], x[j][2 * e2 + e], sum[j][2 * e2 + e]);
      }
  }
}

template <int DK, int DV, typename IO>
__global__ void __launch_bounds__(kThreads, 1) grads_kernel(BwdArgs a) {
  using L = GradSmem<DK>;
  using R = Rec<DK, DV>;
  extern __shared__ __align__(16) float sm[];
  constexpr int NK = DK / 16;  // 8-column tiles of a warp's half of Dk
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
  const int hq = blockIdx.y, group = a.nv / a.nqk;
  const int64_t slot = blockIdx.x;
  int64_t c0, end;
  if (!chunk_at(a, slot, c0, end)) return;
  float *K = sm + L::kK, *Q = sm + L::kQ, *KK = sm + L::kKK, *QK = sm + L::kQK, *T = sm + L::kT, *S = sm + L::kS;
  float *Vn = sm + L::kVn, *O = sm + L::kO, *X = sm + L::kX;
  float *gc = sm + L::kGc, *bt = sm + L::kBeta, *eg = sm + L::kEg, *el = sm + L::kEl, *nq = sm + L::kNq, *nk = sm + L::kNk;
  float *red = sm + L::kRed, *col = sm + L::kCol, *dots = sm + L::kDot;

  load_rows<DK, L::KP>(static_cast<const IO*>(a.k), c0, end, a.nqk, hq, K, nk, (float*)nullptr, a.qk_l2norm != 0, warp, lane);
  load_rows<DK, L::KP>(static_cast<const IO*>(a.q), c0, end, a.nqk, hq, Q, nq, (float*)nullptr, a.qk_l2norm != 0, warp, lane);
  __syncthreads();
  // warp: rows 16 wr .. + 15 of every product, columns by the half wc; thread: rows r0, r0 + 8
  const int wr = 16 * (warp & 3), wc = warp >> 2, r0 = wr + g8;
  const bool low = 32 * wc < wr + 16;  // the warp's 16 x 32 block of a [C][C] product touches the lower triangle
  for (int m = 0; m < 2; ++m) {
    float* D = m ? QK : KK;
    const float* Xq = m ? Q : K;
    float acc[4][4] = {};
    if (low)
      warp_gemm<4>(acc, 0, DK, [&](int r, int k) { return Xq[(wr + r) * L::KP + k]; },
                   [&](int k, int n) { return K[(32 * wc + n) * L::KP + k]; }, g8, t4);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) D[(r0 + 8 * (e >> 1)) * TP + 32 * wc + 8 * j + 2 * t4 + (e & 1)] = acc[j][e];
  }
  float dq[NK][4] = {}, dk[NK][4] = {};  // summed over the v-heads of the group

  for (int h = hq * group; h < (hq + 1) * group; ++h) {
    const float* rec = rec_at<DK, DV>(a, slot, h);
    __syncthreads();  // the tiles and sums of the head before are consumed
    if (tid < C) {
      float gv = 0.f, bv = 0.f;
      if (c0 + tid < end) load_gate(a, (size_t)(c0 + tid) * a.nv + h, h, gv, bv);
      gc[tid] = gv;
      bt[tid] = bv;
    }
    __syncthreads();
    if (warp == 0) cumsum_chunk(gc, lane);
    for (int i = tid; i < C * C; i += kThreads) T[(i / C) * TP + i % C] = rec[R::kT + i];
    __syncthreads();
    if (tid < C) {
      eg[tid] = expf(gc[tid]);
      el[tid] = expf(gc[C - 1] - gc[tid]);
    }
    float dA[4][4] = {}, dP[4][4] = {};
    float s_gc[2] = {0.f, 0.f}, s_bt[2] = {0.f, 0.f}, s_th[2] = {0.f, 0.f}, s_dot = 0.f;
    for (int v0 = 0; v0 < DV; v0 += 64) {
      __syncthreads();
      for (int i = tid; i < C * 64; i += kThreads) {
        const int r = i / 64, cc = i % 64;
        Vn[r * TP + cc] = rec[R::kU + (size_t)(v0 + r) * C + cc];  // (column of Dv, token)
        X[r * TP + cc] = rec[R::kY + (size_t)(v0 + r) * C + cc];
        O[r * TP + cc] = c0 + r < end ? to_f32(static_cast<const IO*>(a.dout)[((size_t)(c0 + r) * a.nv + h) * DV + v0 + cc]) : 0.f;
      }
      for (int i = tid; i < 64 * DK; i += kThreads) S[(i / DK) * L::SP + i % DK] = rec[R::kS + (size_t)v0 * DK + i];
      __syncthreads();
      {  // dX = T^T dV'; dV = diag(b) dX
        float x[4][4] = {};
        warp_gemm<4>(x, wr, C, [&](int m, int k) { return T[k * TP + wr + m]; },
                     [&](int k, int n) { return X[(32 * wc + n) * TP + k]; }, g8, t4);
        __syncthreads();  // dV' is consumed
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = r0 + 8 * (e >> 1), cc = 32 * wc + 8 * j + 2 * t4 + (e & 1);
            X[cc * TP + r] = x[j][e];
            if (c0 + r < end) {
              const size_t at = ((size_t)(c0 + r) * a.nv + h) * DV + v0 + cc;
              s_bt[e >> 1] = fmaf(x[j][e], to_f32(static_cast<const IO*>(a.v)[at]), s_bt[e >> 1]);
              static_cast<IO*>(a.dv_out)[at] = from_f32<IO>(bt[r] * x[j][e]);
            }
          }
        __syncthreads();
      }
      if (low) {
        warp_gemm<4>(dA, 0, 64, [&](int m, int k) { return X[k * TP + wr + m]; },
                     [&](int k, int n) { return Vn[k * TP + 32 * wc + n]; }, g8, t4);
        warp_gemm<4>(dP, 0, 64, [&](int m, int k) { return O[(wr + m) * TP + k]; },
                     [&](int k, int n) { return Vn[k * TP + 32 * wc + n]; }, g8, t4);
      }
      // the products with the state: their row dots with q_hat or k_hat, and their shares of dq, dk
      float f[2], dot[2];
      f[0] = a.scale * eg[r0];
      f[1] = a.scale * eg[r0 + 8];
      with_state<NK, L::KP, L::SP, false>(O, S, Q, wr, wc, f, dq, dot, g8, t4);
#pragma unroll
      for (int e = 0; e < 2; ++e) s_gc[e] = fmaf(f[e], dot[e], s_gc[e]);
      f[0] = -bt[r0] * eg[r0];
      f[1] = -bt[r0 + 8] * eg[r0 + 8];
      with_state<NK, L::KP, L::SP, true>(X, S, K, wr, wc, f, dk, dot, g8, t4);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s_gc[e] = fmaf(f[e], dot[e], s_gc[e]);
        s_bt[e] = fmaf(-eg[r0 + 8 * e], dot[e], s_bt[e]);
      }
      __syncthreads();  // S is consumed
      for (int i = tid; i < 64 * DK; i += kThreads) {
        const float d = rec[R::kD + (size_t)v0 * DK + i];
        float* p = S + (i / DK) * L::SP + i % DK;
        s_dot = fmaf(*p, d, s_dot);
        *p = d;
      }
      __syncthreads();
      f[0] = el[r0];
      f[1] = el[r0 + 8];
      with_state<NK, L::KP, L::SP, true>(Vn, S, K, wr, wc, f, dk, dot, g8, t4);
#pragma unroll
      for (int e = 0; e < 2; ++e) s_th[e] = fmaf(f[e], dot[e], s_th[e]);
    }
    __syncthreads();  // V', dO are consumed
    float cs[4][2] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + 8 * (e >> 1), i = 32 * wc + 8 * j + 2 * t4 + (e & 1);
        const float gamma = i <= r ? expf(gc[r] - gc[i]) : 0.f;  // masked before exp
        const float kd = i < r ? KK[r * TP + i] * gamma : 0.f;
        const float da = i < r ? dA[j][e] : 0.f;
        const float dp = i <= r ? a.scale * dP[j][e] * gamma : 0.f;
        const float both = i < r ? dp * QK[r * TP + i] - bt[r] * kd * da : 0.f;
        s_bt[e >> 1] = fmaf(-da, kd, s_bt[e >> 1]);
        s_gc[e >> 1] += both;
        cs[j][e & 1] += both;
        Vn[r * TP + i] = dp;                                   // N
        O[r * TP + i] = i < r ? -bt[r] * da * gamma : 0.f;     // B
      }
    // row sums over the quad of lanes, column sums over the eight rows of lanes
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        s_gc[e] += __shfl_xor_sync(0xffffffffu, s_gc[e], o);
        s_bt[e] += __shfl_xor_sync(0xffffffffu, s_bt[e], o);
        s_th[e] += __shfl_xor_sync(0xffffffffu, s_th[e], o);
      }
      if (t4 == 0) {
        red[(3 * wc + 0) * C + r0 + 8 * e] = s_gc[e];
        red[(3 * wc + 1) * C + r0 + 8 * e] = s_bt[e];
        red[(3 * wc + 2) * C + r0 + 8 * e] = s_th[e];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) cs[j][e] += __shfl_xor_sync(0xffffffffu, cs[j][e], o);
        if (g8 == 0) col[(warp & 3) * C + 32 * wc + 8 * j + 2 * t4 + e] = cs[j][e];
      }
    s_dot = warp_sum(s_dot);
    if (lane == 0) dots[warp] = s_dot;
    __syncthreads();
    // dq += N K,  dk += N^T Q + (B + B^T) K
    warp_gemm<NK>(dq, 0, wr + 16, [&](int m, int k) { return Vn[(wr + m) * TP + k]; },
                  [&](int k, int n) { return K[k * L::KP + 8 * NK * wc + n]; }, g8, t4);
    warp_gemm<NK>(dk, wr, C, [&](int m, int k) { return Vn[k * TP + wr + m]; },
                  [&](int k, int n) { return Q[k * L::KP + 8 * NK * wc + n]; }, g8, t4);
    warp_gemm<NK>(dk, 0, C, [&](int m, int k) { return O[(wr + m) * TP + k] + O[k * TP + wr + m]; },
                  [&](int k, int n) { return K[k * L::KP + 8 * NK * wc + n]; }, g8, t4);
    if (warp == 0) {
      // dgc of rows 2 lane, 2 lane + 1; then the suffix sums
      float d[2], th = 0.f, bsum[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * lane + e;
        const float thr = red[2 * C + r] + red[5 * C + r];
        th += thr;
        d[e] = red[r] + red[3 * C + r] - thr - ((col[r] + col[C + r]) + (col[2 * C + r] + col[3 * C + r]));
        bsum[e] = red[C + r] + red[4 * C + r];
      }
      th = warp_sum(th);
      float dot = lane < 8 ? dots[lane] : 0.f;
      dot = warp_sum(dot);
      if (lane == 31) d[1] += th + eg[C - 1] * dot;
      float suf = d[0] + d[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, suf, o);
        if (lane + o < 32) suf += y;
      }
      float beyond = __shfl_down_sync(0xffffffffu, suf, 1);
      if (lane == 31) beyond = 0.f;
      const float dg[2] = {suf, beyond + d[1]};
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (c0 + 2 * lane + e < end) {
          const size_t at = (size_t)(c0 + 2 * lane + e) * a.nv + h;
          static_cast<IO*>(a.dg)[at] = from_f32<IO>(dg[e]);
          static_cast<IO*>(a.dbeta)[at] = from_f32<IO>(bsum[e]);
        }
    }
  }
  __syncthreads();
  // the norms: d(raw) = (d(hat) - hat (hat . d(hat))) / |raw|
  float dotq[2] = {0.f, 0.f}, dotk[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < NK; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = (r0 + 8 * (e >> 1)) * L::KP + 8 * (NK * wc + j) + 2 * t4 + (e & 1);
      dotq[e >> 1] = fmaf(dq[j][e], Q[at], dotq[e >> 1]);
      dotk[e >> 1] = fmaf(dk[j][e], K[at], dotk[e >> 1]);
    }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      dotq[e] += __shfl_xor_sync(0xffffffffu, dotq[e], o);
      dotk[e] += __shfl_xor_sync(0xffffffffu, dotk[e], o);
    }
    if (t4 == 0) {
      red[(2 * wc) * C + r0 + 8 * e] = dotq[e];
      red[(2 * wc + 1) * C + r0 + 8 * e] = dotk[e];
    }
  }
  __syncthreads();
#pragma unroll
  for (int e2 = 0; e2 < 2; ++e2) {
    const int r = r0 + 8 * e2;
    if (c0 + r >= end) continue;
    const float pq = a.qk_l2norm ? red[r] + red[2 * C + r] : 0.f, pk = a.qk_l2norm ? red[C + r] + red[3 * C + r] : 0.f;
    const size_t at = ((size_t)(c0 + r) * a.nqk + hq) * DK + 8 * NK * wc + 2 * t4;
#pragma unroll
    for (int j = 0; j < NK; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int d = 8 * (NK * wc + j) + 2 * t4 + e;
        static_cast<IO*>(a.dq)[at + 8 * j + e] = from_f32<IO>(nq[r] * (dq[j][2 * e2 + e] - Q[r * L::KP + d] * pq));
        static_cast<IO*>(a.dk)[at + 8 * j + e] = from_f32<IO>(nk[r] * (dk[j][2 * e2 + e] - K[r * L::KP + d] * pk));
      }
  }
}

template <typename F>
static cudaError_t set_smem(F kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int DK, int DV, typename IO>
static cudaError_t launch_one(const BwdArgs& a, cudaStream_t stream) {
  const unsigned int slots = (unsigned int)(a.total_tokens / C + a.num_seqs);
  cudaError_t e;
  if (a.total_tokens > 0) {
    if ((e = set_smem(prepare_kernel<DK, DV, IO>, PrepSmem<DK, DV>::kBytes)) != cudaSuccess) return e;
    prepare_kernel<DK, DV, IO><<<dim3(slots, a.nv), kThreads, PrepSmem<DK, DV>::kBytes, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = set_smem(states_kernel<DK, DV>, StateSmem<DK>::kBytes)) != cudaSuccess) return e;
  states_kernel<DK, DV><<<dim3(2 * DV / (16 * kStateWarps), a.nv, a.num_seqs), kStateThreads, StateSmem<DK>::kBytes, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || a.total_tokens == 0) return e;
  if ((e = set_smem(grads_kernel<DK, DV, IO>, GradSmem<DK>::kBytes)) != cudaSuccess) return e;
  grads_kernel<DK, DV, IO><<<dim3(slots, a.nqk), kThreads, GradSmem<DK>::kBytes, stream>>>(a);
  return cudaGetLastError();
}

template <int DK, int DV>
static cudaError_t launch_io(const BwdArgs& a, int io_bf16, cudaStream_t s) {
  return io_bf16 ? launch_one<DK, DV, __nv_bfloat16>(a, s) : launch_one<DK, DV, float>(a, s);
}

}  // namespace bwd

int64_t chunk_bwd_workspace(int64_t total_tokens, int num_seqs, int nqk, int nv, int dk, int dv) {
  if (total_tokens == 0) return 0;
  const int64_t c = bwd::C, rec = c * (c + dk + 3 * dv + 2) + 2 * (int64_t)dk * dv + dv;
  return (total_tokens / c + num_seqs) * (nv * rec + nqk * 2 * c * dk) * (int64_t)sizeof(float);
}

cudaError_t launch_chunk_bwd(const BwdArgs& a, int dk, int dv, int io_bf16, cudaStream_t s) {
  static_assert(bwd::Rec<128, 64>::kFloats == 64 * (64 + 128 + 3 * 64 + 2) + 2 * 128 * 64 + 64, "workspace size");
  static_assert(bwd::QkRec<128>::kFloats == 2 * 64 * 128, "workspace size");
  if (dk == 64 && dv == 64) return bwd::launch_io<64, 64>(a, io_bf16, s);
  if (dk == 64 && dv == 128) return bwd::launch_io<64, 128>(a, io_bf16, s);
  if (dk == 128 && dv == 64) return bwd::launch_io<128, 64>(a, io_bf16, s);
  if (dk == 128 && dv == 128) return bwd::launch_io<128, 128>(a, io_bf16, s);
  return cudaErrorInvalidValue;
}

}  // namespace gdn
