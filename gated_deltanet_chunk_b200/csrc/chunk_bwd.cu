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
//      the next product's A operand up to a permutation of k, so a chunk is two
//      (or three) chained products without a shared-memory round trip or a
//      block-wide wait.  The two directions need nothing of each other and run
//      in the same launch.
//   3. gradients (every chunk and qk-head at once): the rest.  One block takes
//      all the v-heads that share a qk-head, one after another, so dq and dk
//      are summed in registers, in a fixed order.
// What they pass on is fp32 in the caller's workspace.  Every product is a warp
// TF32 MMA with operands split hi + lo (three MMAs, about 2^-22 per product;
// two where one operand comes straight from bf16, which TF32 holds exactly).
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
  static constexpr size_t kW = kT + C * C;        // [C][DK] W
  static constexpr size_t kU = kW + C * DK;       // [C][DV] U, then V'
  static constexpr size_t kY = kU + C * DV;       // [C][DV] P^T dO, then dV'
  static constexpr size_t kS = kY + C * DV;       // [DV][DK] S^T before the chunk
  static constexpr size_t kD = kS + DV * DK;      // [DV][DK] dS'^T behind the chunk
  static constexpr size_t kKw = kD + DV * DK;     // [C] l_r / |k_r|: raw key row -> written key
  static constexpr size_t kQe = kKw + C;          // [C] s e_r / |q_r|: raw query row -> s diag(e) Q
  static constexpr size_t kGl = kQe + C;          // [1] e_last (padded to C)
  static constexpr size_t kFloats = kGl + C;
};

// Rows [c0, c0 + C) of one head of a [T, heads, D] tensor into a tile of pitch P
// (rows from `end` on as zeros), and the L2-norm factor of every row into
// norm[] when it is not null.  One warp per row, 8 rows in turn per warp.
template <int D, int P, typename IO>
__device__ __forceinline__ void load_rows(const IO* x, int64_t c0, int64_t end, int heads, int head, float* tile,
                                          float* norm, bool l2, int warp, int lane) {
  constexpr int PER = D / 32;
#pragma unroll 4
  for (int r = warp; r < C; r += kThreads / 32) {
    const int64_t tk = c0 + r;
    const bool valid = tk < end;
    const IO* src = x + ((size_t)(valid ? tk : c0) * heads + head) * D;
    float v[PER], ss = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      v[e] = valid ? to_f32(src[lane + 32 * e]) : 0.f;
      ss = fmaf(v[e], v[e], ss);
    }
    float f = 1.f;
    if (norm) {
      ss = warp_sum(ss);
      f = l2 ? 1.f / sqrtf(ss + kNormEps) : 1.f;
      if (lane == 0) norm[r] = f;
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
  static constexpr int kBe = kBeta + C;        // [C] beta e
  static constexpr int kNq = kBe + C;          // [C] 1 / |q|
  static constexpr int kNk = kNq + C;          // [C] 1 / |k|
  static constexpr int kTotal = kNk + C;
  static constexpr size_t kBytes = size_t(kTotal) * sizeof(float);
  static_assert(kBytes <= 232448, "shared memory budget");
};

// One warp's 16 rows (from wr) and column half wc of an [C x 16 NT] product, to dst.
template <int NT, typename FA, typename FB>
__device__ __forceinline__ void product(float* dst, int wr, int wc, int k0, int k1, FA a, FB b, int g, int t) {
  float x[NT][4] = {};
  const int n0 = 8 * NT * wc;
  warp_gemm<NT>(x, k0, k1, a, [&](int k, int n) { return b(k, n0 + n); }, g, t);
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; e += 2)
      *reinterpret_cast<float2*>(dst + (wr + g + 4 * e) * (16 * NT) + n0 + 8 * j + 2 * t) = make_float2(x[j][e], x[j][e + 1]);
}

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
  float* rec = a.ws + ((size_t)slot * a.nv + h) * R::kFloats;

  load_rows<DK, L::KP>(static_cast<const IO*>(a.k), c0, end, a.nqk, hq, K, nk, a.qk_l2norm != 0, warp, lane);
  load_rows<DK, L::KP>(static_cast<const IO*>(a.q), c0, end, a.nqk, hq, Q, nq, a.qk_l2norm != 0, warp, lane);
  load_rows<DV, L::VP>(static_cast<const IO*>(a.v), c0, end, a.nv, h, V, (float*)nullptr, false, warp, lane);
  load_rows<DV, L::VP>(static_cast<const IO*>(a.dout), c0, end, a.nv, h, O, (float*)nullptr, false, warp, lane);
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
    rec[R::kKw + tid] = expf(gc[C - 1] - gc[tid]) * nk[tid];
    rec[R::kQe + tid] = a.scale * e * nq[tid];
    if (tid == C - 1) rec[R::kGl] = e;
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
  // W = T diag(b e) K,  U = T diag(b) V,  Y = P^T dO
  auto fT = [&](int m, int k) { return A[(wr + m) * TP + k]; };
  product<DK / 16>(rec + R::kW, wr, wc, 0, wr + 16, fT, [&](int k, int n) { return be[k] * K[k * L::KP + n]; }, g8, t4);
  product<DV / 16>(rec + R::kU, wr, wc, 0, wr + 16, fT, [&](int k, int n) { return bt[k] * V[k * L::VP + n]; }, g8, t4);
  product<DV / 16>(rec + R::kY, wr, wc, wr, C, [&](int m, int k) { return P[k * TP + wr + m]; },
                   [&](int k, int n) { return O[k * L::VP + n]; }, g8, t4);
}

// ------------------------------------------------------------------ 2. states

constexpr int kStateWarps = 4;  // 64 Dv columns per block
constexpr int kStateThreads = 32 * kStateWarps;

template <typename IO> struct Tile;  // a raw row element as the fp32 it stands for
template <> struct Tile<float> { static constexpr bool exact = false; static constexpr int pad4 = 4, pad8 = 8; };
template <> struct Tile<__nv_bfloat16> { static constexpr bool exact = true; static constexpr int pad4 = 8, pad8 = 8; };

template <int DK, typename IO>
struct StateSmem {
  static constexpr int P4 = DK + 4, P8 = DK + 8;               // pitches of the fp32 W tile (backwards, forwards)
  static constexpr int X4 = DK + Tile<IO>::pad4, X8 = DK + Tile<IO>::pad8;  // of the raw tiles
  static constexpr size_t kW = 0;
  static constexpr size_t kK = kW + sizeof(float) * C * P8;
  static constexpr size_t kQ = kK + sizeof(IO) * C * X8;
  static constexpr size_t kStage = kQ + sizeof(IO) * C * X4;
  static constexpr size_t kBytes = 2 * kStage;
  static_assert(kStage % 16 == 0 && kBytes <= 232448, "shared memory budget");
};

__device__ __forceinline__ void cp16(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(ptx::smem_u32(dst)), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}

// rows of `bytes` (a multiple of 16) from src (pitch spitch) to dst (pitch dpitch), rows from `rows` on as zeros
__device__ __forceinline__ void copy_rows(uint8_t* dst, int dpitch, const uint8_t* src, size_t spitch, int bytes, int rows,
                                          int tid) {
  const int per = bytes / 16;
  for (int i = tid; i < C * per; i += kStateThreads) {
    const int r = i / per, c = (i % per) * 16;
    const bool valid = r < rows;
    cp16(dst + r * dpitch + c, src + (valid ? r : 0) * spitch + c, valid);
  }
}

// A operand of k-step j from accumulators: slot t of k holds column 8 j + 2 t, slot t + 4 column 8 j + 2 t + 1.
__device__ __forceinline__ void frag_of_acc(const float* c, float f0, float f1, uint32_t* ah, uint32_t* al) {
  split_tf32(c[0] * f0, ah[0], al[0]);
  split_tf32(c[2] * f0, ah[1], al[1]);
  split_tf32(c[1] * f1, ah[2], al[2]);
  split_tf32(c[3] * f1, ah[3], al[3]);
}

template <int DK, int DV, typename IO, bool kBackward>
__device__ __forceinline__ void walk(const BwdArgs& a, uint8_t* sm, int n, int h, int col0) {
  using L = StateSmem<DK, IO>;
  using R = Rec<DK, DV>;
  constexpr bool XT = Tile<IO>::exact;
  constexpr int ND = DK / 8, NR = C / 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int c = col0 + 16 * warp + g;  // this thread's columns of Dv: c and c + 8
  const int hq = h / (a.nv / a.nqk);
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

  auto chunk_of = [&](int64_t i) { return kBackward ? chunks - 1 - i : i; };
  auto rec_of = [&](int64_t i) { return a.ws + ((size_t)(slot0 + chunk_of(i)) * a.nv + h) * R::kFloats; };
  auto fetch = [&](int64_t i) {
    if (i < chunks) {
      uint8_t* st = sm + (i & 1) * L::kStage;
      const int64_t c0 = start + chunk_of(i) * C;
      const int rows = (int)min((int64_t)C, end - c0);
      copy_rows(st + L::kW, 4 * (kBackward ? L::P4 : L::P8), reinterpret_cast<const uint8_t*>(rec_of(i) + R::kW), 4 * DK,
                4 * DK, C, tid);
      const size_t off = ((size_t)c0 * a.nqk + hq) * DK, pitch = (size_t)a.nqk * DK * sizeof(IO);
      copy_rows(st + L::kK, (int)sizeof(IO) * (kBackward ? L::X8 : L::X4),
                reinterpret_cast<const uint8_t*>(static_cast<const IO*>(a.k) + off), pitch, DK * sizeof(IO), rows, tid);
      if (kBackward)
        copy_rows(st + L::kQ, (int)sizeof(IO) * L::X4, reinterpret_cast<const uint8_t*>(static_cast<const IO*>(a.q) + off),
                  pitch, DK * sizeof(IO), rows, tid);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
  fetch(0);
  for (int64_t i = 0; i < chunks; ++i) {
    float* rec = rec_of(i);
    // U^T or Y^T of this chunk: rows c, c + 8, columns r = 8 j + 2 t, + 1
    float* uv = rec + (kBackward ? R::kY : R::kU) + c;
    float u[NR][4];
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) u[j][e] = uv[(size_t)(8 * j + 2 * t + (e & 1)) * DV + 8 * (e >> 1)];
    fetch(i + 1);
    // the state as this chunk meets it, for the gradients
    float* sv = rec + (kBackward ? R::kD : R::kS) + (size_t)c * DK + 2 * t;
#pragma unroll
    for (int j = 0; j < ND; ++j) {
      *reinterpret_cast<float2*>(sv + 8 * j) = make_float2(s[j][0], s[j][1]);
      *reinterpret_cast<float2*>(sv + 8 * DK + 8 * j) = make_float2(s[j][2], s[j][3]);
    }
    const float gl = rec[R::kGl];
    asm volatile("cp.async.wait_group 1;\n" ::: "memory");
    __syncthreads();
    const uint8_t* st = sm + (i & 1) * L::kStage;
    const float* W = reinterpret_cast<const float*>(st + L::kW);
    const IO* K = reinterpret_cast<const IO*>(st + L::kK);
    const IO* Q = reinterpret_cast<const IO*>(st + L::kQ);
    // x = S^T W^T (forwards) or dS'^T K^T (backwards), [16 x C]
    float x[NR][4] = {};
#pragma unroll
    for (int j = 0; j < ND; ++j) {
      uint32_t ah[4], al[4];
      frag_of_acc(s[j], 1.f, 1.f, ah, al);
#pragma unroll
      for (int m = 0; m < NR; ++m) {
        uint32_t bh[2], bl[2];
        float b0, b1;
        if (kBackward) {
          b0 = to_f32(K[(8 * m + g) * L::X8 + 8 * j + 2 * t]);
          b1 = to_f32(K[(8 * m + g) * L::X8 + 8 * j + 2 * t + 1]);
        } else {
          const float2 w = *reinterpret_cast<const float2*>(W + (8 * m + g) * L::P8 + 8 * j + 2 * t);
          b0 = w.x;
          b1 = w.y;
        }
        split_tf32(b0, bh[0], bl[0]);
        split_tf32(b1, bh[1], bl[1]);
        mma3<false, kBackward && XT>(x[m], ah, al, bh, bl);
      }
    }
    // forwards V'^T = U^T - x, backwards dV'^T = Y^T + x diag(kw); stored over U, Y
    const float* kw = rec + R::kKw + 2 * t;
    const float* qe = rec + R::kQe + 2 * t;
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[j][e] = kBackward ? fmaf(x[j][e], kw[8 * j + (e & 1)], u[j][e]) : u[j][e] - x[j][e];
        uv[(size_t)(8 * j + 2 * t + (e & 1)) * DV + 8 * (e >> 1)] = x[j][e];
      }
#pragma unroll
    for (int j = 0; j < ND; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] *= gl;
    // forwards S^T += (V' diag(kw))^T K, backwards dS^T += (dO diag(qe))^T Q - dV'^T W
    const int64_t c0 = start + chunk_of(i) * C;
    const IO* dout = static_cast<const IO*>(a.dout) + ((size_t)c0 * a.nv + h) * DV + c;
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      uint32_t ah[4], al[4], oh[4], ol[4];
      if (kBackward) {
        frag_of_acc(x[j], -1.f, -1.f, ah, al);
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t r = 8 * j + 2 * t + (e & 1);
          o[e] = c0 + r < end ? to_f32(dout[(size_t)r * a.nv * DV + 8 * (e >> 1)]) : 0.f;
        }
        frag_of_acc(o, qe[8 * j], qe[8 * j + 1], oh, ol);
      } else {
        frag_of_acc(x[j], kw[8 * j], kw[8 * j + 1], ah, al);
      }
#pragma unroll
      for (int m = 0; m < ND; ++m) {
        uint32_t bh[2], bl[2];
        if (kBackward) {
          split_tf32(W[(8 * j + 2 * t) * L::P4 + 8 * m + g], bh[0], bl[0]);
          split_tf32(W[(8 * j + 2 * t + 1) * L::P4 + 8 * m + g], bh[1], bl[1]);
          mma3<false, false>(s[m], ah, al, bh, bl);
          split_tf32(to_f32(Q[(8 * j + 2 * t) * L::X4 + 8 * m + g]), bh[0], bl[0]);
          split_tf32(to_f32(Q[(8 * j + 2 * t + 1) * L::X4 + 8 * m + g]), bh[1], bl[1]);
          mma3<false, XT>(s[m], oh, ol, bh, bl);
        } else {
          split_tf32(to_f32(K[(8 * j + 2 * t) * L::X4 + 8 * m + g]), bh[0], bl[0]);
          split_tf32(to_f32(K[(8 * j + 2 * t + 1) * L::X4 + 8 * m + g]), bh[1], bl[1]);
          mma3<false, XT>(s[m], ah, al, bh, bl);
        }
      }
    }
    __syncthreads();  // the stage is free for the fetch after next
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
template <int DK, int DV, typename IO>
__global__ void __launch_bounds__(kStateThreads) states_kernel(BwdArgs a) {
  extern __shared__ __align__(16) uint8_t smb[];
  const int col0 = 16 * kStateWarps * (blockIdx.x >> 1);
  if (blockIdx.x & 1)
    walk<DK, DV, IO, true>(a, smb, blockIdx.z, blockIdx.y, col0);
  else
    walk<DK, DV, IO, false>(a, smb, blockIdx.z, blockIdx.y, col0);
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
  static constexpr int kVn = kS + 64 * SP;      // [C][TP] V' columns, then N
  static constexpr int kO = kVn + C * TP;       // [C][TP] dO columns, then B
  static constexpr int kX = kO + C * TP;        // [C][TP] dV' columns, then dX
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

// x = D[C x 64] S[64 x Dk] (rows wr .., column half wc): sum += f x by rows, dot = x . Y by rows (this thread's part).
template <int NK, int KP, int SP>
__device__ __forceinline__ void with_state(const float* D, const float* S, const float* Y, int wr, int wc, const float (&f)[2],
                                           float (&sum)[NK][4], float (&dot)[2], int g, int t) {
  float x[NK][4] = {};
  const int n0 = 8 * NK * wc;
  warp_gemm<NK>(x, 0, 64, [&](int m, int k) { return D[(wr + m) * TP + k]; },
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

  load_rows<DK, L::KP>(static_cast<const IO*>(a.k), c0, end, a.nqk, hq, K, nk, a.qk_l2norm != 0, warp, lane);
  load_rows<DK, L::KP>(static_cast<const IO*>(a.q), c0, end, a.nqk, hq, Q, nq, a.qk_l2norm != 0, warp, lane);
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
    const float* rec = a.ws + ((size_t)slot * a.nv + h) * R::kFloats;
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
        Vn[r * TP + cc] = rec[R::kU + (size_t)r * DV + v0 + cc];
        X[r * TP + cc] = rec[R::kY + (size_t)r * DV + v0 + cc];
        O[r * TP + cc] = c0 + r < end ? to_f32(static_cast<const IO*>(a.dout)[((size_t)(c0 + r) * a.nv + h) * DV + v0 + cc]) : 0.f;
      }
      for (int i = tid; i < 64 * DK; i += kThreads) S[(i / DK) * L::SP + i % DK] = rec[R::kS + (size_t)v0 * DK + i];
      __syncthreads();
      {  // dX = T^T dV'; dV = diag(b) dX
        float x[4][4] = {};
        warp_gemm<4>(x, wr, C, [&](int m, int k) { return T[k * TP + wr + m]; },
                     [&](int k, int n) { return X[k * TP + 32 * wc + n]; }, g8, t4);
        __syncthreads();  // dV' is consumed
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = r0 + 8 * (e >> 1), cc = 32 * wc + 8 * j + 2 * t4 + (e & 1);
            X[r * TP + cc] = x[j][e];
            if (c0 + r < end) {
              const size_t at = ((size_t)(c0 + r) * a.nv + h) * DV + v0 + cc;
              s_bt[e >> 1] = fmaf(x[j][e], to_f32(static_cast<const IO*>(a.v)[at]), s_bt[e >> 1]);
              static_cast<IO*>(a.dv_out)[at] = from_f32<IO>(bt[r] * x[j][e]);
            }
          }
        __syncthreads();
      }
      if (low) {
        warp_gemm<4>(dA, 0, 64, [&](int m, int k) { return X[(wr + m) * TP + k]; },
                     [&](int k, int n) { return Vn[(32 * wc + n) * TP + k]; }, g8, t4);
        warp_gemm<4>(dP, 0, 64, [&](int m, int k) { return O[(wr + m) * TP + k]; },
                     [&](int k, int n) { return Vn[(32 * wc + n) * TP + k]; }, g8, t4);
      }
      // the products with the state: their row dots with q_hat or k_hat, and their shares of dq, dk
      float f[2], dot[2];
      f[0] = a.scale * eg[r0];
      f[1] = a.scale * eg[r0 + 8];
      with_state<NK, L::KP, L::SP>(O, S, Q, wr, wc, f, dq, dot, g8, t4);
#pragma unroll
      for (int e = 0; e < 2; ++e) s_gc[e] = fmaf(f[e], dot[e], s_gc[e]);
      f[0] = -bt[r0] * eg[r0];
      f[1] = -bt[r0 + 8] * eg[r0 + 8];
      with_state<NK, L::KP, L::SP>(X, S, K, wr, wc, f, dk, dot, g8, t4);
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
      with_state<NK, L::KP, L::SP>(Vn, S, K, wr, wc, f, dk, dot, g8, t4);
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
  if ((e = set_smem(states_kernel<DK, DV, IO>, StateSmem<DK, IO>::kBytes)) != cudaSuccess) return e;
  states_kernel<DK, DV, IO><<<dim3(2 * DV / (16 * kStateWarps), a.nv, a.num_seqs), kStateThreads, StateSmem<DK, IO>::kBytes,
                              stream>>>(a);
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

int64_t chunk_bwd_workspace(int64_t total_tokens, int num_seqs, int nv, int dk, int dv) {
  const int64_t rec = bwd::C * (bwd::C + dk + 2 * dv + 3) + 2 * (int64_t)dk * dv;
  return total_tokens == 0 ? 0 : (total_tokens / bwd::C + num_seqs) * nv * rec * (int64_t)sizeof(float);
}

cudaError_t launch_chunk_bwd(const BwdArgs& a, int dk, int dv, int io_bf16, cudaStream_t s) {
  static_assert(bwd::Rec<128, 64>::kFloats == bwd::C * (bwd::C + 128 + 2 * 64 + 3) + 2 * 128 * 64, "workspace size");
  if (dk == 64 && dv == 64) return bwd::launch_io<64, 64>(a, io_bf16, s);
  if (dk == 64 && dv == 128) return bwd::launch_io<64, 128>(a, io_bf16, s);
  if (dk == 128 && dv == 64) return bwd::launch_io<128, 64>(a, io_bf16, s);
  if (dk == 128 && dv == 128) return bwd::launch_io<128, 128>(a, io_bf16, s);
  return cudaErrorInvalidValue;
}

}  // namespace gdn
