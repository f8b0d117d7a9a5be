// chunk_bwd_half.cu -- gradients of the chunked gated delta rule for bf16 tensors.
//
// The mathematics, the notation and the three kernels are those of chunk_bwd.cu.
// Here every product is one warp MMA in fp16 (mma.sync.m16n8k16, fp32
// accumulation): an operand is an fp16 number (11 significant bits) times a power
// of two that its tile, row or column shares, chosen so that the largest
// magnitude is in [2^7, 2^8) or bounded by it.  So
//   - q, k, v and dout, which have 8 significant bits, are exact,
//   - what is formed on the way (T, W, S, V', dS', ...) is rounded by at most
//     2^-12 of its value, or 2^-33 of its tile's largest: an eighth of the bf16
//     rounding that the outputs get, at the cost of one MMA, where bf16 operands
//     of that accuracy would need two or three,
//   - 2^8 against fp16's 65504 leaves room for what follows from a bounded sum.
// The recurrences themselves (S and dS), the cumsums, the inverse, the decays and
// every sum are fp32.
//
// Bounds that the fixed factors of two use (they hold for 0 <= beta <= 2, g <= 0
// and normalised q, k; the prepare kernel checks the gates, and other calls take
// chunk_bwd.cu): decays are at most 1, |T| <= 2 (row r of T is beta_r k_r^T times
// a product of contractions, times k_i), |W| <= 2, |q_r . k_i| <= 1.
#include <cuda_fp16.h>

#include <type_traits>

#include "chunk_bwd.cuh"
#include "gdn_common.cuh"
#include "gdn_launch.h"
#include "sm100_ptx.cuh"

namespace gdn {
namespace bwdh {

using bwd::C;
using bwd::TP;
using bf16 = __nv_bfloat16;

constexpr int HP = C + 8;  // pitch of [..][64] fp16 tiles: rows 16 bytes apart in the banks, as ldmatrix wants

// Workspace record of one (chunk slot, v-head), in bytes.
template <int DK, int DV>
struct Rec {
  static constexpr size_t kT = 0;                      // fp16 [C][C] T 2^7
  static constexpr size_t kW = kT + 2 * C * C;         // fp16 [C][DK] W 2^7
  static constexpr size_t kU = kW + 2 * C * DK;        // fp16 U^T fragments, then V'^T [DV][C]
  static constexpr size_t kY = kU + 2 * C * DV;        // fp16 (P^T dO)^T fragments, then dV'^T [DV][C]
  static constexpr size_t kO = kY + 2 * C * DV;        // fp16 (diag(qe) dO)^T fragments
  static constexpr size_t kS = kO + 2 * C * DV;        // fp16 [DV][DK] S^T before the chunk, columns by swap32
  static constexpr size_t kD = kS + 2 * DK * DV;       // fp16 [DV][DK] dS'^T behind the chunk, the same
  static constexpr size_t kF = kD + 2 * DK * DV;       // floats from here:
  static constexpr int fGc = 0;                        // [C] gcum
  static constexpr int fBeta = fGc + C;                // [C] beta
  static constexpr int fScal = fBeta + C;              // [8] see Scal
  static constexpr int fS = fScal + 8;                 // [DV] factor of every row of S^T
  static constexpr int fD = fS + DV;                   // [DV] of dS'^T
  static constexpr int fV = fD + DV;                   // [DV] of V'^T
  static constexpr int fDV = fV + DV;                  // [DV] of dV'^T
  static constexpr int fKw = fDV + DV;                 // [C] l_r / |k_r| in units of K16
  static constexpr int kFloats = fKw + C;
  static constexpr size_t kBytes = kF + 4 * kFloats;
  static_assert(kBytes % 16 == 0 && fScal % 4 == 0, "16-byte copies");
};
enum Scal { kScalU, kScalY, kScalO, kScalGl, kScalDo };  // factors of U, Y, diag(qe) dO; e_last; factor of dO

// Workspace record of one (chunk slot, qk-head), in bytes.
template <int DK>
struct QkRec {
  static constexpr size_t kK = 0;                 // fp16 [C][DK] K16
  static constexpr size_t kQ = kK + 2 * C * DK;   // fp16 [C][DK] Q16
  static constexpr size_t kF = kQ + 2 * C * DK;   // floats [4][C]: k_hat = kf K16, q_hat = qf Q16, and kf |k|, qf |q| inverted
  static constexpr size_t kBytes = kF + 16 * C;
};

template <int DK, int DV>
__host__ __device__ inline int64_t slots_of(const BwdArgs& a) { return a.total_tokens / C + a.num_seqs; }
template <int DK, int DV>
__device__ __forceinline__ uint8_t* rec_at(const BwdArgs& a, int64_t slot, int h) {
  return reinterpret_cast<uint8_t*>(a.ws) + ((size_t)slot * a.nv + h) * Rec<DK, DV>::kBytes;
}
template <int DK, int DV>
__device__ __forceinline__ uint8_t* qk_at(const BwdArgs& a, int64_t slot, int hq) {
  return reinterpret_cast<uint8_t*>(a.ws) + (size_t)slots_of<DK, DV>(a) * a.nv * Rec<DK, DV>::kBytes +
         ((size_t)slot * a.nqk + hq) * QkRec<DK>::kBytes;
}

// ------------------------------------------------------------------ fragments
// With g = lane / 4, t = lane % 4: A a0 (g, 2t..), a1 (g + 8, 2t..), a2 (g, 2t + 8..), a3 (g + 8, 2t + 8..),
// B b0 (k 2t.., n g), b1 (k 2t + 8.., n g), accumulators as those of m16n8k8.
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, const uint32_t* b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void ldsm(uint32_t* r, const __half* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(ptx::smem_u32(p))
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t* r, const __half* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(ptx::smem_u32(p))
               : "memory");
}
// A (16 x 16 at row m0, k0) of a tile [m][k], or [k][m] (_t); B (16 k x 16 n: two 8-column tiles) of a
// tile [n][k], or [k][n] (_t).  P: the tile's pitch.
template <int P> __device__ __forceinline__ void frag_a(uint32_t* r, const __half* tile, int m0, int k0, int lane) {
  ldsm(r, tile + (m0 + (lane & 15)) * P + k0 + 8 * (lane >> 4));
}
template <int P> __device__ __forceinline__ void frag_a_t(uint32_t* r, const __half* tile, int m0, int k0, int lane) {
  ldsm_t(r, tile + (k0 + (lane & 7) + 8 * (lane >> 4)) * P + m0 + 8 * ((lane >> 3) & 1));
}
template <int P> __device__ __forceinline__ void frag_b(uint32_t* r, const __half* tile, int n0, int k0, int lane) {
  ldsm(r, tile + (n0 + (lane & 7) + 8 * (lane >> 4)) * P + k0 + 8 * ((lane >> 3) & 1));
}
template <int P> __device__ __forceinline__ void frag_b_t(uint32_t* r, const __half* tile, int n0, int k0, int lane) {
  ldsm_t(r, tile + (k0 + (lane & 15)) * P + n0 + 8 * (lane >> 4));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// f = 2^k with top f in [2^7, 2^8), and 1 / f.  Magnitudes below 2^-119 count as 2^-119; an infinite or
// NaN `top` gives a finite factor, so such values stay what they are.
__device__ __forceinline__ void pow2_factor(float top, float& f, float& inv) {
  const uint32_t e = max((__float_as_uint(top) >> 23) & 255u, 8u);
  f = __uint_as_float((261u - e) << 23);
  inv = __uint_as_float((e - 7u) << 23);
}

__device__ __forceinline__ void cp16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16_or_zero(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(ptx::smem_u32(dst)), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

// ------------------------------------------------------------------ 1. prepare
// One block per (slot, qk-head): K16, Q16 and their products once, then its v-heads in turn.

constexpr int kPrepThreads = 256;

template <int DK, int DV>
struct PrepSmem {
  static constexpr int DP = DK + 8, VP = DV + 8;
  static constexpr size_t kK = 0;                                       // fp16 [C][DP] K16
  static constexpr size_t kQ = kK + 2 * C * DP;                         // fp16 [C][DP] Q16, then T beta 2^6 and P 2^8, [C][HP] each
  static constexpr size_t kQBytes = 2 * C * DP > 4 * C * HP ? 2 * C * DP : 4 * C * HP;
  static constexpr size_t kV = kQ + kQBytes;                            // fp16 [C][VP] V
  static constexpr size_t kO = kV + 2 * C * VP;                         // fp16 [C][VP] dO
  static constexpr size_t kA = kO + 2 * C * VP;                         // fp32 [C][TP] A, then T
  static constexpr size_t kY = kA + 4 * C * TP;                         // fp32 [C / 2][TP] scratch of the inverse
  static constexpr size_t kF = kY + 2 * C * TP;                         // fp32 [C] each: gc, beta, kf, qf, T's column factors of W
  static constexpr size_t kQe = kF + 20 * C;                            // fp16 [C] e qf 2^7 (at most 1)
  static constexpr size_t kTop = kQe + 2 * C;                           // fp32 [2][8] largest |v|, |dO| by warp
  static constexpr size_t kBytes = kTop + 64;
  static_assert(kBytes <= 113 * 1024, "two blocks per SM");
};

// Rows of q or k: to fp16 with a factor of two for each row, into a tile (pitch DK + 8) and the workspace,
// and the factors.  DK / 8 lanes per row.  Rows so small that the norm's eps decides are scaled by 2^17, so
// that kf and qf stay within a few powers of two of one another.
template <int DK>
__device__ __forceinline__ void load_qk(const bf16* x, int64_t c0, int64_t end, int heads, int head, __half* tile, __half* ws,
                                        float* f, float* wf, float* wn, int tid) {
  constexpr int L = DK / 8, R = kPrepThreads / L;
  const int lr = tid % L;
#pragma unroll
  for (int p = 0; p < C / R; ++p) {
    const int r = p * R + tid / L;
    const bool valid = c0 + r < end;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (valid) w = *reinterpret_cast<const uint4*>(x + ((size_t)(c0 + r) * heads + head) * DK + 8 * lr);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    float2 v[4];
    float ss = 0.f, top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = bf2(u[i]);
      ss = fmaf(v[i].x, v[i].x, fmaf(v[i].y, v[i].y, ss));
      top = fmaxf(top, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    float s, inv;
    pow2_factor(fmaxf(top, 0x1p-10f), s, inv);
    uint4 h;
    h.x = pack2(v[0].x * s, v[0].y * s);
    h.y = pack2(v[1].x * s, v[1].y * s);
    h.z = pack2(v[2].x * s, v[2].y * s);
    h.w = pack2(v[3].x * s, v[3].y * s);
    *reinterpret_cast<uint4*>(tile + r * (DK + 8) + 8 * lr) = h;
    *reinterpret_cast<uint4*>(ws + r * DK + 8 * lr) = h;
    if (lr == 0) {
      f[r] = inv / sqrtf(ss + kNormEps);
      wf[r] = f[r];
      wn[r] = s;
    }
  }
}

// [C x DV] of v or dout for this thread: NV vectors of 8, vector i at row i R + tid / L
template <int DV>
__device__ __forceinline__ void load_v(const bf16* x, int64_t c0, int64_t end, int nv, int h, uint4 (&w)[C * DV / 8 / kPrepThreads],
                                       float& top, int tid) {
  constexpr int L = DV / 8, R = kPrepThreads / L;
  top = 0.f;
#pragma unroll
  for (int p = 0; p < C / R; ++p) {
    const int r = p * R + tid / L;
    w[p] = make_uint4(0u, 0u, 0u, 0u);
    if (c0 + r < end) w[p] = *reinterpret_cast<const uint4*>(x + ((size_t)(c0 + r) * nv + h) * DV + 8 * (tid % L));
    const uint32_t u[4] = {w[p].x, w[p].y, w[p].z, w[p].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = bf2(u[i]);
      top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
}
template <int DV>
__device__ __forceinline__ void store_v(const uint4 (&w)[C * DV / 8 / kPrepThreads], float s, __half* tile, int tid) {
  constexpr int L = DV / 8, R = kPrepThreads / L;
#pragma unroll
  for (int p = 0; p < C / R; ++p) {
    const uint32_t u[4] = {w[p].x, w[p].y, w[p].z, w[p].w};
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = bf2(u[i]);
      h[i] = pack2(v.x * s, v.y * s);
    }
    *reinterpret_cast<uint4*>(tile + (p * R + tid / L) * (DV + 8) + 8 * (tid % L)) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// A warp's accumulators of 16 rows and 64 columns, times f, as the fragments of A operands
__device__ __forceinline__ void store_frags(uint4* dst, const float (&x)[8][4], float f) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    dst[32 * j] = make_uint4(pack2(x[2 * j][0] * f, x[2 * j][1] * f), pack2(x[2 * j][2] * f, x[2 * j][3] * f),
                             pack2(x[2 * j + 1][0] * f, x[2 * j + 1][1] * f), pack2(x[2 * j + 1][2] * f, x[2 * j + 1][3] * f));
}

template <int DK, int DV>
__global__ void __launch_bounds__(kPrepThreads, 2) prepare_half_kernel(BwdArgs a) {
  using L = PrepSmem<DK, DV>;
  using R = Rec<DK, DV>;
  using QR = QkRec<DK>;
  extern __shared__ __align__(16) uint8_t sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
  const int hq = blockIdx.y, group = a.nv / a.nqk;
  const int64_t slot = blockIdx.x;
  int64_t c0, end;
  if (!bwd::chunk_at(a, slot, c0, end)) return;
  __half *K = reinterpret_cast<__half*>(sm + L::kK), *Q = reinterpret_cast<__half*>(sm + L::kQ);
  __half *TB = Q, *P = Q + C * HP, *V = reinterpret_cast<__half*>(sm + L::kV), *O = reinterpret_cast<__half*>(sm + L::kO);
  float *A = reinterpret_cast<float*>(sm + L::kA), *Y = reinterpret_cast<float*>(sm + L::kY);
  float *gc = reinterpret_cast<float*>(sm + L::kF), *bt = gc + C, *kf = bt + C, *qf = kf + C, *wf = qf + C;
  __half* qe = reinterpret_cast<__half*>(sm + L::kQe);
  float* tops = reinterpret_cast<float*>(sm + L::kTop);
  uint8_t* qrec = qk_at<DK, DV>(a, slot, hq);
  float* qfl = reinterpret_cast<float*>(qrec + QR::kF);

  load_qk<DK>(static_cast<const bf16*>(a.k), c0, end, a.nqk, hq, K, reinterpret_cast<__half*>(qrec + QR::kK), kf, qfl, qfl + 2 * C, tid);
  load_qk<DK>(static_cast<const bf16*>(a.q), c0, end, a.nqk, hq, Q, reinterpret_cast<__half*>(qrec + QR::kQ), qf, qfl + C, qfl + 3 * C, tid);
  __syncthreads();
  // warp: rows 16 wr .., columns 32 wc .. of the [C][C] products; blocks above the diagonal are not formed
  const int wr = 16 * (warp & 3), wc = 32 * (warp >> 2), r0 = wr + g8;
  const bool low = wc < wr + 16;
  float kk[4][4] = {}, qk[4][4] = {};
  if (low) {
#pragma unroll
    for (int k = 0; k < DK; k += 16) {
      uint32_t ak[4], aq[4], b[8];
      frag_a<L::DP>(ak, K, wr, k, lane);
      frag_a<L::DP>(aq, Q, wr, k, lane);
      frag_b<L::DP>(b, K, wc, k, lane);
      frag_b<L::DP>(b + 4, K, wc + 16, k, lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mma_f16(kk[j], ak, b + 2 * j);
        mma_f16(qk[j], aq, b + 2 * j);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = kf[wc + 8 * j + 2 * t4 + (e & 1)];
        kk[j][e] *= kf[r0 + 8 * (e >> 1)] * f;
        qk[j][e] *= qf[r0 + 8 * (e >> 1)] * f;
      }
  }

  for (int h = hq * group; h < (hq + 1) * group; ++h) {
    uint8_t* rec = rec_at<DK, DV>(a, slot, h);
    float* rf = reinterpret_cast<float*>(rec + R::kF);
    uint4 vw[C * DV / 8 / kPrepThreads], ow[C * DV / 8 / kPrepThreads];
    float vtop, otop;
    load_v<DV>(static_cast<const bf16*>(a.v), c0, end, a.nv, h, vw, vtop, tid);
    load_v<DV>(static_cast<const bf16*>(a.dout), c0, end, a.nv, h, ow, otop, tid);
    float gv = 0.f, bv = 0.f;
    if (tid < C && c0 + tid < end) {
      load_gate(a, (size_t)(c0 + tid) * a.nv + h, h, gv, bv);
      if (!(gv <= 0.f) || !(bv >= 0.f && bv <= 2.f)) report_status(a.status, kStatusGate);
    }
    __syncthreads();  // the head before is done with the tiles
    if (lane == 0) {
      tops[warp] = vtop;
      tops[8 + warp] = otop;
    }
    if (tid < C) {
      gc[tid] = gv;
      bt[tid] = bv;
    }
    __syncthreads();
    if (warp == 0) bwd::cumsum_chunk(gc, lane);
    vtop = otop = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      vtop = fmaxf(vtop, tops[i]);
      otop = fmaxf(otop, tops[8 + i]);
    }
    float vs, vinv, os, oinv;
    pow2_factor(vtop, vs, vinv);
    pow2_factor(otop, os, oinv);
    store_v<DV>(vw, vs, V, tid);
    store_v<DV>(ow, os, O, tid);
    __syncthreads();
    if (tid < C) {
      const float e = expf(gc[tid]);
      // 2^7 kf <= 1 (kf is at most 2^-7: the largest element of a row is at most its norm)
      wf[tid] = bt[tid] * e * kf[tid] * 0x1p13f;
      qe[tid] = __float2half_rn(e * qf[tid] * 0x1p7f);
      rf[R::fGc + tid] = gc[tid];
      rf[R::fBeta + tid] = bt[tid];
      rf[R::fKw + tid] = expf(gc[C - 1] - gc[tid]) * kf[tid];
      if (tid == C - 1) {
        rf[R::fScal + kScalU] = 2.f * vinv;
        rf[R::fScal + kScalY] = a.scale * oinv;
        rf[R::fScal + kScalO] = a.scale * oinv * 0x1p-7f;
        rf[R::fScal + kScalGl] = e;
        rf[R::fScal + kScalDo] = oinv;
      }
    }
    float p[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + 8 * (e >> 1), i = wc + 8 * j + 2 * t4 + (e & 1);
        const float gamma = i <= r ? ptx::ex2_approx(1.44269504f * (gc[r] - gc[i])) : 0.f;  // masked before exp
        A[r * TP + i] = i < r ? -bt[r] * (kk[j][e] * gamma) : 0.f;
        p[j][e] = qk[j][e] * gamma * 0x1p8f;
      }
    __syncthreads();
    bwd::invert_chunk<false>(A, Y, warp, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int r = r0 + 4 * e, i = wc + 8 * j + 2 * t4;
        const float2 t = *reinterpret_cast<const float2*>(A + r * TP + i);
        *reinterpret_cast<uint32_t*>(P + r * HP + i) = pack2(p[j][e], p[j][e + 1]);
        *reinterpret_cast<uint32_t*>(TB + r * HP + i) = pack2(t.x * bt[i] * 0x1p6f, t.y * bt[i + 1] * 0x1p6f);
        *reinterpret_cast<uint32_t*>(rec + R::kT + 2 * (r * C + i)) = pack2(t.x * 0x1p7f, t.y * 0x1p7f);
      }
    __syncthreads();
    {  // W 2^7 = (T diag(b e kf) 2^13) K16 2^-6: this warp's 16 rows, one half of the columns
      constexpr int NT = DK / 16;
      float x[NT][4] = {};
      const int n0 = (DK / 2) * (warp >> 2);
#pragma unroll
      for (int k = 0; k < C; k += 16) {  // T's zeros above the diagonal are multiplied too: a branch would cost more
        uint32_t af[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + 8 * (e & 1), i = k + 8 * (e >> 1) + 2 * t4;
          const float2 t = *reinterpret_cast<const float2*>(A + r * TP + i);
          af[e] = pack2(t.x * wf[i], t.y * wf[i + 1]);
        }
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          uint32_t b[4];
          frag_b_t<L::DP>(b, K, n0 + 8 * j, k, lane);
          mma_f16(x[j], af, b);
          mma_f16(x[j + 1], af, b + 2);
        }
      }
      __half* w = reinterpret_cast<__half*>(rec + R::kW) + (size_t)r0 * DK + n0 + 2 * t4;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; e += 2)
          *reinterpret_cast<uint32_t*>(w + 4 * e * DK + 8 * j) = pack2(x[j][e] * 0x1p-6f, x[j][e + 1] * 0x1p-6f);
    }
    // U^T = V^T (T diag(b))^T and Y^T = dO^T P, 16 columns of Dv a unit, and the fragments of (diag(qe) dO)^T
    for (int u = warp; u < DV / 16; u += kPrepThreads / 32) {
      float x[8][4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t af[4];
        frag_a_t<L::VP>(af, V, 16 * u, 16 * k, lane);
#pragma unroll
        for (int j = k; j < 4; ++j) {  // the blocks of the triangle
          uint32_t b[4];
          frag_b<HP>(b, TB, 16 * j, 16 * k, lane);
          mma_f16(x[2 * j], af, b);
          mma_f16(x[2 * j + 1], af, b + 2);
        }
      }
      store_frags(reinterpret_cast<uint4*>(rec + R::kU) + u * 128 + lane, x, 0x1p-7f);
    }
    for (int u = kPrepThreads / 32 - 1 - warp; u < DV / 16; u += kPrepThreads / 32) {
      float x[8][4] = {};
      uint4* dst = reinterpret_cast<uint4*>(rec + R::kO) + u * 128 + lane;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t af[4];
        frag_a_t<L::VP>(af, O, 16 * u, 16 * k, lane);
#pragma unroll
        for (int j = 0; j <= k; ++j) {
          uint32_t b[4];
          frag_b_t<HP>(b, P, 16 * j, 16 * k, lane);
          mma_f16(x[2 * j], af, b);
          mma_f16(x[2 * j + 1], af, b + 2);
        }
        const uint32_t lo = *reinterpret_cast<const uint32_t*>(qe + 16 * k + 2 * t4), hi = *reinterpret_cast<const uint32_t*>(qe + 16 * k + 8 + 2 * t4);
        dst[32 * k] = make_uint4(mul2(af[0], lo), mul2(af[1], lo), mul2(af[2], hi), mul2(af[3], hi));
      }
      store_frags(reinterpret_cast<uint4*>(rec + R::kY) + u * 128 + lane, x, 0x1p-8f);
    }
  }
}

// ------------------------------------------------------------------ 2. states

constexpr int kStateWarps = 4;  // 64 Dv columns per block
constexpr int kStateThreads = 32 * kStateWarps;

template <int DK>
struct StateSmem {
  static constexpr int DP = DK + 8;
  static constexpr size_t kW = 0;                       // fp16 [C][DP] W
  static constexpr size_t kK = kW + 2 * C * DP;         // fp16 [C][DP] K16
  static constexpr size_t kQ = kK + 2 * C * DP;         // fp16 [C][DP] Q16 (backwards)
  static constexpr size_t kKw = kQ + 2 * C * DP;        // fp32 [C]
  static constexpr size_t kStage = kKw + 4 * C;
  static constexpr size_t kBytes = 2 * kStage;
  static_assert(kBytes <= 113 * 1024, "two blocks per SM");
};

// Rows c, c + 8 of an accumulator [NT] (16 x 8 tiles) as fp16 with a factor of two for each row:
// the A fragments of the next product, and 1 / factor.
template <int NT>
__device__ __forceinline__ void scale_rows(const float (&s)[NT][4], uint32_t (&f)[NT / 2][4], float (&inv)[2]) {
  float top[2] = {0.f, 0.f}, fac[2];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    top[0] = fmaxf(top[0], fmaxf(fabsf(s[j][0]), fabsf(s[j][1])));
    top[1] = fmaxf(top[1], fmaxf(fabsf(s[j][2]), fabsf(s[j][3])));
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
    top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
    pow2_factor(top[e], fac[e], inv[e]);
  }
#pragma unroll
  for (int j = 0; j < NT / 2; ++j) {
    f[j][0] = pack2(s[2 * j][0] * fac[0], s[2 * j][1] * fac[0]);
    f[j][1] = pack2(s[2 * j][2] * fac[1], s[2 * j][3] * fac[1]);
    f[j][2] = pack2(s[2 * j + 1][0] * fac[0], s[2 * j + 1][1] * fac[0]);
    f[j][3] = pack2(s[2 * j + 1][2] * fac[1], s[2 * j + 1][3] * fac[1]);
  }
}

template <int DK, int DV, bool kBackward>
__device__ __forceinline__ void walk(const BwdArgs& a, uint8_t* sm, int n, int h, int col0) {
  using L = StateSmem<DK>;
  using R = Rec<DK, DV>;
  using QR = QkRec<DK>;
  constexpr int ND = DK / 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int slice = col0 / 16 + warp, c = 16 * slice + g;  // this thread's columns of Dv: c and c + 8
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

  auto slot_of = [&](int64_t i) { return slot0 + (kBackward ? chunks - 1 - i : i); };
  auto fetch = [&](int64_t i) {
    if (i < chunks) {
      uint8_t* st = sm + (i & 1) * L::kStage;
      const uint8_t* rec = rec_at<DK, DV>(a, slot_of(i), h);
      const uint8_t* qrec = qk_at<DK, DV>(a, slot_of(i), hq);
#pragma unroll
      for (int m = 0; m < (kBackward ? 3 : 2); ++m) {
        const uint8_t* src = m == 0 ? rec + R::kW : (m == 1 ? qrec + QR::kK : qrec + QR::kQ);
        uint8_t* dst = st + (m == 0 ? L::kW : (m == 1 ? L::kK : L::kQ));
#pragma unroll
        for (int x = 0; x < C * DK / 8 / kStateThreads; ++x) {
          const int v = x * kStateThreads + tid, r = v / (DK / 8), cc = v % (DK / 8);
          cp16(dst + r * (2 * L::DP) + 16 * cc, src + 16 * v);
        }
      }
      if (tid < C / 4) cp16(st + L::kKw + 16 * tid, rec + R::kF + 4 * R::fKw + 16 * tid);
    }
    cp_commit();
  };
  fetch(0);
  for (int64_t i = 0; i < chunks; ++i) {
    uint8_t* rec = rec_at<DK, DV>(a, slot_of(i), h);
    float* rf = reinterpret_cast<float*>(rec + R::kF);
    uint4 uw[4], ow[4];  // U^T or Y^T as accumulators, and (diag(qe) dO)^T as A fragments
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uw[j] = reinterpret_cast<const uint4*>(rec + (kBackward ? R::kY : R::kU))[slice * 128 + 32 * j + lane];
      if (kBackward) ow[j] = reinterpret_cast<const uint4*>(rec + R::kO)[slice * 128 + 32 * j + lane];
    }
    const float us = rf[R::fScal + (kBackward ? kScalY : kScalU)], os = rf[R::fScal + kScalO], gl = rf[R::fScal + kScalGl];
    fetch(i + 1);
    // the state as this chunk meets it, in fp16: kept for the gradients, and the next product's operand
    uint32_t sf[ND / 2][4];
    float sinv[2];
    scale_rows<ND>(s, sf, sinv);
    {
      __half* sv = reinterpret_cast<__half*>(rec + (kBackward ? R::kD : R::kS)) + (size_t)c * DK + 8 * t;
#pragma unroll
      for (int j = 0; j < ND / 4; ++j) {  // 32 columns: each lane its 8 in one vector (columns 8 b + 2 t, + 1 at 8 t + 2 b, + 1)
        *reinterpret_cast<uint4*>(sv + 32 * j) = make_uint4(sf[2 * j][0], sf[2 * j][2], sf[2 * j + 1][0], sf[2 * j + 1][2]);
        *reinterpret_cast<uint4*>(sv + 8 * DK + 32 * j) = make_uint4(sf[2 * j][1], sf[2 * j][3], sf[2 * j + 1][1], sf[2 * j + 1][3]);
      }
      if (t == 0) {
        rf[(kBackward ? R::fD : R::fS) + c] = sinv[0];
        rf[(kBackward ? R::fD : R::fS) + c + 8] = sinv[1];
      }
    }
    cp_wait<1>();
    __syncthreads();
    const uint8_t* st = sm + (i & 1) * L::kStage;
    const __half *W = reinterpret_cast<const __half*>(st + L::kW), *K = reinterpret_cast<const __half*>(st + L::kK);
    const __half* Q = reinterpret_cast<const __half*>(st + L::kQ);
    const float* kw = reinterpret_cast<const float*>(st + L::kKw);
    // x = S^T W^T (forwards) or dS'^T K^T (backwards), [16 x C]
    float x[8][4] = {};
#pragma unroll
    for (int k = 0; k < ND / 2; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t b[4];
        frag_b<L::DP>(b, kBackward ? K : W, 16 * j, 16 * k, lane);
        mma_f16(x[2 * j], sf[k], b);
        mma_f16(x[2 * j + 1], sf[k], b + 2);
      }
    // forwards V'^T = U^T - x, backwards dV'^T = Y^T + x diag(kw)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint4 w = uw[j / 2];
      const float2 u0 = unpack2(j & 1 ? w.z : w.x), u1 = unpack2(j & 1 ? w.w : w.y);
      const float2 f = kBackward ? *reinterpret_cast<const float2*>(kw + 8 * j + 2 * t) : make_float2(-0x1p-7f, -0x1p-7f);
      x[j][0] = fmaf(x[j][0] * sinv[0], f.x, us * u0.x);
      x[j][1] = fmaf(x[j][1] * sinv[0], f.y, us * u0.y);
      x[j][2] = fmaf(x[j][2] * sinv[1], f.x, us * u1.x);
      x[j][3] = fmaf(x[j][3] * sinv[1], f.y, us * u1.y);
    }
    uint32_t vf[4][4];
    float vinv[2];
    scale_rows<8>(x, vf, vinv);
    __syncwarp();  // the fragments of U or Y that these rows replace are all read
    {
      __half* vv = reinterpret_cast<__half*>(rec + (kBackward ? R::kY : R::kU)) + c * C + 2 * t;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t*>(vv + (e & 1) * 8 * C + 16 * j + 8 * (e >> 1)) = vf[j][e];
      if (t == 0) {
        rf[(kBackward ? R::fDV : R::fV) + c] = vinv[0];
        rf[(kBackward ? R::fDV : R::fV) + c + 8] = vinv[1];
      }
    }
    // forwards S^T = e_last S^T + (V' diag(kw))^T K, backwards dS^T = e_last dS'^T + (dO diag(qe))^T Q - dV'^T W
    const float f0 = vinv[0] * (kBackward ? -0x1p-7f : 0x1p-7f), f1 = vinv[1] * (kBackward ? -0x1p-7f : 0x1p-7f);
    if (!kBackward) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 lo = *reinterpret_cast<const float2*>(kw + 16 * j + 2 * t);
        const float2 hi = *reinterpret_cast<const float2*>(kw + 16 * j + 8 + 2 * t);
        const uint32_t l2 = pack2(lo.x * 0x1p7f, lo.y * 0x1p7f), h2 = pack2(hi.x * 0x1p7f, hi.y * 0x1p7f);
        vf[j][0] = mul2(vf[j][0], l2);
        vf[j][1] = mul2(vf[j][1], l2);
        vf[j][2] = mul2(vf[j][2], h2);
        vf[j][3] = mul2(vf[j][3], h2);
      }
    }
#pragma unroll
    for (int m = 0; m < ND; m += 8) {  // 64 columns of Dk at a time
      float y[8][4] = {}, z[8][4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t b[4];
          frag_b_t<L::DP>(b, kBackward ? W : K, 8 * m + 16 * j, 16 * k, lane);
          mma_f16(y[2 * j], vf[k], b);
          mma_f16(y[2 * j + 1], vf[k], b + 2);
          if (kBackward) {
            const uint32_t of[4] = {ow[k].x, ow[k].y, ow[k].z, ow[k].w};
            frag_b_t<L::DP>(b, Q, 8 * m + 16 * j, 16 * k, lane);
            mma_f16(z[2 * j], of, b);
            mma_f16(z[2 * j + 1], of, b + 2);
          }
        }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = gl * s[m + j][e];
          if (kBackward) v = fmaf(os, z[j][e], v);
          s[m + j][e] = fmaf(e < 2 ? f0 : f1, y[j][e], v);
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
template <int DK, int DV>
__global__ void __launch_bounds__(kStateThreads, 2) states_half_kernel(BwdArgs a) {
  extern __shared__ __align__(16) uint8_t sm[];
  const int col0 = 16 * kStateWarps * (blockIdx.x >> 1);
  if (blockIdx.x & 1)
    walk<DK, DV, true>(a, sm, blockIdx.z, blockIdx.y, col0);
  else
    walk<DK, DV, false>(a, sm, blockIdx.z, blockIdx.y, col0);
}

// ------------------------------------------------------------------ 3. gradients
// One block of 16 warps per (slot, qk-head), which takes its v-heads in turn.  A v-head's tiles come in by
// cp.async, and each buffer is filled for the next v-head as soon as this one is done with it.  Their rows' own
// factors are first made one for the tile (exactly, but for what underflows beside the tile's largest element),
// so that the products need no scaling on the way.

constexpr int kGradThreads = 512;

template <int DK, int DV>
struct GradSmem {
  static constexpr int DP = DK + 8, VP = DV + 8;
  static constexpr size_t kS = 0;                             // fp16 [DV][DP] S^T
  static constexpr size_t kD = kS + 2 * DV * DP;              // fp16 [DV][DP] dS'^T
  static constexpr size_t kV = kD + 2 * DV * DP;              // fp16 [DV][HP] V'^T
  static constexpr size_t kX = kV + 2 * DV * HP;              // fp16 [DV][HP] dV'^T
  static constexpr size_t kO = kX + 2 * DV * HP;              // [C][VP] dO: bf16, then fp16
  static constexpr size_t kT = kO + 2 * C * VP;               // fp16 [C][HP] T
  static constexpr size_t kF = kT + 2 * C * HP;               // two of: the record's floats up to fKw
  static constexpr size_t kFBytes = 4 * Rec<DK, DV>::fKw;
  static constexpr size_t kK = kF + 2 * kFBytes;              // fp16 [C][DP] K16, columns by swap32
  static constexpr size_t kQ = kK + 2 * C * DP;               // fp16 [C][DP] Q16, the same
  static constexpr size_t kDx = kQ + 2 * C * DP;              // fp16 [DV][HP] dX^T
  static constexpr size_t kN = kDx + 2 * DV * HP;             // fp16 [C][HP] N
  static constexpr size_t kB = kN + 2 * C * HP;               // fp16 [C][HP] B
  static constexpr size_t kQf = kB + 2 * C * HP;              // fp32 [4][C] kf, qf, and their shares of the norm
  static constexpr size_t kE = kQf + 16 * C;                  // fp32 [2][C] e, l
  static constexpr size_t kRed = kE + 8 * C;                  // fp32 [4][3][C] row sums by column block; [4][2][C] at the end
  static constexpr size_t kCol = kRed + 48 * C;               // fp32 [4][C] column sums by row block
  static constexpr size_t kDot = kCol + 16 * C;               // fp32 [16] <S, dS'> by warp
  static constexpr size_t kBytes = kDot + 64;
  static_assert(kF % 16 == 0 && kFBytes % 16 == 0 && kBytes <= 232448, "shared memory budget");
};

// Column d of a row of 32 stands at swap32(d): lane t's columns 8 b + 2 t, + 1 of the states' accumulators
// (b = 0..3) are next to one another, so that they were stored as one vector.  Pairs stay pairs, and the swap is
// its own inverse.
__device__ __forceinline__ int swap32(int d) { return (d & ~31) | (((d >> 1) & 3) << 3) | (((d >> 3) & 3) << 1) | (d & 1); }

// The largest of n factors (powers of two, n = 64 or 128), by a warp, and its inverse
__device__ __forceinline__ float top_factor(const float* f, int n, int lane) {
  uint32_t top = 0u;
  for (int i = lane; i < n; i += 32) top = max(top, __float_as_uint(f[i]));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, top));
}
__device__ __forceinline__ uint32_t half2_of(float x) { return pack2(x, x); }

template <int DK, int DV>
__global__ void __launch_bounds__(kGradThreads, 1) grads_half_kernel(BwdArgs a) {
  using L = GradSmem<DK, DV>;
  using R = Rec<DK, DV>;
  using QR = QkRec<DK>;
  extern __shared__ __align__(16) uint8_t sm[];
  constexpr int NK = DK / 32;       // 8-column tiles of a warp's quarter of Dk
  constexpr int KV = DV / 16;       // steps over the columns of Dv
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
  const int hq = blockIdx.y, group = a.nv / a.nqk, h0 = hq * group;
  const int64_t slot = blockIdx.x;
  int64_t c0, end;
  if (!bwd::chunk_at(a, slot, c0, end)) return;
  const int rows = (int)min((int64_t)C, end - c0);
  __half *S = reinterpret_cast<__half*>(sm + L::kS), *D = reinterpret_cast<__half*>(sm + L::kD);
  __half *V = reinterpret_cast<__half*>(sm + L::kV), *X = reinterpret_cast<__half*>(sm + L::kX);
  __half *O = reinterpret_cast<__half*>(sm + L::kO), *T = reinterpret_cast<__half*>(sm + L::kT);
  __half *K = reinterpret_cast<__half*>(sm + L::kK), *Q = reinterpret_cast<__half*>(sm + L::kQ);
  __half *Dx = reinterpret_cast<__half*>(sm + L::kDx), *N = reinterpret_cast<__half*>(sm + L::kN);
  __half* B = reinterpret_cast<__half*>(sm + L::kB);
  float *kf = reinterpret_cast<float*>(sm + L::kQf), *qf = kf + C, *kn = qf + C, *qn = kn + C;
  float *eg = reinterpret_cast<float*>(sm + L::kE), *el = eg + C, *red = reinterpret_cast<float*>(sm + L::kRed);
  float *col = reinterpret_cast<float*>(sm + L::kCol), *dots = reinterpret_cast<float*>(sm + L::kDot);

  // [rows of 2 W bytes] from the record to a tile of pitch 2 P
  auto copy = [&](size_t at, const uint8_t* src, auto width, auto pitch, auto count) {
    constexpr int W = decltype(width)::value / 8, NV = decltype(count)::value * W;  // vectors of a row, of all
#pragma unroll
    for (int x = 0; x < NV / kGradThreads; ++x) {
      const int v = x * kGradThreads + tid;
      cp16(sm + at + (v / W) * (2 * decltype(pitch)::value) + 16 * (v % W), src + 16 * v);
    }
  };
  using IDK = std::integral_constant<int, DK>;
  using IDV = std::integral_constant<int, DV>;
  using IDP = std::integral_constant<int, L::DP>;
  using IC = std::integral_constant<int, C>;
  using IHP = std::integral_constant<int, HP>;
  auto fetch_early = [&](int h) {  // dV'^T, T, dS'^T, dO and the floats
    if (h < h0 + group) {
      const uint8_t* rec = rec_at<DK, DV>(a, slot, h);
      copy(L::kX, rec + R::kY, IC{}, IHP{}, IDV{});
      copy(L::kT, rec + R::kT, IC{}, IHP{}, IC{});
      copy(L::kD, rec + R::kD, IDK{}, IDP{}, IDV{});
#pragma unroll
      for (int x = 0; x < C * DV / 8 / kGradThreads; ++x) {
        const int v = x * kGradThreads + tid, r = v / (DV / 8), c = v % (DV / 8);
        cp16_or_zero(sm + L::kO + r * (2 * L::VP) + 16 * c,
                     static_cast<const bf16*>(a.dout) + ((size_t)(c0 + (r < rows ? r : 0)) * a.nv + h) * DV + 8 * c, r < rows);
      }
      if (tid < R::fKw / 4) cp16(sm + L::kF + ((h - h0) & 1) * L::kFBytes + 16 * tid, rec + R::kF + 16 * tid);
    }
  };
  auto fetch_late = [&](int h) {  // S^T and V'^T
    if (h < h0 + group) {
      const uint8_t* rec = rec_at<DK, DV>(a, slot, h);
      copy(L::kS, rec + R::kS, IDK{}, IDP{}, IDV{});
      copy(L::kV, rec + R::kU, IC{}, IHP{}, IDV{});
    }
    cp_commit();
  };
  fetch_early(h0);
  fetch_late(h0);
  {  // K16, Q16 with their columns swapped as the states' are
    const uint8_t* qrec = qk_at<DK, DV>(a, slot, hq);
#pragma unroll
    for (int x = 0; x < 2 * C * DK / 8 / kGradThreads; ++x) {
      const int v = x * kGradThreads + tid, m = v / (C * DK / 8), r = v / (DK / 8) % C, d = 8 * (v % (DK / 8));
      const uint4 w = *reinterpret_cast<const uint4*>(qrec + 16 * v);
      __half* dst = (m ? Q : K) + r * L::DP;
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(dst + swap32(d + 2 * i)) = u[i];
    }
    if (tid < 4 * C) kf[tid] = reinterpret_cast<const float*>(qrec + QR::kF)[tid];
  }
  __syncthreads();
  // warp: rows 16 wr .., a quarter wc of the columns; thread: rows r0, r0 + 8
  const int wr = 16 * (warp & 3), wc = warp >> 2, r0 = wr + g8;
  const bool low = 16 * wc <= wr;  // the warp's 16 x 16 block of a [C][C] product is not above the diagonal
  uint32_t kk[2][2], qk[2][2];     // k_r . k_i and q_r . k_i, pairs of columns in fp16 (at most 1)
  {
    float xk[2][4] = {}, xq[2][4] = {};
    if (low) {
#pragma unroll
      for (int k = 0; k < DK; k += 16) {
        uint32_t ak[4], aq[4], b[4];
        frag_a<L::DP>(ak, K, wr, k, lane);
        frag_a<L::DP>(aq, Q, wr, k, lane);
        frag_b<L::DP>(b, K, 16 * wc, k, lane);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          mma_f16(xk[j], ak, b + 2 * j);
          mma_f16(xq[j], aq, b + 2 * j);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = r0 + 8 * e, i = 16 * wc + 8 * j + 2 * t4;
        kk[j][e] = pack2(xk[j][2 * e] * kf[r] * kf[i], xk[j][2 * e + 1] * kf[r] * kf[i + 1]);
        qk[j][e] = pack2(xq[j][2 * e] * qf[r] * kf[i], xq[j][2 * e + 1] * qf[r] * kf[i + 1]);
      }
  }
  // kf dk_hat and qf dq_hat, summed over the group's v-heads
  float dq[NK][4] = {}, dk[NK][4] = {};

  for (int h = h0; h < h0 + group; ++h) {
    const float* rf = reinterpret_cast<const float*>(sm + L::kF + ((h - h0) & 1) * L::kFBytes);
    cp_wait<0>();
    __syncthreads();
    // this thread's share of V: rows r0, r0 + 8, columns 16 k + 2 t, + 8 for k = wc and wc + 4
    uint32_t vraw[KV / 4][4];
#pragma unroll
    for (int x = 0; x < KV / 4; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + 8 * (e & 1), c = 16 * (wc + 4 * x) + 8 * (e >> 1) + 2 * t4;
        vraw[x][e] = r < rows ? *reinterpret_cast<const uint32_t*>(static_cast<const bf16*>(a.v) + ((size_t)(c0 + r) * a.nv + h) * DV + c) : 0u;
      }
    // one factor for a tile
    const float mS = top_factor(rf + R::fS, DV, lane), mD = top_factor(rf + R::fD, DV, lane);
    const float mV = top_factor(rf + R::fV, DV, lane), mX = top_factor(rf + R::fDV, DV, lane);
    const float oinv = rf[R::fScal + kScalDo];
    float s_dot = 0.f;
#pragma unroll
    for (int x = 0; x < DV * DK / 8 / kGradThreads; ++x) {
      const int v = x * kGradThreads + tid, c = v / (DK / 8), at = c * L::DP + 8 * (v % (DK / 8));
      const uint32_t fS = half2_of(__fdividef(rf[R::fS + c], mS)), fD = half2_of(__fdividef(rf[R::fD + c], mD));
      uint4 p = *reinterpret_cast<const uint4*>(S + at), q = *reinterpret_cast<const uint4*>(D + at);
      p = make_uint4(mul2(p.x, fS), mul2(p.y, fS), mul2(p.z, fS), mul2(p.w, fS));
      q = make_uint4(mul2(q.x, fD), mul2(q.y, fD), mul2(q.z, fD), mul2(q.w, fD));
      *reinterpret_cast<uint4*>(S + at) = p;
      *reinterpret_cast<uint4*>(D + at) = q;
      const uint32_t ps[4] = {p.x, p.y, p.z, p.w}, qs[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = unpack2(ps[i]), w = unpack2(qs[i]);
        s_dot = fmaf(u.x, w.x, fmaf(u.y, w.y, s_dot));
      }
    }
#pragma unroll
    for (int x = 0; x < DV * C / 8 / kGradThreads; ++x) {
      const int v = x * kGradThreads + tid, c = v / (C / 8), at = c * HP + 8 * (v % (C / 8));
      const uint32_t f = half2_of(__fdividef(rf[R::fV + c], mV));
      const uint4 p = *reinterpret_cast<const uint4*>(V + at);
      *reinterpret_cast<uint4*>(V + at) = make_uint4(mul2(p.x, f), mul2(p.y, f), mul2(p.z, f), mul2(p.w, f));
    }
#pragma unroll
    for (int x = 0; x < C * DV / 8 / kGradThreads; ++x) {
      const int v = x * kGradThreads + tid, at = (v / (DV / 8)) * L::VP + 8 * (v % (DV / 8));
      const uint4 w = *reinterpret_cast<const uint4*>(O + at);
      const float os = __fdividef(1.f, oinv);  // a power of two
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = bf2(u[i]);
        r[i] = pack2(f.x * os, f.y * os);
      }
      *reinterpret_cast<uint4*>(O + at) = make_uint4(r[0], r[1], r[2], r[3]);
    }
    if (tid < C) {
      eg[tid] = expf(rf[R::fGc + tid]);
      el[tid] = expf(rf[R::fGc + C - 1] - rf[R::fGc + tid]);
    }
    __syncthreads();
    {  // dX^T = dV'^T T, times 2^7 for T and 2^-7: 16 columns of Dv by two blocks of 16 tokens, of like cost together
      const int cb = 16 * (warp % KV);
      uint32_t af[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) frag_a<HP>(af[k], X, cb, 16 * k, lane);
      const float f0 = __fdividef(rf[R::fDV + cb + g8], mX) * 0x1p-7f, f1 = __fdividef(rf[R::fDV + cb + g8 + 8], mX) * 0x1p-7f;
#pragma unroll
      for (int u = 0; u < KV / 4; ++u) {
        // DV = 128: warps 0..7 take blocks 0 and 3, 8..15 blocks 1 and 2; DV = 64: one block a warp
        const int ib = KV == 8 ? (warp < 8 ? 3 * u : 1 + u) : warp / KV;
        float x[2][4] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // T's zeros above the diagonal are multiplied too: a branch would cost more
          uint32_t b[4];
          frag_b_t<HP>(b, T, 16 * ib, 16 * k, lane);
          mma_f16(x[0], af[k], b);
          mma_f16(x[1], af[k], b + 2);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          __half* dst = Dx + (cb + g8) * HP + 16 * ib + 8 * j + 2 * t4;
          *reinterpret_cast<uint32_t*>(dst) = pack2(x[j][0] * f0, x[j][1] * f0);
          *reinterpret_cast<uint32_t*>(dst + 8 * HP) = pack2(x[j][2] * f1, x[j][3] * f1);
        }
      }
    }
    // x[NK] += A fragment times 16 rows of a [DV][DP] tile: this warp's rows, its quarter of the columns of Dk
    auto with_state = [&](float (&x)[NK][4], const uint32_t* f, int k, const __half* tile) {
#pragma unroll
      for (int j = 0; j < NK; j += 2) {
        uint32_t b[4];
        frag_b_t<L::DP>(b, tile, 8 * (NK * wc + j), 16 * k, lane);
        mma_f16(x[j], f, b);
        mma_f16(x[j + 1], f, b + 2);
      }
    };
    // rows' dots with a tile, and x times their factors into a sum
    auto take = [&](const float (&x)[NK][4], const __half* Y, const float (&f)[2], float (&sum)[NK][4], float (&dot)[2]) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        dot[e] = 0.f;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          const float2 y = unpack2(*reinterpret_cast<const uint32_t*>(Y + (r0 + 8 * e) * L::DP + 8 * (NK * wc + j) + 2 * t4));
          dot[e] = fmaf(x[j][2 * e], y.x, fmaf(x[j][2 * e + 1], y.y, dot[e]));
          sum[j][2 * e] = fmaf(f[e], x[j][2 * e], sum[j][2 * e]);
          sum[j][2 * e + 1] = fmaf(f[e], x[j][2 * e + 1], sum[j][2 * e + 1]);
        }
      }
    };
    float dA[2][4] = {}, dP[2][4] = {}, s_gc[2], s_bt[2] = {0.f, 0.f}, s_th[2], f[2], dot[2];
    {  // dO S^T and dP
      float x[NK][4] = {};
#pragma unroll
      for (int k = 0; k < KV; ++k) {
        uint32_t af[4];
        frag_a<L::VP>(af, O, wr, 16 * k, lane);
        with_state(x, af, k, S);
      }
      if (low) {
#pragma unroll
        for (int k = 0; k < KV; ++k) {
          uint32_t af[4], b[4];
          frag_a<L::VP>(af, O, wr, 16 * k, lane);
          frag_b_t<HP>(b, V, 16 * wc, 16 * k, lane);
          mma_f16(dP[0], af, b);
          mma_f16(dP[1], af, b + 2);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) f[e] = a.scale * eg[r0 + 8 * e] * qf[r0 + 8 * e] * oinv * mS;
      take(x, Q, f, dq, dot);
#pragma unroll
      for (int e = 0; e < 2; ++e) s_gc[e] = f[e] * dot[e];
    }
    {  // V' dS'^T
      float x[NK][4] = {};
#pragma unroll
      for (int k = 0; k < KV; ++k) {
        uint32_t af[4];
        frag_a_t<HP>(af, V, wr, 16 * k, lane);
        with_state(x, af, k, D);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) f[e] = el[r0 + 8 * e] * kf[r0 + 8 * e] * mV * mD;
      take(x, K, f, dk, dot);
#pragma unroll
      for (int e = 0; e < 2; ++e) s_th[e] = f[e] * dot[e];
    }
    __syncthreads();  // dX is here; dV', T, dS' and dO are done with
    fetch_early(h + 1);
    {  // dX S^T, dA; dV = diag(b) dX and its part of dbeta
      float x[NK][4] = {};
#pragma unroll
      for (int k = 0; k < KV; ++k) {
        uint32_t af[4];
        frag_a_t<HP>(af, Dx, wr, 16 * k, lane);
        with_state(x, af, k, S);
      }
      if (low) {
#pragma unroll
        for (int k = 0; k < KV; ++k) {
          uint32_t af[4], b[4];
          frag_a_t<HP>(af, Dx, wr, 16 * k, lane);
          frag_b_t<HP>(b, V, 16 * wc, 16 * k, lane);
          mma_f16(dA[0], af, b);
          mma_f16(dA[1], af, b + 2);
        }
      }
#pragma unroll
      for (int m = 0; m < KV / 4; ++m) {
        const int k = wc + 4 * m;
        uint32_t af[4];
        frag_a_t<HP>(af, Dx, wr, 16 * k, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + 8 * (e & 1), c = 16 * k + 8 * (e >> 1) + 2 * t4;
          float2 d = unpack2(af[e]);
          d.x *= mX;
          d.y *= mX;
          const float2 v = bf2(vraw[m][e]);
          s_bt[e & 1] = fmaf(d.x, v.x, fmaf(d.y, v.y, s_bt[e & 1]));
          const float b = rf[R::fBeta + r];
          if (r < rows)
            *reinterpret_cast<uint32_t*>(static_cast<bf16*>(a.dv_out) + ((size_t)(c0 + r) * a.nv + h) * DV + c) =
                ptx::pack_bf16x2(b * d.x, b * d.y);
        }
      }
      float u[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        u[e] = -eg[r0 + 8 * e] * kf[r0 + 8 * e] * mX * mS;
        f[e] = rf[R::fBeta + r0 + 8 * e] * u[e];
      }
      take(x, K, f, dk, dot);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s_bt[e] = fmaf(u[e], dot[e], s_bt[e]);
        s_gc[e] = fmaf(f[e], dot[e], s_gc[e]);
      }
    }
    // what goes through A and P
    const float sP = oinv * mV, sA = mX * mV;
    float cs[2][2];
    {
      const float *gc = rf + R::fGc, *bt = rf + R::fBeta;
      constexpr float kLog2e = 1.44269504f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i0 = 16 * wc + 8 * j + 2 * t4;
        cs[j][0] = cs[j][1] = 0.f;
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          const int r = r0 + 8 * e2;
          const float2 kd2 = unpack2(kk[j][e2]), qk2 = unpack2(qk[j][e2]);
          float nn[2], bb[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = i0 + e;
            // masked before exp; the strict triangle for A
            const float gamma = i <= r ? ptx::ex2_approx(kLog2e * (gc[r] - gc[i])) : 0.f, strict = i < r ? gamma : 0.f;
            const float dp = dP[j][2 * e2 + e], da = dA[j][2 * e2 + e];
            const float kd = (e ? kd2.y : kd2.x) * strict, akd = sA * da * kd;
            const float both = fmaf(-bt[r], akd, a.scale * sP * dp * strict * (e ? qk2.y : qk2.x));
            s_bt[e2] -= akd;
            s_gc[e2] += both;
            cs[j][e] += both;
            nn[e] = dp * gamma * (qf[r] * kf[i]) * 0x1p6f;                // 2^14 for the factors, 2^-8
            bb[e] = -da * bt[r] * strict * (kf[r] * kf[i]) * 0x1p-2f;     // 2^14, 2^-16
          }
          *reinterpret_cast<uint32_t*>(N + r * HP + i0) = pack2(nn[0], nn[1]);
          *reinterpret_cast<uint32_t*>(B + r * HP + i0) = pack2(bb[0], bb[1]);
        }
      }
    }
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
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) cs[j][e] += __shfl_xor_sync(0xffffffffu, cs[j][e], o);
        if (g8 == 0) col[(warp & 3) * C + 16 * wc + 8 * j + 2 * t4 + e] = cs[j][e];
      }
    s_dot = warp_sum(s_dot);
    if (lane == 0) dots[warp] = s_dot * mS * mD;
    __syncthreads();  // N, B and the sums are here; S and V' are done with
    fetch_late(h + 1);
    {  // qf dq_hat += N K16, kf dk_hat += N^T Q16 + (B + B^T) K16 (zeros of the triangle included: see dX)
      float xq[NK][4] = {}, xn[NK][4] = {}, xb[NK][4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t an[4], ant[4], ab[4], abt[4];
        frag_a<HP>(an, N, wr, 16 * k, lane);
        frag_a<HP>(ab, B, wr, 16 * k, lane);
        frag_a_t<HP>(ant, N, wr, 16 * k, lane);
        frag_a_t<HP>(abt, B, wr, 16 * k, lane);
#pragma unroll
        for (int j = 0; j < NK; j += 2) {
          uint32_t bk[4], bq[4];
          frag_b_t<L::DP>(bk, K, 8 * (NK * wc + j), 16 * k, lane);
          frag_b_t<L::DP>(bq, Q, 8 * (NK * wc + j), 16 * k, lane);
          mma_f16(xq[j], an, bk);
          mma_f16(xq[j + 1], an, bk + 2);
          mma_f16(xb[j], ab, bk);
          mma_f16(xb[j + 1], ab, bk + 2);
          mma_f16(xn[j], ant, bq);
          mma_f16(xn[j + 1], ant, bq + 2);
          mma_f16(xb[j], abt, bk);
          mma_f16(xb[j + 1], abt, bk + 2);
        }
      }
      const float sN = a.scale * sP * 0x1p-6f, sB = sA * 0x1p2f;
#pragma unroll
      for (int j = 0; j < NK; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dq[j][e] = fmaf(sN, xq[j][e], dq[j][e]);
          dk[j][e] = fmaf(sN, xn[j][e], fmaf(sB, xb[j][e], dk[j][e]));
        }
    }
    if (warp == 0) {
      // dgc of rows 2 lane, 2 lane + 1; then the suffix sums
      float d[2], th = 0.f, bsum[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * lane + e;
        float sum[3], cols = 0.f;
#pragma unroll
        for (int m = 0; m < 3; ++m) sum[m] = (red[m * C + r] + red[(3 + m) * C + r]) + (red[(6 + m) * C + r] + red[(9 + m) * C + r]);
#pragma unroll
        for (int m = 0; m < 4; ++m) cols += col[m * C + r];
        th += sum[2];
        d[e] = sum[0] - sum[2] - cols;
        bsum[e] = sum[1];
      }
      th = warp_sum(th);
      const float dsum = warp_sum(lane < 16 ? dots[lane] : 0.f);
      if (lane == 31) d[1] += th + eg[C - 1] * dsum;
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
        if (2 * lane + e < rows) {
          const size_t at = (size_t)(c0 + 2 * lane + e) * a.nv + h;
          static_cast<bf16*>(a.dg)[at] = __float2bfloat16_rn(dg[e]);
          static_cast<bf16*>(a.dbeta)[at] = __float2bfloat16_rn(bsum[e]);
        }
    }
  }
  __syncthreads();
  // the norms: with y = qf dq_hat, dq = (y - qf^2 Q16 (Q16 . y)) / (qf |q|)
  float dotq[2], dotk[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    dotq[e] = dotk[e] = 0.f;
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      const int at = (r0 + 8 * e) * L::DP + 8 * (NK * wc + j) + 2 * t4;
      const float2 y = unpack2(*reinterpret_cast<const uint32_t*>(Q + at)), z = unpack2(*reinterpret_cast<const uint32_t*>(K + at));
      dotq[e] = fmaf(dq[j][2 * e], y.x, fmaf(dq[j][2 * e + 1], y.y, dotq[e]));
      dotk[e] = fmaf(dk[j][2 * e], z.x, fmaf(dk[j][2 * e + 1], z.y, dotk[e]));
    }
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
  for (int e = 0; e < 2; ++e) {
    const int r = r0 + 8 * e;
    if (r >= rows) continue;
    const float pq = qf[r] * qf[r] * ((red[r] + red[2 * C + r]) + (red[4 * C + r] + red[6 * C + r]));
    const float pk = kf[r] * kf[r] * ((red[C + r] + red[3 * C + r]) + (red[5 * C + r] + red[7 * C + r]));
    const size_t row = ((size_t)(c0 + r) * a.nqk + hq) * DK;
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      const int p = 8 * (NK * wc + j) + 2 * t4;
      const float2 y = unpack2(*reinterpret_cast<const uint32_t*>(Q + r * L::DP + p)), z = unpack2(*reinterpret_cast<const uint32_t*>(K + r * L::DP + p));
      const size_t at = row + swap32(p);
      *reinterpret_cast<uint32_t*>(static_cast<bf16*>(a.dq) + at) =
          ptx::pack_bf16x2(qn[r] * (dq[j][2 * e] - y.x * pq), qn[r] * (dq[j][2 * e + 1] - y.y * pq));
      *reinterpret_cast<uint32_t*>(static_cast<bf16*>(a.dk) + at) =
          ptx::pack_bf16x2(kn[r] * (dk[j][2 * e] - z.x * pk), kn[r] * (dk[j][2 * e + 1] - z.y * pk));
    }
  }
}

template <typename F>
static cudaError_t set_smem(F kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int DK, int DV>
static cudaError_t launch_one(const BwdArgs& a, cudaStream_t stream) {
  const unsigned int slots = (unsigned int)slots_of<DK, DV>(a);
  cudaError_t e;
  if (a.total_tokens > 0) {
    if ((e = set_smem(prepare_half_kernel<DK, DV>, PrepSmem<DK, DV>::kBytes)) != cudaSuccess) return e;
    prepare_half_kernel<DK, DV><<<dim3(slots, a.nqk), kPrepThreads, PrepSmem<DK, DV>::kBytes, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = set_smem(states_half_kernel<DK, DV>, StateSmem<DK>::kBytes)) != cudaSuccess) return e;
  states_half_kernel<DK, DV><<<dim3(2 * DV / (16 * kStateWarps), a.nv, a.num_seqs), kStateThreads, StateSmem<DK>::kBytes, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || a.total_tokens == 0) return e;
  if ((e = set_smem(grads_half_kernel<DK, DV>, GradSmem<DK, DV>::kBytes)) != cudaSuccess) return e;
  grads_half_kernel<DK, DV><<<dim3(slots, a.nqk), kGradThreads, GradSmem<DK, DV>::kBytes, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace bwdh

int64_t chunk_bwd_half_workspace(int64_t total_tokens, int num_seqs, int nqk, int nv, int dk, int dv) {
  if (total_tokens == 0) return 0;
  const int64_t c = bwdh::C;
  const int64_t rec = 2 * (c * (c + dk + 3 * dv) + 2 * (int64_t)dk * dv) + 4 * (3 * c + 8 + 4 * dv);
  return (total_tokens / c + num_seqs) * (nv * rec + nqk * (4 * c * dk + 16 * c));
}

cudaError_t launch_chunk_bwd_half(const BwdArgs& a, int dk, int dv, cudaStream_t s) {
  static_assert(bwdh::Rec<128, 64>::kBytes == 2 * (64 * (64 + 128 + 3 * 64) + 2 * 128 * 64) + 4 * (3 * 64 + 8 + 4 * 64), "workspace size");
  static_assert(bwdh::QkRec<128>::kBytes == 4 * 64 * 128 + 16 * 64, "workspace size");
  if (dk == 64 && dv == 64) return bwdh::launch_one<64, 64>(a, s);
  if (dk == 64 && dv == 128) return bwdh::launch_one<64, 128>(a, s);
  if (dk == 128 && dv == 64) return bwdh::launch_one<128, 64>(a, s);
  if (dk == 128 && dv == 128) return bwdh::launch_one<128, 128>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace gdn
