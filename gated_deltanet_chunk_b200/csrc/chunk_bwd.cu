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
//   2. states: two warps per 16 Dv columns walk their sequence, forwards for S
//      and V', backwards for dS' and dV'.  The state slice stays in their
//      registers as S^T [16 x Dk] MMA accumulators, half of Dk each, whose layout
//      is that of the next product's A operand, so a chunk is two (or three)
//      chained products, and all that goes through shared memory is one sum of
//      what both have.  The two directions need nothing of each other and run in
//      the same launch.
//   3. gradients (every chunk and qk-head at once): the rest.  One block takes
//      all the v-heads that share a qk-head, one after another, so dq and dk
//      are summed in registers, in a fixed order.
// Every operand of a product is a pair hi + lo of fp16, scaled by a power of two that
// a row or a tile shares, and a product is three MMAs: within about 2^-22 of its value.
// Rows of W and the columns of V' diag(kw), dV' diag(wr) and diag(s e) dO have factors
// of their own: they take any number of binades over a chunk, with the decay.
// Pairs are formed once, where a tile is made, and stand in the caller's workspace as
// images that one bulk copy brings into shared memory.  An MMA of fp16 takes twice the
// terms of one of TF32, and ldmatrix feeds it; with pairs of TF32 split as they were
// loaded the three kernels took 0.56, 2.26 and 1.25 ms for 4 x 4096 tokens, 4 / 8 heads
// of 128, against 0.27, 0.47 and 0.46 now (1 x 256 tokens, one head of 64: 16, 17 and
// 14 us).  Partial sums of one MMA step (16 terms) are added in fp32: the MMA itself
// truncates, and over long sums that showed (3.8e-6 relative against 64 bits; now
// 2.7e-7).  Only the inverse's blocks off its 16 x 16 diagonal split TF32.  The sums of
// gates are pairs of fp32, so that decays do not lose digits behind a strong one.
//
// Bound by latency: prepare and gradients run one block per SM in 7 waves and issue in
// a third of the cycles (the tensor pipe is busy in 16 and 24 %); states has 128
// blocks, whose 64 chunks wait for one another, 13,500 cycles each, of which the MMAs
// are 4,600.

#include "chunk_bwd.cuh"
#include "train_common.cuh"
#include "gdn_launch.h"
#include "sm100_ptx.cuh"

namespace gdn {
namespace bwd {

constexpr int kThreads = 512;  // prepare and gradients

// A pair image: an image (chunk_bwd.cuh) of the hi parts and one of the lo parts, in blocks of 16 rows, hi then lo,
// so that any 16 rows are one piece.  Byte of element (r, col) of hi; lo stands 16 RB behind.
template <int RB> __host__ __device__ __forceinline__ int pair_at(int r, int col) {
  return (r >> 4) * (32 * RB) + (r & 15) * RB + ((((col >> 3) ^ (r & 7)) << 4) | ((col & 7) * 2));
}
template <int RB> __device__ __forceinline__ uint32_t pair_word(uint32_t img, int r, int col) {
  return img + (uint32_t)pair_at<RB>(r, col);
}
// Fragments of a pair image, hi and lo
template <int RB> __device__ __forceinline__ void pair_a(uint32_t* h, uint32_t* l, uint32_t img, int m0, int k0, const Lane& ln) {
  const uint32_t p = img_addr<RB, true>(img, m0, k0, ln.ra, ln.sa);
  ldsm(h, p);
  ldsm(l, p + 16 * RB);
}
template <int RB> __device__ __forceinline__ void pair_a_t(uint32_t* h, uint32_t* l, uint32_t img, int m0, int k0, const Lane& ln) {
  const uint32_t p = img_addr<RB, true>(img, k0, m0, ln.rb, ln.sb);
  ldsm_t(h, p);
  ldsm_t(l, p + 16 * RB);
}
template <int RB> __device__ __forceinline__ void pair_b(uint32_t* h, uint32_t* l, uint32_t img, int n0, int k0, const Lane& ln) {
  const uint32_t p = img_addr<RB, true>(img, n0, k0, ln.rb, ln.sb);
  ldsm(h, p);
  ldsm(l, p + 16 * RB);
}
template <int RB> __device__ __forceinline__ void pair_b_t(uint32_t* h, uint32_t* l, uint32_t img, int n0, int k0, const Lane& ln) {
  const uint32_t p = img_addr<RB, true>(img, k0, n0, ln.ra, ln.sa);
  ldsm_t(h, p);
  ldsm_t(l, p + 16 * RB);
}
// x += (ah + al) (bh + bl), the 16 terms of one step; added to x in fp32, since the MMA truncates as it adds
__device__ __forceinline__ void mma_pair(float* x, const uint32_t* ah, const uint32_t* al, const uint32_t* bh, const uint32_t* bl) {
  float d[4] = {};
  mma_f16(d, al, bh);
  mma_f16(d, ah, bl);
  mma_f16(d, ah, bh);
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] += d[e];
}
// x f as a pair, two values at a time
__device__ __forceinline__ void pair2(float x, float y, float f, uint32_t& hi, uint32_t& lo) {
  x *= f;
  y *= f;
  hi = pack2(x, y);
  const float2 h = unpack2(hi);
  lo = pack2(x - h.x, y - h.y);
}
__device__ __forceinline__ float2 both2(uint32_t hi, uint32_t lo) {
  const float2 h = unpack2(hi), l = unpack2(lo);
  return make_float2(h.x + l.x, h.y + l.y);
}

// One record per (chunk slot, v-head) in the workspace, in bytes.
template <int DK, int DV>
struct Rec {
  static constexpr size_t kX = 0;                      // (P^T dO)^T as accumulators, then pair image of dV'^T [DV][C]
  static constexpr size_t kV = kX + 4 * C * DV;        // U^T as accumulators, then pair image of V'^T [DV][C]
  static constexpr size_t kT = kV + 4 * C * DV;        // pair image of T [C][C]
  static constexpr size_t kS = kT + 4 * C * C;         // pair image of S^T [DV][DK] before the chunk, columns by swap32
  static constexpr size_t kD = kS + 4 * DK * DV;       // of dS'^T behind the chunk
  static constexpr size_t kO = kD + 4 * DK * DV;       // pair images of dO, 64 columns at a time: [C][64]
  static constexpr size_t kW = kO + 4 * C * DV;        // pair image of W [C][DK]
  static constexpr size_t kOq = kW + 4 * C * DK;       // (diag(qe) dO)^T as A fragments: hi, lo
  static constexpr size_t kF = kOq + 4 * C * DV;       // floats from here:
  static constexpr int fGc = 0;                        // [C] gcum, and [C] what it has beyond fp32
  static constexpr int fBeta = fGc + 2 * C;            // [C] beta
  static constexpr int fScal = fBeta + C;              // [8] see Scal
  static constexpr int fS = fScal + 8;                 // [DV] factor of every row of S^T (one for 64 rows)
  static constexpr int fD = fS + DV;                   // [DV] of dS'^T
  static constexpr int fV = fD + DV;                   // [DV] of V'^T
  static constexpr int fDV = fV + DV;                  // [DV] of dV'^T
  static constexpr int fKw = fDV + DV;                 // [C] l_r over the factor of row r of K16
  static constexpr int fWr = fKw + C;                  // [C] factor of the rows of W
  static constexpr int fOq = fWr + C;                  // [DV] factor of the rows of Oq
  static constexpr int kFloats = fOq + DV;
  static constexpr size_t kBytes = kF + 4 * kFloats;
  static_assert(kBytes % 16 == 0 && fScal % 4 == 0 && fKw % 4 == 0, "16-byte copies");
};
enum Scal { kScalGl, kScalT, kScalDo };  // e_last; factors of T, dO

// One record per (chunk slot, qk-head), in bytes.
template <int DK>
struct QkRec {
  static constexpr size_t kK = 0;                 // pair image [C][DK] of K16
  static constexpr size_t kQ = kK + 4 * C * DK;   // of Q16
  static constexpr size_t kKs = kQ + 4 * C * DK;  // of K16 with its columns by swap32
  static constexpr size_t kQs = kKs + 4 * C * DK;
  static constexpr size_t kF = kQs + 4 * C * DK;  // floats [4][C]: k_hat = kf K16, q_hat = qf Q16, 1 / (kf |k|), 1 / (qf |q|)
  static constexpr size_t kLoad = kF + 16 * C - kKs;  // what the gradients keep in shared memory
  static constexpr size_t kKk = kF + 16 * C;      // k_hat_r . k_hat_i as accumulators: float4 [16-row block][8-column block][lane]
  static constexpr size_t kQk = kKk + 4 * C * C;  // q_hat_r . k_hat_i
  static constexpr size_t kBytes = kQk + 4 * C * C;
};
template <int DK, int DV>
__device__ __forceinline__ uint8_t* rec_at(const BwdArgs& a, int64_t slot, int h) {
  return reinterpret_cast<uint8_t*>(a.ws) + ((size_t)slot * a.nv + h) * Rec<DK, DV>::kBytes;
}
template <int DK, int DV>
__device__ __forceinline__ uint8_t* qk_at(const BwdArgs& a, int64_t slot, int hq) {
  const size_t slots = (size_t)(a.total_tokens / C + a.num_seqs);
  return reinterpret_cast<uint8_t*>(a.ws) + slots * a.nv * Rec<DK, DV>::kBytes + ((size_t)slot * a.nqk + hq) * QkRec<DK>::kBytes;
}

// Eight consecutive values as fp32
template <typename IO> __device__ __forceinline__ void load8(const IO* p, bool valid, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (!valid) return;
  if constexpr (sizeof(IO) == 4) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ float top8(const float (&v)[8]) {
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) t = fmaxf(t, fabsf(v[i]));
  return t;
}
__device__ __forceinline__ float warp_top(float x) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x))); }
// Eight values times f, as 16-byte vectors of hi and lo
__device__ __forceinline__ void pair8(const float (&v)[8], float f, uint4& hi, uint4& lo) {
  pair2(v[0], v[1], f, hi.x, lo.x);
  pair2(v[2], v[3], f, hi.y, lo.y);
  pair2(v[4], v[5], f, hi.z, lo.z);
  pair2(v[6], v[7], f, hi.w, lo.w);
}

// exp(gcum_r - gcum_i) from [C] gcum and [C] its low part
__device__ __forceinline__ float decay(const float* gc, int r, int i) { return expf((gc[r] - gc[i]) + (gc[C + r] - gc[C + i])); }

// ------------------------------------------------------------------ 1. prepare
// One block of 16 warps per (slot, qk-head): K16, Q16 and their products once, then its v-heads in turn.

template <int DK, int DV>
struct PrepSmem {
  static constexpr size_t kK = 0;                                   // pair image [C][DK] of K16
  static constexpr size_t kQ = kK + 4 * C * DK;                     // of Q16; then of T diag(b) and of P, [C][C] each
  static constexpr size_t kQBytes = DK == 128 ? 4 * C * DK : 8 * C * C;
  static constexpr size_t kV = kQ + kQBytes;                        // of V [C][DV]
  static constexpr size_t kO = kV + 4 * C * DV;                     // of dO, [C][64] for 64 columns at a time
  static constexpr size_t kA = kO + 4 * C * DV;                     // fp32 [C][TP] A, then T
  static constexpr size_t kY = kA + 4 * C * TP;                     // fp32 [C / 2][TP] scratch of the inverse
  static constexpr size_t kF = kY + 2 * C * TP;                     // fp32 [C] each: gc, its low part, beta, kf, qf, beta e kf, s e qf
  static constexpr size_t kTop = kF + 28 * C;                       // fp32 [4][16] largest elements by warp; [4][C] of rows
  static constexpr size_t kBytes = kTop + 256 + 16 * C;
  static_assert(kBytes <= 232448, "shared memory budget");
};

// The largest of 16 warps' values
__device__ __forceinline__ float top16(const float* t, int lane) { return warp_top(t[lane & 15]); }

// Rows of q or k, one vector of 8 for each of a thread's rows; `norm`: the factors of the L2 norm (1 without it)
template <int DK, typename IO>
__device__ __forceinline__ void load_qk(const IO* x, int64_t c0, int64_t end, int heads, int head, bool l2,
                                        float (&v)[C * DK / 8 / kThreads][8], float (&norm)[C * DK / 8 / kThreads], float* row_top,
                                        int tid) {
  constexpr int L = DK / 8, R = kThreads / L;
#pragma unroll
  for (int p = 0; p < C / R; ++p) {
    const int r = p * R + tid / L;
    load8<IO>(x + ((size_t)(c0 + r < end ? c0 + r : c0) * heads + head) * DK + 8 * (tid % L), c0 + r < end, v[p]);
  }
#pragma unroll
  for (int p = 0; p < C / R; ++p) {
    float ss = 0.f, top = top8(v[p]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[p][i], v[p][i], ss);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    norm[p] = l2 ? 1.f / sqrtf(ss + kNormEps) : 1.f;
    if (tid % L == 0) row_top[p * R + tid / L] = top * norm[p];
  }
}
// The same rows, normalised, as a pair image in shared memory and two in the workspace.  A row's factor of two goes
// by its largest element, but not by less than 2^-12 of the tile's (1 with the L2 norm): the factors of the rows
// stay within reach of one another, and a row of zeros has one.
template <int DK>
__device__ __forceinline__ void store_qk(const float (&v)[C * DK / 8 / kThreads][8], const float (&norm)[C * DK / 8 / kThreads], bool l2,
                                         const float* row_top, uint8_t* tile, uint8_t* plain, uint8_t* swapped, float* f, float* wf,
                                         float* wn, int tid) {
  constexpr int L = DK / 8, R = kThreads / L, RB = 2 * DK;
  const int lr = tid % L, lane = tid & 31;
  float all = 1.f;
  if (!l2) {
    all = warp_top(fmaxf(row_top[lane], row_top[32 + lane]));
    if (!(all > 0.f)) all = 1.f;
  }
#pragma unroll
  for (int p = 0; p < C / R; ++p) {
    const int r = p * R + tid / L;
    float s, inv;
    pow2_factor(fmaxf(row_top[r], all * 0x1p-12f), s, inv);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[p][i] * norm[p];
    uint4 hi, lo;
    pair8(x, s, hi, lo);
    const int at = pair_at<RB>(r, 8 * lr);
    *reinterpret_cast<uint4*>(tile + at) = hi;
    *reinterpret_cast<uint4*>(tile + at + 16 * RB) = lo;
    *reinterpret_cast<uint4*>(plain + at) = hi;
    *reinterpret_cast<uint4*>(plain + at + 16 * RB) = lo;
    transpose4(hi, lr);
    transpose4(lo, lr);
    const int w = pair_at<RB>(r, (8 * lr & ~31) + 8 * (lr & 3));
    *reinterpret_cast<uint4*>(swapped + w) = hi;
    *reinterpret_cast<uint4*>(swapped + w + 16 * RB) = lo;
    if (lr == 0) {
      f[r] = wf[r] = inv;
      wn[r] = norm[p] * s;
    }
  }
}

template <int DK, int DV, typename IO>
__global__ void __launch_bounds__(kThreads, 1) prepare_kernel(BwdArgs a) {
  let_next_begin();
  using L = PrepSmem<DK, DV>;
  using R = Rec<DK, DV>;
  using QR = QkRec<DK>;
  extern __shared__ __align__(128) uint8_t sm[];
  constexpr int RK = 2 * DK, RV = 2 * DV, RC = 2 * C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Lane ln(lane);
  const int hq = blockIdx.x, group = a.nv / a.nqk;
  const int64_t slot = grid_slot();
  if (slot >= a.total_tokens / C + a.num_seqs) return;
  int64_t c0, end;
  if (!chunk_at(a, slot, c0, end)) return;
  const uint32_t base = ptx::smem_u32(sm);
  const uint32_t K = base + L::kK, Q = base + L::kQ, TB = Q, P = Q + 4 * C * C, V = base + L::kV, O = base + L::kO;
  float *A = reinterpret_cast<float*>(sm + L::kA), *Y = reinterpret_cast<float*>(sm + L::kY);
  float *gc = reinterpret_cast<float*>(sm + L::kF), *gl = gc + C, *bt = gl + C, *kf = bt + C, *qf = kf + C, *wf = qf + C, *qe = wf + C;
  float *tops = reinterpret_cast<float*>(sm + L::kTop), *rows = tops + 64;
  uint8_t* qrec = qk_at<DK, DV>(a, slot, hq);
  float* qfl = reinterpret_cast<float*>(qrec + QR::kF);
  const bool l2 = a.qk_l2norm != 0;
  {
    constexpr int N = C * DK / 8 / kThreads;
    float kv[N][8], qv[N][8], kn[N], qn[N];
    load_qk<DK, IO>(static_cast<const IO*>(a.k), c0, end, a.nqk, hq, l2, kv, kn, rows, tid);
    load_qk<DK, IO>(static_cast<const IO*>(a.q), c0, end, a.nqk, hq, l2, qv, qn, rows + C, tid);
    constexpr int LN = DV * sizeof(IO) / 128;  // v and dout of the group come into L2 meanwhile, a line of 128 bytes a thread
    const int pr = tid % (C * LN) / LN;
    if (tid < 2 * C * LN && c0 + pr < end) {
      const IO* x = static_cast<const IO*>(tid < C * LN ? a.v : a.dout) + ((size_t)(c0 + pr) * a.nv + hq * group) * DV + tid % LN * (128 / sizeof(IO));
      for (int h = 0; h < group; ++h) asm volatile("prefetch.global.L2 [%0];" ::"l"(x + (size_t)h * DV));
    }
    __syncthreads();
    store_qk<DK>(kv, kn, l2, rows, sm + L::kK, qrec + QR::kK, qrec + QR::kKs, kf, qfl, qfl + 2 * C, tid);
    store_qk<DK>(qv, qn, l2, rows + C, sm + L::kQ, qrec + QR::kQ, qrec + QR::kQs, qf, qfl + C, qfl + 3 * C, tid);
  }
  __syncthreads();
  // warp: rows 16 wr .., columns 16 wc .. of the [C][C] products; blocks above the diagonal are zero
  const int wr = 16 * (warp & 3), wc = 16 * (warp >> 2), r0 = wr + ln.g, i0 = wc + 2 * ln.t;
  float kk[2][4] = {}, qk[2][4] = {};
  if (wc <= wr) {
#pragma unroll 2
    for (int k = 0; k < DK; k += 16) {
      uint32_t kh[4], kl[4], qh[4], ql[4], bh[4], bl[4];
      pair_a<RK>(kh, kl, K, wr, k, ln);
      pair_a<RK>(qh, ql, Q, wr, k, ln);
      pair_b<RK>(bh, bl, K, wc, k, ln);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mma_pair(kk[j], kh, kl, bh + 2 * j, bl + 2 * j);
        mma_pair(qk[j], qh, ql, bh + 2 * j, bl + 2 * j);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = kf[i0 + 8 * j + (e & 1)];
        kk[j][e] *= kf[r0 + 8 * (e >> 1)] * f;
        qk[j][e] *= qf[r0 + 8 * (e >> 1)] * f;
      }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {  // zero above the diagonal
    const int at = ((wr >> 4) * 8 + (wc >> 3) + j) * 32 + lane;
    reinterpret_cast<float4*>(qrec + QR::kKk)[at] = make_float4(kk[j][0], kk[j][1], kk[j][2], kk[j][3]);
    reinterpret_cast<float4*>(qrec + QR::kQk)[at] = make_float4(qk[j][0], qk[j][1], qk[j][2], qk[j][3]);
  }

  for (int h = hq * group; h < (hq + 1) * group; ++h) {
    uint8_t* rec = rec_at<DK, DV>(a, slot, h);
    float* rf = reinterpret_cast<float*>(rec + R::kF);
    constexpr int N = C * DV / 8 / kThreads, LV = DV / 8;
    float vv[N][8], ov[N][8], vtop = 0.f, otop = 0.f;
#pragma unroll
    for (int p = 0; p < N; ++p) {
      const int r = (p * kThreads + tid) / LV, c = 8 * (tid % LV);
      const bool valid = c0 + r < end;
      const size_t at = ((size_t)(valid ? c0 + r : c0) * a.nv + h) * DV + c;
      load8<IO>(static_cast<const IO*>(a.v) + at, valid, vv[p]);
      load8<IO>(static_cast<const IO*>(a.dout) + at, valid, ov[p]);
    }
    float gv = 0.f, bv = 0.f;
    if (tid < C && c0 + tid < end) load_gate(a, (size_t)(c0 + tid) * a.nv + h, h, gv, bv);
#pragma unroll
    for (int p = 0; p < N; ++p) {
      vtop = fmaxf(vtop, top8(vv[p]));
      otop = fmaxf(otop, top8(ov[p]));
    }
    vtop = warp_top(vtop);
    otop = warp_top(otop);
    __syncthreads();  // the head before is done with the tiles
    if (lane == 0) {
      tops[warp] = vtop;
      tops[16 + warp] = otop;
    }
    if (tid < C) {
      gc[tid] = gv;
      bt[tid] = bv;
    }
    __syncthreads();
    if (warp == 0) cumsum_chunk(gc, gl, lane);
    float vs, vinv, os, oinv;
    pow2_factor(top16(tops, lane), vs, vinv);
    pow2_factor(top16(tops + 16, lane), os, oinv);
#pragma unroll
    for (int p = 0; p < N; ++p) {
      const int r = (p * kThreads + tid) / LV, c = 8 * (tid % LV);
      uint4 hi, lo;
      pair8(vv[p], vs, hi, lo);
      *reinterpret_cast<uint4*>(sm + L::kV + pair_at<RV>(r, c)) = hi;
      *reinterpret_cast<uint4*>(sm + L::kV + pair_at<RV>(r, c) + 16 * RV) = lo;
      pair8(ov[p], os, hi, lo);
      const int at = (c >> 6) * (4 * C * 64) + pair_at<128>(r, c & 63);
      *reinterpret_cast<uint4*>(sm + L::kO + at) = hi;
      *reinterpret_cast<uint4*>(sm + L::kO + at + 16 * 128) = lo;
      *reinterpret_cast<uint4*>(rec + R::kO + at) = hi;
      *reinterpret_cast<uint4*>(rec + R::kO + at + 16 * 128) = lo;
    }
    __syncthreads();
    float p[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + 8 * (e >> 1), i = i0 + 8 * j + (e & 1);
        const float gamma = i <= r ? decay(gc, r, i) : 0.f;  // masked before exp
        A[r * TP + i] = i < r ? -bt[r] * (kk[j][e] * gamma) : 0.f;
        p[j][e] = i <= r ? a.scale * qk[j][e] * gamma : 0.f;
      }
    __syncthreads();
    if (tid >= 128 && tid < 128 + C) {  // while warps 0-3 substitute
      const int i = tid - 128;
      const float e = expf(gc[i] + gl[i]);
      wf[i] = bt[i] * e * kf[i];
      qe[i] = a.scale * e * qf[i];
      rf[R::fGc + i] = gc[i];
      rf[R::fGc + C + i] = gl[i];
      rf[R::fBeta + i] = bt[i];
      rf[R::fKw + i] = decay(gc, C - 1, i) * kf[i];
      if (i == C - 1) {
        rf[R::fScal + kScalGl] = e;
        rf[R::fScal + kScalDo] = oinv;
      }
    }
    invert_chunk<false>(A, Y, warp, lane);
    {  // pairs of T, T diag(b) and P, each under one factor
      float2 t[2][2], tb[2][2];
      float top[3] = {0.f, 0.f, 0.f}, f[3], inv[3];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = r0 + 8 * e, i = i0 + 8 * j;
          t[j][e] = *reinterpret_cast<const float2*>(A + r * TP + i);
          tb[j][e] = make_float2(t[j][e].x * bt[i], t[j][e].y * bt[i + 1]);
          top[0] = fmaxf(top[0], fmaxf(fabsf(t[j][e].x), fabsf(t[j][e].y)));
          top[1] = fmaxf(top[1], fmaxf(fabsf(tb[j][e].x), fabsf(tb[j][e].y)));
          top[2] = fmaxf(top[2], fmaxf(fabsf(p[j][2 * e]), fabsf(p[j][2 * e + 1])));
        }
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        top[m] = warp_top(top[m]);
        if (lane == 0) tops[16 * m + warp] = top[m];
      }
      __syncthreads();
#pragma unroll
      for (int m = 0; m < 3; ++m) pow2_factor(top16(tops + 16 * m, lane), f[m], inv[m]);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int at = pair_at<RC>(r0 + 8 * e, i0 + 8 * j);
          uint32_t hi, lo;
          pair2(t[j][e].x, t[j][e].y, f[0], hi, lo);
          *reinterpret_cast<uint32_t*>(rec + R::kT + at) = hi;
          *reinterpret_cast<uint32_t*>(rec + R::kT + at + 16 * RC) = lo;
          pair2(tb[j][e].x, tb[j][e].y, f[1], hi, lo);
          sts32(TB + at, hi);
          sts32(TB + at + 16 * RC, lo);
          pair2(p[j][2 * e], p[j][2 * e + 1], f[2], hi, lo);
          sts32(P + at, hi);
          sts32(P + at + 16 * RC, lo);
        }
      if (tid == 0) rf[R::fScal + kScalT] = inv[0];
      vinv *= inv[1];  // of U and Y from here on
      oinv *= inv[2];
    }
    __syncthreads();
    ln.again();
    {  // W = T diag(b e) k_hat: this warp's 16 rows, a quarter of the columns; pairs under a factor for every row, since
       // the rows fall with the decay up to their token, and the walk multiplies that out again
      constexpr int NT = DK / 32;
      const int n0 = (DK / 4) * (warp >> 2);
      float t[4][2][4], top[2] = {0.f, 0.f}, f[2], inv[2], x[NT][4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // t[k][m]: columns 16 k + 8 m + 2 t, + 1 of rows g and g + 8
            const int i = 16 * k + 8 * m + 2 * ln.t;
            const float2 v = *reinterpret_cast<const float2*>(A + (wr + ln.g + 8 * e) * TP + i);
            t[k][m][2 * e] = v.x * wf[i];
            t[k][m][2 * e + 1] = v.y * wf[i + 1];
            top[e] = fmaxf(top[e], fmaxf(fabsf(t[k][m][2 * e]), fabsf(t[k][m][2 * e + 1])));
          }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
        pow2_factor(top[e], f[e], inv[e]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t ah[4], al[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pair2(t[k][e >> 1][2 * (e & 1)], t[k][e >> 1][2 * (e & 1) + 1], f[e & 1], ah[e], al[e]);
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          uint32_t bh[4], bl[4];
          pair_b_t<RK>(bh, bl, K, n0 + 8 * j, 16 * k, ln);
          mma_pair(x[j], ah, al, bh, bl);
          mma_pair(x[j + 1], ah, al, bh + 2, bl + 2);
        }
      }
      top[0] = top[1] = 0.f;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[j][e] *= inv[e >> 1];
          top[e >> 1] = fmaxf(top[e >> 1], fabsf(x[j][e]));
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
        if (ln.t == 0) rows[(warp >> 2) * C + wr + ln.g + 8 * e] = top[e];
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = wr + ln.g + 8 * e;
        pow2_factor(fmaxf(fmaxf(rows[r], rows[C + r]), fmaxf(rows[2 * C + r], rows[3 * C + r])), f[e], inv[e]);
        if (warp < 4 && ln.t == 0) rf[R::fWr + r] = inv[e];
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint8_t* dst = rec + R::kW + pair_at<RK>(wr + ln.g + 8 * e, n0 + 8 * j + 2 * ln.t);
          uint32_t hi, lo;
          pair2(x[j][2 * e], x[j][2 * e + 1], f[e], hi, lo);
          *reinterpret_cast<uint32_t*>(dst) = hi;
          *reinterpret_cast<uint32_t*>(dst + 16 * RK) = lo;
        }
    }
    // U^T = V^T (T diag(b))^T and Y^T = dO^T P, 16 columns of Dv a warp, and the fragments of (diag(qe) dO)^T
    if (warp < DV / 8) {
      const bool isY = warp >= DV / 16;
      const int u = isY ? warp - DV / 16 : warp, m0 = 16 * u;
      const uint32_t Oh = O + (m0 >> 6) * (4 * C * 64);
      float x[8][4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t ah[4], al[4];
        if (isY) pair_a_t<128>(ah, al, Oh, m0 & 63, 16 * k, ln); else pair_a_t<RV>(ah, al, V, m0, 16 * k, ln);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t bh[4], bl[4];
          if (isY) pair_b_t<RC>(bh, bl, P, 16 * j, 16 * k, ln); else pair_b<RC>(bh, bl, TB, 16 * j, 16 * k, ln);
          mma_pair(x[2 * j], ah, al, bh, bl);
          mma_pair(x[2 * j + 1], ah, al, bh + 2, bl + 2);
        }
      }
      const float f = isY ? oinv : vinv;
      float4* dst = reinterpret_cast<float4*>(rec + (isY ? R::kX : R::kV)) + u * 256 + lane;
#pragma unroll
      for (int j = 0; j < 8; ++j) dst[32 * j] = make_float4(x[j][0] * f, x[j][1] * f, x[j][2] * f, x[j][3] * f);
      if (isY) {
        float top[2] = {0.f, 0.f}, fq[2], inv[2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // x is free: (diag(s e) dO)^T over Q16's factors, in units of dO's factor
          uint32_t ah[4], al[4];
          pair_a_t<128>(ah, al, Oh, m0 & 63, 16 * k, ln);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 o = both2(ah[e], al[e]), q = *reinterpret_cast<const float2*>(qe + 16 * k + 8 * (e >> 1) + 2 * ln.t);
            float* d = &x[2 * k + (e >> 1)][2 * (e & 1)];
            d[0] = o.x * q.x;
            d[1] = o.y * q.y;
            top[e & 1] = fmaxf(top[e & 1], fmaxf(fabsf(d[0]), fabsf(d[1])));
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
          top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
          pow2_factor(top[e], fq[e], inv[e]);
          if (ln.t == 0) rf[R::fOq + m0 + ln.g + 8 * e] = inv[e] / os;
        }
        uint4* od = reinterpret_cast<uint4*>(rec + R::kOq) + u * 128 + lane;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) pair2(x[2 * k + (e >> 1)][2 * (e & 1)], x[2 * k + (e >> 1)][2 * (e & 1) + 1], fq[e & 1], hi[e], lo[e]);
          od[32 * k] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          od[DV * 8 + 32 * k] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ 2. states
// One block per (sequence, v-head, direction, 64 columns of Dv).  Two warps, w and w + 4, share 16 columns of Dv, and
// each keeps half of the columns of Dk: x is the sum of what both have, and each forms V' for itself.

constexpr int kStateSlices = 4;
constexpr int kStateThreads = 64 * kStateSlices;

template <int DK>
struct StateSmem {
  static constexpr size_t kTile = 4 * C * DK;            // a pair image: W, K16 and (backwards) Q16
  static constexpr size_t kStage = 3 * kTile + 8 * C;    // and kw, wr
  static constexpr size_t kX = 2 * kStage;               // float4 [8 warps][8][32] a warp's part of x
  static constexpr size_t kTop = kX + 8 * 4096;          // fp32 [2][8] the warps' largest of the state
  static constexpr size_t kBar = kTop + 64;
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
// x[NT] (8 NT columns from n0) += (hi + lo) B[16 k .. + 15], B a pair image [n][k] (kT: [k][n])
template <int RB, bool kT, int NT>
__device__ __forceinline__ void mma_pairs(float (&x)[NT][4], const uint32_t* hi, const uint32_t* lo, uint32_t img, int n0, int k,
                                          const Lane& ln) {
#pragma unroll
  for (int j = 0; j < NT / 2; ++j) {
    uint32_t bh[4], bl[4];
    if (kT) pair_b_t<RB>(bh, bl, img, n0 + 16 * j, 16 * k, ln); else pair_b<RB>(bh, bl, img, n0 + 16 * j, 16 * k, ln);
    mma_pair(x[2 * j], hi, lo, bh, bl);
    mma_pair(x[2 * j + 1], hi, lo, bh + 2, bl + 2);
  }
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <int DK, int DV, bool kBackward>
__device__ __forceinline__ void walk(const BwdArgs& a, uint8_t* sm, int n, int h, int col0) {
  using L = StateSmem<DK>;
  using R = Rec<DK, DV>;
  using QR = QkRec<DK>;
  constexpr int ND = DK / 16, RB = 2 * DK, RC = 2 * C;  // ND: 8-column tiles of a warp's half of Dk
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int half = warp >> 2, d0 = DK / 2 * half;
  const int slice = col0 / 16 + (warp & 3), c = 16 * slice + g;  // this thread's columns of Dv: c and c + 8
  const int hq = h / (a.nv / a.nqk);
  Lane ln(lane);
  float4* xs = reinterpret_cast<float4*>(sm + L::kX);
  float* tops = reinterpret_cast<float*>(sm + L::kTop);
  auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory"); };  // warps w and w + 4
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::kBar);
  int64_t start, end;
  seq_bounds(a, n, start, end);
  const int64_t chunks = (end - start + C - 1) / C, slot0 = start / C + n;

  float s[ND][4];  // S^T or dS^T: rows c, c + 8, columns d = d0 + 8 j + 2 t, + 1
  const float* init = kBackward ? a.ds_final : a.s0;
  const size_t state_off = ((size_t)n * a.nv + h) * (size_t)DK * DV;
#pragma unroll
  for (int j = 0; j < ND; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s[j][e] = init ? init[state_off + (size_t)(d0 + 8 * j + 2 * t + (e & 1)) * DV + c + 8 * (e >> 1)] : 0.f;

  auto slot_of = [&](int64_t i) { return slot0 + (kBackward ? chunks - 1 - i : i); };
  auto fetch = [&](int64_t i) {  // by one thread
    if (i >= chunks) return;
    uint8_t* st = sm + (i & 1) * L::kStage;
    const uint8_t* rec = rec_at<DK, DV>(a, slot_of(i), h);
    constexpr uint32_t tiles = (kBackward ? 2 : 1) * L::kTile;
    ptx::mbar_arrive_expect_tx(bar + (i & 1), (uint32_t)(L::kTile + tiles + 8 * C));
    bulk_copy(st, rec + R::kW, L::kTile, bar + (i & 1));
    bulk_copy(st + L::kTile, qk_at<DK, DV>(a, slot_of(i), hq) + QR::kK, tiles, bar + (i & 1));  // Q16 stands behind K16
    bulk_copy(st + 3 * L::kTile, rec + R::kF + 4 * R::fKw, 8 * C, bar + (i & 1));  // and the factors of W behind it
  };
  if (tid == 0) {
    ptx::mbar_init(bar, 1);
    ptx::mbar_init(bar + 1, 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();
  // the largest element of the block's state; also the barrier behind which a chunk's stage is free
  auto join_top = [&](int64_t i, bool ok) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < ND; ++j) m = fmaxf(fmaxf(m, fmaxf(fabsf(s[j][0]), fabsf(s[j][1]))), fmaxf(fabsf(s[j][2]), fabsf(s[j][3])));
    m = warp_top(m);
    if (lane == 0) tops[8 * (i & 1) + warp] = m;
    return __syncthreads_or(!ok);
  };
  if (tid == 0) {
    fetch(0);
    fetch(1);
  }
  join_top(1, true);
  for (int64_t i = 0; i < chunks; ++i) {
    uint8_t* rec = rec_at<DK, DV>(a, slot_of(i), h);
    float* rf = reinterpret_cast<float*>(rec + R::kF);
    const float gl = rf[R::fScal + kScalGl];
    const float4* uw = reinterpret_cast<const float4*>(rec + (kBackward ? R::kX : R::kV)) + slice * 256 + lane;
    float4 u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = uw[32 * j];
    if (i + 1 < chunks) {  // the next chunk's U^T, or Y^T and half of Oq each, a line a lane
      const uint8_t* nx = rec_at<DK, DV>(a, slot_of(i + 1), h);
      if (half == 0) prefetch_l2(nx + (kBackward ? R::kX : R::kV) + 4096 * slice + 128 * lane);
      if (half == 1 && lane < 8) prefetch_l2(nx + R::kF + min((size_t)(128 * lane), (size_t)(4 * R::kFloats - 4)));
      if (kBackward && half == 1) prefetch_l2(nx + R::kOq + (lane >> 4) * (2 * C * DV) + 2048 * slice + 128 * (lane & 15));
    }
    // the state as this chunk meets it
    float top[2], sf, sinv;
    pow2_factor(warp_top(tops[8 * ((i + 1) & 1) + (lane & 7)]), sf, sinv);
    if (t == 0 && half == 0) rf[(kBackward ? R::fD : R::fS) + c] = rf[(kBackward ? R::fD : R::fS) + c + 8] = sinv;
    const bool ok = ptx::mbar_wait_bounded(bar + (i & 1), (uint32_t)((i >> 1) & 1), kWaitLimitNs);
    const uint8_t* st = sm + (i & 1) * L::kStage;
    const uint32_t W = ptx::smem_u32(st), K = W + (uint32_t)L::kTile, Q = K + (uint32_t)L::kTile;
    const float *kw = reinterpret_cast<const float*>(st + 3 * L::kTile), *wr = kw + C;
    // x = S^T W^T (forwards) or dS'^T K^T (backwards), [16 x C]; the operand is also what the gradients read: two
    // steps of 16 columns are one vector a lane
    float x[8][4] = {};
    uint8_t* img = rec + (kBackward ? R::kD : R::kS);
#pragma unroll
    for (int k2 = 0; k2 < ND / 4; ++k2) {
      uint32_t hi[2][4], lo[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        pair_frag(s[4 * k2 + 2 * m], s[4 * k2 + 2 * m + 1], sf, sf, hi[m], lo[m]);
        mma_pairs<RB, false, 8>(x, hi[m], lo[m], kBackward ? K : W, 0, d0 / 16 + 2 * k2 + m, ln);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint8_t* dst = img + pair_at<RB>(c + 8 * e, d0 + 32 * k2 + 8 * t);
        *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0][e], hi[0][2 + e], hi[1][e], hi[1][2 + e]);
        *reinterpret_cast<uint4*>(dst + 16 * RB) = make_uint4(lo[0][e], lo[0][2 + e], lo[1][e], lo[1][2 + e]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) xs[256 * warp + 32 * j + lane] = make_float4(x[j][0], x[j][1], x[j][2], x[j][3]);
    pair_sync();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 y = xs[256 * (warp ^ 4) + 32 * j + lane];
      x[j][0] += y.x;
      x[j][1] += y.y;
      x[j][2] += y.z;
      x[j][3] += y.w;
    }
    // forwards V'^T = U^T - x diag(wr), backwards dV'^T = Y^T + x diag(kw); stored over U^T, Y^T (these warps' 4 KB, read by both)
    top[0] = top[1] = 0.f;
    float vf[2], vinv[2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float2 f = *reinterpret_cast<const float2*>((kBackward ? kw : wr) + 8 * j + 2 * t);
      if (!kBackward) f = make_float2(-f.x, -f.y);
      x[j][0] = fmaf(x[j][0] * sinv, f.x, u[j].x);
      x[j][1] = fmaf(x[j][1] * sinv, f.y, u[j].y);
      x[j][2] = fmaf(x[j][2] * sinv, f.x, u[j].z);
      x[j][3] = fmaf(x[j][3] * sinv, f.y, u[j].w);
      top[0] = fmaxf(top[0], fmaxf(fabsf(x[j][0]), fabsf(x[j][1])));
      top[1] = fmaxf(top[1], fmaxf(fabsf(x[j][2]), fabsf(x[j][3])));
    }
    row_factors(top, vf, vinv);
    if (t == 0 && half == 0) {
      rf[(kBackward ? R::fDV : R::fV) + c] = vinv[0];
      rf[(kBackward ? R::fDV : R::fV) + c + 8] = vinv[1];
    }
    uint32_t vh[4][4], vl[4][4];
    img = rec + (kBackward ? R::kX : R::kV);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      pair_frag(x[2 * k], x[2 * k + 1], vf[0], vf[1], vh[k], vl[k]);
      if ((k >> 1) != half) continue;  // each warp stores half of the columns
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint8_t* dst = img + pair_at<RC>(c + 8 * (e & 1), 16 * k + 8 * (e >> 1) + 2 * t);
        *reinterpret_cast<uint32_t*>(dst) = vh[k][e];
        *reinterpret_cast<uint32_t*>(dst + 16 * RC) = vl[k][e];
      }
    }
    // the operand of the update is V' diag(kw) or dV' diag(wr), with factors of its own
    top[0] = top[1] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 w = *reinterpret_cast<const float2*>((kBackward ? wr : kw) + 8 * j + 2 * t);
      x[j][0] *= w.x;
      x[j][1] *= w.y;
      x[j][2] *= w.x;
      x[j][3] *= w.y;
      top[0] = fmaxf(top[0], fmaxf(fabsf(x[j][0]), fabsf(x[j][1])));
      top[1] = fmaxf(top[1], fmaxf(fabsf(x[j][2]), fabsf(x[j][3])));
    }
    row_factors(top, vf, vinv);
#pragma unroll
    for (int k = 0; k < 4; ++k) pair_frag(x[2 * k], x[2 * k + 1], vf[0], vf[1], vh[k], vl[k]);
    // forwards S^T = e_last S^T + (V' diag(kw))^T K, backwards dS^T = e_last dS'^T + (s diag(e) dO)^T Q - (dV' diag(wr))^T W
    const float f0 = kBackward ? -vinv[0] : vinv[0], f1 = kBackward ? -vinv[1] : vinv[1];
    {
      float y[ND][4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_pairs<RB, true, ND>(y, vh[k], vl[k], kBackward ? W : K, d0, k, ln);
#pragma unroll
      for (int j = 0; j < ND; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = fmaf(e < 2 ? f0 : f1, y[j][e], gl * s[j][e]);
    }
    if (kBackward) {
      const uint4* ow = reinterpret_cast<const uint4*>(rec + R::kOq) + slice * 128 + lane;
      const float o0 = rf[R::fOq + c], o1 = rf[R::fOq + c + 8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 h4 = ow[32 * k], l4 = ow[DV * 8 + 32 * k];
        vh[k][0] = h4.x; vh[k][1] = h4.y; vh[k][2] = h4.z; vh[k][3] = h4.w;
        vl[k][0] = l4.x; vl[k][1] = l4.y; vl[k][2] = l4.z; vl[k][3] = l4.w;
      }
      float y[ND][4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_pairs<RB, true, ND>(y, vh[k], vl[k], Q, d0, k, ln);
#pragma unroll
      for (int j = 0; j < ND; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = fmaf(e < 2 ? o0 : o1, y[j][e], s[j][e]);
    }
    if (join_top(i, ok)) {  // a copy never came: report it, wait once more for what is in flight, and leave
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
        a.ds0[state_off + (size_t)(d0 + 8 * j + 2 * t + (e & 1)) * DV + c + 8 * (e >> 1)] = s[j][e];
  }
}

// blockIdx.x: direction and 64-column slice, y: v-head, z: sequence
template <int DK, int DV>
__global__ void __launch_bounds__(kStateThreads) states_kernel(BwdArgs a) {
  let_next_begin();
  wait_for_previous();
  extern __shared__ __align__(128) uint8_t sm[];
  const int col0 = 16 * kStateSlices * (blockIdx.x >> 1);
  if (blockIdx.x & 1)
    walk<DK, DV, true>(a, sm, blockIdx.z, blockIdx.y, col0);
  else
    walk<DK, DV, false>(a, sm, blockIdx.z, blockIdx.y, col0);
}

// ------------------------------------------------------------------ 3. gradients
// One block of 16 warps per (slot, qk-head), which takes its v-heads in turn, and of each 64 columns of Dv at a time:
//   1. all warps: dX^T = dV'^T T; V'^T to one factor for all its rows
//   2. warps 0-7: dO S^T and dV; warps 8-15: V' dS'^T, then dX S^T; warps 0-9: dA and dP, a 16 x 16 block of the
//      triangle each; all: <S, dS'>
// and after a v-head's last columns
//   3. warps 0-9: N and B
//   4. warps 0-7: N K, and keep dq; warps 8-15: N^T Q + (B + B^T) K, and keep dk

template <int DK, int DV>
struct GradSmem {
  using R = Rec<DK, DV>;
  static constexpr size_t kHalf = 4 * 64 * C;                 // a pair image of 64 rows of 64
  static constexpr size_t kK = 0;                             // pair images of K16, Q16 (columns by swap32), and their floats
  static constexpr size_t kKBytes = QkRec<DK>::kLoad;
  static constexpr size_t kS = kK + kKBytes;                  // 64 rows of S^T
  static constexpr size_t kD = kS + 4 * 64 * DK;              // of dS'^T
  static constexpr size_t kV = kD + 4 * 64 * DK;              // of V'^T
  static constexpr size_t kX = kV + kHalf;                    // of dV'^T; then N
  static constexpr size_t kO = kX + kHalf;                    // 64 columns of dO; then B
  static constexpr size_t kDx = kO + kHalf;                   // 64 rows of dX^T
  static constexpr size_t kT = kDx + kHalf;                   // T
  static constexpr size_t kF = kT + kHalf;                    // the record's floats up to fKw
  static constexpr size_t kFBytes = 4 * R::fKw;
  static constexpr size_t kRed = kF + kFBytes;                // fp32 [3][4][C] rows' dots by column block
  static constexpr size_t kRedA = kRed + 48 * C;              // fp32 [10][C] row sums: through A and P by column block (dgc, dbeta), dX V (two)
  static constexpr size_t kCol = kRedA + 40 * C;              // fp32 [4][C] column sums by row block
  static constexpr size_t kDot = kCol + 16 * C;               // fp32 [16] <S, dS'> by warp; [2][16] largest of N and B
  static constexpr size_t kBar = kDot + 192;
  static constexpr size_t kBytes = kBar + 16;
  static_assert(kS % 128 == 0 && kF % 16 == 0 && kFBytes % 16 == 0, "images and bulk copies");
  static_assert(kBytes <= 232448, "shared memory budget");
};

// x[2][NT] (32 rows from m0, 8 NT columns from n0) += A B over k in [16 K0, 16 K1); pair images A [m][k] (kAT: [k][m]), B [k][n]
template <int NT, int K0, int K1, int RA, bool kAT, int RB>
__device__ __forceinline__ void gemm32(float (&x)[2][NT][4], uint32_t A, int m0, uint32_t B, int n0, const Lane& l) {
#pragma unroll 1
  for (int k = K0; k < K1; ++k) {
    uint32_t ah[2][4], al[2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (kAT) pair_a_t<RA>(ah[m], al[m], A, m0 + 16 * m, 16 * k, l); else pair_a<RA>(ah[m], al[m], A, m0 + 16 * m, 16 * k, l);
    }
#pragma unroll
    for (int j = 0; j < NT; j += 2) {
      uint32_t bh[4], bl[4];
      pair_b_t<RB>(bh, bl, B, n0 + 8 * j, 16 * k, l);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        mma_pair(x[m][j], ah[m], al[m], bh, bl);
        mma_pair(x[m][j + 1], ah[m], al[m], bh + 2, bl + 2);
      }
    }
  }
}

template <int RB> __device__ __forceinline__ float2 lds_pair(uint32_t img, int r, int col) {
  const uint32_t p = pair_word<RB>(img, r, col);
  return both2(lds32(p), lds32(p + 16 * RB));
}

// Rows' dots of x (as gemm32 leaves it) with a pair image Y, this thread's part of row m0 + 16 m + 8 e + g in dot[m][e];
// and sum += f x by rows.
template <int NT, int RB>
__device__ __forceinline__ void take(const float (&x)[2][NT][4], uint32_t Y, int m0, int n0, const float (&f)[2][2],
                                     float (&sum)[2][NT][4], float (&dot)[2][2], const Lane& l) {
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = m0 + 16 * m + 8 * e + l.g;
      dot[m][e] = 0.f;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float2 y = lds_pair<RB>(Y, r, n0 + 8 * j + 2 * l.t);
        dot[m][e] = fmaf(x[m][j][2 * e], y.x, fmaf(x[m][j][2 * e + 1], y.y, dot[m][e]));
        sum[m][j][2 * e] = fmaf(f[m][e], x[m][j][2 * e], sum[m][j][2 * e]);
        sum[m][j][2 * e + 1] = fmaf(f[m][e], x[m][j][2 * e + 1], sum[m][j][2 * e + 1]);
      }
    }
}

// A row's sum over the quad of lanes, added to dst[row] by one of them (first: put there)
__device__ __forceinline__ void put_row(float v, float* dst, int t, bool first) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  if (t == 0) *dst = first ? v : *dst + v;
}

// Every row of `rows` rows of a pair image (RB bytes each) times its factor over `top`; factors f of its first row on
template <int RB>
__device__ __forceinline__ void rescale(uint8_t* img, const float* f, float top, int tid) {
  constexpr int NV = 64 * RB * 2 / 16;
#pragma unroll
  for (int x = 0; x < NV / kThreads; ++x) {
    const int v = x * kThreads + tid, at = 16 * v, r = at / (32 * RB) * 16 + at % (16 * RB) / RB;
    const float y = f[r] / top;  // a power of two
    const __half2 s = __floats2half2_rn(y, y);
    uint4* p = reinterpret_cast<uint4*>(img) + v;
    uint4 w = *p;
    __half2* h = reinterpret_cast<__half2*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __hmul2(h[i], s);
    *p = w;
  }
}

template <int DK, int DV, typename IO>
__global__ void __launch_bounds__(kThreads, 1) grads_kernel(BwdArgs a) {
  wait_for_previous();
  using L = GradSmem<DK, DV>;
  using R = Rec<DK, DV>;
  using QR = QkRec<DK>;
  extern __shared__ __align__(128) uint8_t sm[];
  constexpr int NT = DK / 32;        // 8-column tiles of a warp's quarter of Dk
  constexpr int RK = 2 * DK, RC = 2 * C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Lane ln(lane);
  const bool first = warp < 8;       // warps 0-7, which keep dq
  const int w8 = warp & 7;
  const int hq = blockIdx.x, group = a.nv / a.nqk, h0 = hq * group;
  const int64_t slot = grid_slot();
  if (slot >= a.total_tokens / C + a.num_seqs) return;
  int64_t c0, end;
  if (!chunk_at(a, slot, c0, end)) return;
  const int rows = (int)min((int64_t)C, end - c0);
  const uint8_t* qrec = qk_at<DK, DV>(a, slot, hq);
  const uint32_t base = ptx::smem_u32(sm);
  const uint32_t K = base + L::kK, Q = K + 4 * C * DK, S = base + L::kS, D = base + L::kD, V = base + L::kV, X = base + L::kX;
  const uint32_t O = base + L::kO, Dx = base + L::kDx, T = base + L::kT, N = X, B = O;
  const float *kf = reinterpret_cast<const float*>(sm + L::kK + 8 * C * DK), *qf = kf + C, *kn = qf + C, *qn = kn + C;
  const float* rf = reinterpret_cast<const float*>(sm + L::kF);
  float *red = reinterpret_cast<float*>(sm + L::kRed), *reda = reinterpret_cast<float*>(sm + L::kRedA);
  float *col = reinterpret_cast<float*>(sm + L::kCol), *dots = reinterpret_cast<float*>(sm + L::kDot), *ntop = dots + 16;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::kBar);
  if (tid == 0) {
    ptx::mbar_init(bar, 1);
    ptx::fence_mbar_init();
  }
  // a warp's 32 rows and quarter of the columns of Dk for products with the state
  const int m0 = 32 * (w8 & 1), n0 = (DK / 4) * (w8 >> 1);
  // of [C][C], warps 0-9 have block (rb, cb) of the triangle; what they leave of the sums is zero
  const bool tri = warp < 10;
  const int rb = warp < 1 ? 0 : warp < 3 ? 1 : warp < 6 ? 2 : 3, cb = warp - rb * (rb + 1) / 2;
  for (int i = tid; i < 4 * C; i += kThreads) {
    const int q = i / C, r = i % C;      // column block or row block q, row or column r
    if (r / 16 < q) reda[i] = reda[4 * C + i] = 0.f;
    if (r / 16 > q) col[i] = 0.f;
  }
  float dA[2][4], dP[2][4];
  float sum[2][NT][4] = {};              // qf dq_hat (warps 0-7) or kf dk_hat (warps 8-15), over the group's v-heads
  bool quit = false;
  uint32_t it = 0;
  for (int h = h0; h < h0 + group && !quit; ++h) {
    float s_dot = 0.f;
    for (int v0 = 0; v0 < DV; v0 += 64, ++it) {
      ptx::fence_proxy_async_smem();  // tiles were rewritten in place before a copy comes over them
      __syncthreads();                // and are done with
      if (tid == 0) {
        const uint8_t* rec = rec_at<DK, DV>(a, slot, h);
        const bool k = it == 0, t = v0 == 0;
        ptx::mbar_arrive_expect_tx(bar, (uint32_t)((k ? L::kKBytes : 0) + 8 * 64 * DK + 3 * L::kHalf + (t ? L::kHalf + L::kFBytes : 0)));
        if (t) bulk_copy(sm + L::kF, rec + R::kF, L::kFBytes, bar);
        bulk_copy(sm + L::kX, rec + R::kX + 4 * (size_t)v0 * C, L::kHalf, bar);
        if (t) bulk_copy(sm + L::kT, rec + R::kT, L::kHalf, bar);
        bulk_copy(sm + L::kV, rec + R::kV + 4 * (size_t)v0 * C, L::kHalf, bar);
        bulk_copy(sm + L::kS, rec + R::kS + 4 * (size_t)v0 * DK, 4 * 64 * DK, bar);
        bulk_copy(sm + L::kD, rec + R::kD + 4 * (size_t)v0 * DK, 4 * 64 * DK, bar);
        bulk_copy(sm + L::kO, rec + R::kO + 4 * (size_t)v0 * C, L::kHalf, bar);
        if (k) bulk_copy(sm + L::kK, qrec + QR::kKs, L::kKBytes, bar);
      }
      const bool ok = ptx::mbar_wait_bounded(bar, it & 1, kWaitLimitNs);
      ln.again();
      // ---- 1.
      const float mS = rf[R::fS + v0], mD = rf[R::fD + v0];
      float mV, mX;
      {
        auto top = [&](const float* f) {
          float m = 0.f;
          for (int i = lane; i < DV; i += 32) m = fmaxf(m, f[i]);
          return warp_top(m);
        };
        mV = top(rf + R::fV);
        mX = top(rf + R::fDV);
      }
      rescale<RC>(sm + L::kV, rf + R::fV + v0, mV, tid);
      {
        const int cb = 16 * (warp & 3), ib = 16 * (warp >> 2);
        // T and dV' are below 2^8, their products' sum below 2^22
        const float f0 = rf[R::fDV + v0 + cb + ln.g] / mX * 0x1p-8f, f1 = rf[R::fDV + v0 + cb + ln.g + 8] / mX * 0x1p-8f;
        float x[2][4] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t ah[4], al[4], bh[4], bl[4];
          pair_a<RC>(ah, al, X, cb, 16 * k, ln);
          pair_b_t<RC>(bh, bl, T, ib, 16 * k, ln);
          mma_pair(x[0], ah, al, bh, bl);
          mma_pair(x[1], ah, al, bh + 2, bl + 2);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t at = pair_word<RC>(Dx, cb + ln.g + 8 * e, ib + 8 * j + 2 * ln.t);
            uint32_t hi, lo;
            pair2(x[j][2 * e], x[j][2 * e + 1], e ? f1 : f0, hi, lo);
            sts32(at, hi);
            sts32(at + 16 * RC, lo);
          }
      }
      mX *= 0x1p8f * rf[R::fScal + kScalT];  // of dX from here on
      quit = __syncthreads_or(!ok);
      if (quit) break;
      ln.again();
      // ---- 2.
      const float oinv = rf[R::fScal + kScalDo];
      const bool head = v0 == 0;
      {  // <S, dS'>: the diagonal of S^T dS', 16 columns of Dv and a quarter of Dk a warp
        constexpr int KS = DK / 64;
        const int cb = 16 * (warp & 3), k0 = KS * (warp >> 2);
        float x[2][4] = {};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t ah[4], al[4], bh[4], bl[4];
          pair_a<RK>(ah, al, S, cb, 16 * (k0 + k), ln);
          pair_b<RK>(bh, bl, D, cb, 16 * (k0 + k), ln);
          mma_pair(x[0], ah, al, bh, bl);
          mma_pair(x[1], ah, al, bh + 2, bl + 2);
        }
        s_dot = fmaf(mS * mD, (2 * ln.t == ln.g ? x[0][0] + x[1][2] : 0.f) + (2 * ln.t + 1 == ln.g ? x[0][1] + x[1][3] : 0.f), s_dot);
      }
      const float* gc = rf + R::fGc;
      if (first) {
        float f[2][2], dot[2][2];
        {
          float x[2][NT][4] = {};
          gemm32<NT, 0, 4, RC, false, RK>(x, O, m0, S, n0, ln);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = m0 + 16 * m + 8 * e + ln.g;
              f[m][e] = a.scale * expf(gc[r] + gc[C + r]) * qf[r] * oinv * mS;
            }
          take<NT, RK>(x, Q, m0, n0, f, sum, dot, ln);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) put_row(f[m][e] * dot[m][e], red + (w8 >> 1) * C + m0 + 16 * m + 8 * e + ln.g, ln.t, head);
        ln.again();
        // dV = diag(b) dX and its part of dbeta: 16 rows, 32 columns a warp
        const int r0 = 16 * (w8 & 3) + ln.g, k0 = 2 * (w8 >> 2);
        float s_v[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t hi[4], lo[4];
          pair_a_t<RC>(hi, lo, Dx, 16 * (w8 & 3), 16 * (k0 + k), ln);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = r0 + 8 * (e & 1), c = v0 + 16 * (k0 + k) + 8 * (e >> 1) + 2 * ln.t;
            if (r >= rows) continue;
            float2 d = both2(hi[e], lo[e]);
            d.x *= mX;
            d.y *= mX;
            const size_t at = ((size_t)(c0 + r) * a.nv + h) * DV + c;
            const float b = rf[R::fBeta + r];
            if constexpr (sizeof(IO) == 4) {
              const float2 v = *reinterpret_cast<const float2*>(static_cast<const float*>(a.v) + at);
              s_v[e & 1] = fmaf(d.x, v.x, fmaf(d.y, v.y, s_v[e & 1]));
              *reinterpret_cast<float2*>(static_cast<float*>(a.dv_out) + at) = make_float2(b * d.x, b * d.y);
            } else {
              const uint32_t v = *reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.v) + at);
              s_v[e & 1] = fmaf(d.x, __uint_as_float(v << 16), fmaf(d.y, __uint_as_float(v & 0xffff0000u), s_v[e & 1]));
              *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.dv_out) + at) = ptx::pack_bf16x2(b * d.x, b * d.y);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) put_row(s_v[e], reda + (8 + (w8 >> 2)) * C + r0 + 8 * e, ln.t, head);
      } else {
        float f[2][2], dot[2][2];
        {
          float x[2][NT][4] = {};
          gemm32<NT, 0, 4, RC, true, RK>(x, V, m0, D, n0, ln);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = m0 + 16 * m + 8 * e + ln.g;
              f[m][e] = decay(gc, C - 1, r) * kf[r] * mV * mD;
            }
          take<NT, RK>(x, K, m0, n0, f, sum, dot, ln);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) put_row(f[m][e] * dot[m][e], red + (4 + (w8 >> 1)) * C + m0 + 16 * m + 8 * e + ln.g, ln.t, head);
        ln.again();
        float u[2][2];
        {
          float x[2][NT][4] = {};
          gemm32<NT, 0, 4, RC, true, RK>(x, Dx, m0, S, n0, ln);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = m0 + 16 * m + 8 * e + ln.g;
              u[m][e] = -expf(gc[r] + gc[C + r]) * kf[r] * mX * mS;
              f[m][e] = rf[R::fBeta + r] * u[m][e];
            }
          take<NT, RK>(x, K, m0, n0, f, sum, dot, ln);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) put_row(u[m][e] * dot[m][e], red + (8 + (w8 >> 1)) * C + m0 + 16 * m + 8 * e + ln.g, ln.t, head);
      }
      if (tri) {
        ln.again();
        if (head) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) dA[j][e] = dP[j][e] = 0.f;
        }
#pragma unroll 2
        for (int k = 0; k < 4; ++k) {
          uint32_t xh[4], xl[4], oh[4], ol[4], bh[4], bl[4];
          pair_a_t<RC>(xh, xl, Dx, 16 * rb, 16 * k, ln);
          pair_a<RC>(oh, ol, O, 16 * rb, 16 * k, ln);
          pair_b_t<RC>(bh, bl, V, 16 * cb, 16 * k, ln);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mma_pair(dA[j], xh, xl, bh + 2 * j, bl + 2 * j);
            mma_pair(dP[j], oh, ol, bh + 2 * j, bl + 2 * j);
          }
        }
      }
      if (v0 + 64 < DV) continue;
      // ---- 3. what goes through A and P
      s_dot = warp_sum(s_dot);
      if (lane == 0) dots[warp] = s_dot;
      const float sP = oinv * mV, sA = mX * mV;
      if (tri) {
        ln.again();
        const int r0 = 16 * rb + ln.g, i0 = 16 * cb + 2 * ln.t;
        const float* bt = rf + R::fBeta;
        float s_gc[2] = {0.f, 0.f}, s_bt[2] = {0.f, 0.f}, top[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int at = (rb * 8 + 2 * cb + j) * 32 + lane;
          const float4 kk4 = reinterpret_cast<const float4*>(qrec + QR::kKk)[at], qk4 = reinterpret_cast<const float4*>(qrec + QR::kQk)[at];
          const float kk[4] = {kk4.x, kk4.y, kk4.z, kk4.w}, qk[4] = {qk4.x, qk4.y, qk4.z, qk4.w};
          float cs[2] = {0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = r0 + 8 * (e >> 1), i = i0 + 8 * j + (e & 1);
            const float gamma = i <= r ? decay(gc, r, i) : 0.f, strict = i < r ? gamma : 0.f;  // masked before exp
            const float da = sA * dA[j][e], dp = a.scale * sP * dP[j][e];
            const float fk = kf[r] * kf[i], fq = qf[r] * kf[i];
            const float akd = da * (kk[e] * strict);
            const float both = fmaf(-bt[r], akd, dp * strict * qk[e]);
            s_bt[e >> 1] -= akd;
            s_gc[e >> 1] += both;
            cs[e & 1] += both;
            dP[j][e] = dp * gamma * fq;             // N
            dA[j][e] = -da * bt[r] * strict * fk;   // B
            top[0] = fmaxf(top[0], fabsf(dP[j][e]));
            top[1] = fmaxf(top[1], fabsf(dA[j][e]));
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) cs[e] += __shfl_xor_sync(0xffffffffu, cs[e], o);
            if (ln.g == 0) col[rb * C + i0 + 8 * j + e] = cs[e];
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          put_row(s_gc[e], reda + cb * C + r0 + 8 * e, ln.t, true);
          put_row(s_bt[e], reda + (4 + cb) * C + r0 + 8 * e, ln.t, true);
          top[e] = warp_top(top[e]);
          if (lane == 0) ntop[16 * e + warp] = top[e];
        }
        asm volatile("bar.sync 1, 320;" ::: "memory");  // of warps 0-9, which alone read dO: N and B come over dV' and dO
        float f[2], inv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) pow2_factor(warp_top(lane < 10 ? ntop[16 * e + lane] : 0.f), f[e], inv[e]);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t hi, lo;
            const uint32_t at = (uint32_t)pair_at<RC>(r0 + 8 * e, i0 + 8 * j);
            pair2(dP[j][2 * e], dP[j][2 * e + 1], f[0], hi, lo);
            sts32(N + at, hi);
            sts32(N + at + 16 * RC, lo);
            pair2(dA[j][2 * e], dA[j][2 * e + 1], f[1], hi, lo);
            sts32(B + at, hi);
            sts32(B + at + 16 * RC, lo);
            if (cb == rb && (rb & 1) == 0) {  // the block on the right of it is read too, and above the diagonal
              const uint32_t right = (uint32_t)pair_at<RC>(r0 + 8 * e, i0 + 8 * j + 16);
              sts32(N + right, 0u);
              sts32(N + right + 16 * RC, 0u);
              sts32(B + right, 0u);
              sts32(B + right + 16 * RC, 0u);
            }
          }
      }
      __syncthreads();
      // ---- 4.
      ln.again();
      float sN, sB, unused;
      pow2_factor(warp_top(lane < 10 ? ntop[lane] : 0.f), unused, sN);
      pow2_factor(warp_top(lane < 10 ? ntop[16 + lane] : 0.f), unused, sB);
      {
        float x[2][NT][4] = {};
        if (first) {
          if (m0 == 0)
            gemm32<NT, 0, 2, RC, false, RK>(x, N, m0, K, n0, ln);
          else
            gemm32<NT, 0, 4, RC, false, RK>(x, N, m0, K, n0, ln);
        } else {
          if (m0 == 0)
            gemm32<NT, 0, 4, RC, true, RK>(x, N, m0, Q, n0, ln);
          else
            gemm32<NT, 2, 4, RC, true, RK>(x, N, m0, Q, n0, ln);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              sum[m][j][e] = fmaf(sN, x[m][j][e], sum[m][j][e]);
              x[m][j][e] = 0.f;
            }
        if (!first) {
          if (m0 == 0) {
            gemm32<NT, 0, 2, RC, false, RK>(x, B, m0, K, n0, ln);
            gemm32<NT, 0, 4, RC, true, RK>(x, B, m0, K, n0, ln);
          } else {
            gemm32<NT, 0, 4, RC, false, RK>(x, B, m0, K, n0, ln);
            gemm32<NT, 2, 4, RC, true, RK>(x, B, m0, K, n0, ln);
          }
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) sum[m][j][e] = fmaf(sB, x[m][j][e], sum[m][j][e]);
        }
      }
      if (warp == 0) {
        // dgc of rows 2 lane, 2 lane + 1; then the suffix sums.  l_r k_r . (V' dS'^T)_r is taken from dgc_r and added to the
        // last row: in dg_t only the rows before t are left of it, and are added as such, since the difference of the two
        // sums would have no digits where a chunk's own decay is small beside it (one token behind a strong gate).
        auto four = [&](const float* x, int r) { return (x[r] + x[C + r]) + (x[2 * C + r] + x[3 * C + r]); };
        float d[2], th[2], bsum[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 2 * lane + e;
          const float u = four(red + 8 * C, r);
          th[e] = four(red + 4 * C, r);
          d[e] = four(reda, r) + four(red, r) + rf[R::fBeta + r] * u - four(col, r);
          bsum[e] = four(reda + 4 * C, r) + (reda[8 * C + r] + reda[9 * C + r]) + u;
        }
        const float dsum = warp_sum(lane < 16 ? dots[lane] : 0.f) * rf[R::fScal + kScalGl];
        float suf = d[0] + d[1], pre = th[0] + th[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float y = __shfl_down_sync(0xffffffffu, suf, o), z = __shfl_up_sync(0xffffffffu, pre, o);
          if (lane + o < 32) suf += y;
          if (lane >= o) pre += z;
        }
        float beyond = __shfl_down_sync(0xffffffffu, suf, 1), before = __shfl_up_sync(0xffffffffu, pre, 1);
        if (lane == 31) beyond = 0.f;
        if (lane == 0) before = 0.f;
        const float dg[2] = {suf + (before + dsum), beyond + d[1] + (before + th[0] + dsum)};
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (2 * lane + e < rows) {
            const size_t at = (size_t)(c0 + 2 * lane + e) * a.nv + h;
            static_cast<IO*>(a.dg)[at] = from_f32<IO>(dg[e]);
            static_cast<IO*>(a.dbeta)[at] = from_f32<IO>(bsum[e]);
          }
      }
    }
  }
  if (quit) {  // a copy never came: report it, wait once more for what is in flight, and leave
    if (tid == 0) {
      report_status(a.status, kStatusTimeout);
      ptx::mbar_wait_bounded(bar, it & 1, kWaitLimitNs);
    }
    return;
  }
  __syncthreads();  // the last v-head's sums are read
  // the norms: with y = qf dq_hat, dq = (y - qf^2 Q16 (Q16 . y)) / (qf |q|), and dk alike
  ln.again();
  const uint32_t Yi = first ? Q : K;
  const float *yf = first ? qf : kf, *yn = first ? qn : kn;
  float* part = red + (first ? 0 : 4 * C);
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = m0 + 16 * m + 8 * e + ln.g;
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float2 y = lds_pair<RK>(Yi, r, n0 + 8 * j + 2 * ln.t);
        dot = fmaf(sum[m][j][2 * e], y.x, fmaf(sum[m][j][2 * e + 1], y.y, dot));
      }
      put_row(dot, part + (w8 >> 1) * C + r, ln.t, true);
    }
  __syncthreads();
  IO* out = static_cast<IO*>(first ? a.dq : a.dk);
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = m0 + 16 * m + 8 * e + ln.g;
      if (r >= rows) continue;
      const float p = a.qk_l2norm ? yf[r] * yf[r] * ((part[r] + part[C + r]) + (part[2 * C + r] + part[3 * C + r])) : 0.f, fn = yn[r];
      float w[2 * NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float2 y = lds_pair<RK>(Yi, r, n0 + 8 * j + 2 * ln.t);
        w[2 * j] = fn * (sum[m][j][2 * e] - y.x * p);
        w[2 * j + 1] = fn * (sum[m][j][2 * e + 1] - y.y * p);
      }
      // by swap32 this thread's pairs are neighbours: 8 columns (Dk = 128) or 4 (Dk = 64)
      IO* dst = out + ((size_t)(c0 + r) * a.nqk + hq) * DK + swap32(n0 + 2 * ln.t);
#pragma unroll
      for (int j = 0; j < NT; j += 2) {
        if constexpr (sizeof(IO) == 4)
          *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(w[2 * j], w[2 * j + 1], w[2 * j + 2], w[2 * j + 3]);
        else
          *reinterpret_cast<uint2*>(dst + 2 * j) = make_uint2(ptx::pack_bf16x2(w[2 * j], w[2 * j + 1]), ptx::pack_bf16x2(w[2 * j + 2], w[2 * j + 3]));
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
    prepare_kernel<DK, DV, IO><<<slot_grid(slots, a.nqk), kThreads, PrepSmem<DK, DV>::kBytes, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = set_smem(states_kernel<DK, DV>, StateSmem<DK>::kBytes)) != cudaSuccess) return e;
  e = launch_next(states_kernel<DK, DV>, dim3(2 * DV / (16 * kStateSlices), a.nv, a.num_seqs), kStateThreads, StateSmem<DK>::kBytes, stream, a);
  if (e != cudaSuccess || a.total_tokens == 0) return e;
  if ((e = set_smem(grads_kernel<DK, DV, IO>, GradSmem<DK, DV>::kBytes)) != cudaSuccess) return e;
  return launch_next(grads_kernel<DK, DV, IO>, slot_grid(slots, a.nqk), kThreads, GradSmem<DK, DV>::kBytes, stream, a);
}

template <int DK, int DV>
static cudaError_t launch_io(const BwdArgs& a, int io_bf16, cudaStream_t s) {
  return io_bf16 ? launch_one<DK, DV, __nv_bfloat16>(a, s) : launch_one<DK, DV, float>(a, s);
}

}  // namespace bwd

int64_t chunk_bwd_workspace(int64_t total_tokens, int num_seqs, int nqk, int nv, int dk, int dv) {
  if (total_tokens == 0) return 0;
  const int64_t c = bwd::C, rec = 4 * (c * (c + dk + 4 * dv) + 2 * (int64_t)dk * dv) + 4 * (5 * c + 8 + 5 * dv);
  return (total_tokens / c + num_seqs) * (nv * rec + nqk * (16 * c * dk + 16 * c + 8 * c * c));
}

cudaError_t launch_chunk_bwd(const BwdArgs& a, int dk, int dv, int io_bf16, cudaStream_t s) {
  static_assert(bwd::Rec<128, 64>::kBytes == 4 * (64 * (64 + 128 + 4 * 64) + 2 * 128 * 64) + 4 * (5 * 64 + 8 + 5 * 64), "workspace size");
  static_assert(bwd::QkRec<128>::kBytes == 16 * 64 * 128 + 16 * 64 + 8 * 64 * 64, "workspace size");
  if (dk == 64 && dv == 64) return bwd::launch_io<64, 64>(a, io_bf16, s);
  if (dk == 64 && dv == 128) return bwd::launch_io<64, 128>(a, io_bf16, s);
  if (dk == 128 && dv == 64) return bwd::launch_io<128, 64>(a, io_bf16, s);
  if (dk == 128 && dv == 128) return bwd::launch_io<128, 128>(a, io_bf16, s);
  return cudaErrorInvalidValue;
}

}  // namespace gdn
