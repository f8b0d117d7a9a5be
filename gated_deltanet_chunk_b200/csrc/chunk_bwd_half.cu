// chunk_bwd_half.cu -- gradients of the chunked gated delta rule for bf16 tensors.
//
// The mathematics, the notation and the three kernels are those of chunk_bwd.cu.
// Here a product is one MMA in fp16 with fp32 accumulation (mma.sync.m16n8k16; tcgen05 in
// the states kernel, where the next chunk waits for it): an operand is an fp16 number (11
// significant bits) times a power of two that its tile, row or column shares, chosen so that
// the largest magnitude is in [2^7, 2^8) or bounded by it.  So
//   - q, k, v and dout, which have 8 significant bits, are exact,
//   - what is formed on the way (T, W, S, V', dS', ...) is rounded by at most 2^-11 of its
//     value, or 2^-32 of its tile's largest: an eighth of the bf16 rounding that the outputs
//     get, at the cost of one MMA, where bf16 operands of that accuracy would need two or
//     three.  A gradient meets up to eleven of them, 2e-4 to 1.3e-3 of its largest element,
//   - W's operand T diag(b e), whose terms cancel where keys repeat, is a pair hi + lo,
//   - 2^8 against fp16's 65504 leaves room for what follows from a bounded sum.
// The recurrences themselves (S and dS), the cumsums, the decays and every sum are fp32; the
// inverse is fp32 in its 16 x 16 diagonal blocks and products of TF32 pairs off them.
//
// Bounds that the factors of two use (they hold for 0 <= beta <= 2, g <= 0 and normalised q,
// k; the prepare kernel reports gates outside, where the results are undefined): decays are
// at most 1, |T_ri| <= 2 (row r of T is beta_r k_r^T times a product of contractions, times
// k_i), |W_r| <= beta_r e_r, |q_r . k_i| <= 1.  T and P have a fixed factor, since T's
// diagonal is 1 and P's products are of unit rows.  Factors that depend on the gates follow
// them: e takes any number of binades over a chunk and from one to the next, beta any value,
// so W has a power of two for every row, T diag(b), diag(qe) dO, V' diag(kw) and dV' diag(wr)
// one of their largest (6 % of prepare's time for diag(qe) dO, 4 to 10 % of states' for its
// two, against fixed ones, which lost all digits behind strong gates).
//
// Measured for 2 x 32768 tokens, 16 / 32 heads of 128, as prepare + states + gradients:
// 1.51 + 1.29 + 2.48 ms (0.39 + 0.30 + 0.65 ms for 15,928 packed tokens).  What they read
// and write, the tiles that they pass on included, is 5.1 + 6.5 + 6.1 GB, 2.7 ms at the
// copy bandwidth: states is nearest (77 %), prepare at 52 % (a block's loads, its
// inverse and its stores wait for one another, and two blocks per SM is what shared
// memory holds), gradients at 37 % (17,000 cycles a v-head, of which the MMAs are
// 6,000: the element-wise parts between them and two barriers are the rest).  Passing
// tiles on in fp16 costs bytes but no second walk over the chunk; forming T, U and W
// again in the gradients would cost more than the 1.3 GB it saves.
#include <cuda_fp16.h>

#include <type_traits>

#include "chunk_bwd.cuh"
#include "train_common.cuh"
#include "gdn_launch.h"
#include "sm100_ptx.cuh"

namespace gdn {
namespace bwdh {

using namespace bwd;
using bf16 = __nv_bfloat16;

constexpr int HP = C + 8;  // pitch of the prepare kernel's [..][64] fp16 tiles: rows 16 bytes apart in the banks

// Workspace record of one (chunk slot, v-head), in bytes; images: see chunk_bwd.cuh.
template <int DK, int DV>
struct Rec {
  static constexpr size_t kX = 0;                      // image of (P^T dO)^T [DV][C], columns by swap32; then of dV'^T
  static constexpr size_t kT = kX + 2 * C * DV;        // image of T 2^7 [C][C]
  static constexpr size_t kV = kT + 2 * C * C;         // image of U^T [DV][C], columns by swap32; then of V'^T
  static constexpr size_t kS = kV + 2 * C * DV;        // image of S^T [DV][DK] before the chunk, in panels, columns by swap32
  static constexpr size_t kO = kS + 2 * DK * DV;       // image of dO [C][DV]
  static constexpr size_t kD = kO + 2 * C * DV;        // of dS'^T behind the chunk, alike
  static constexpr size_t kW = kD + 2 * DK * DV;       // image of W [C][DK], a factor a row, in panels, columns by swap32
  static constexpr size_t kOq = kW + 2 * C * DK;       // image of diag(qe) dO [C][DV], in panels
  static constexpr size_t kF = kOq + 2 * C * DV;       // floats from here:
  static constexpr int fGc = 0;                        // [C] gcum
  static constexpr int fBeta = fGc + C;                // [C] beta
  static constexpr int fScal = fBeta + C;              // [8] see Scal
  static constexpr int fDV = fScal + 8;                // [DV] factor of every row of dV'^T
  static constexpr int fKw = fDV + DV;                 // [C] l_r / |k_r| in units of K16
  static constexpr int fWr = fKw + C;                  // [C] factor of every row of W
  static constexpr int kFloats = fWr + C;
  static constexpr size_t kBytes = kF + 4 * kFloats;
  static_assert(kBytes % 16 == 0 && fScal % 4 == 0 && fKw % 4 == 0, "16-byte copies");
};
// factors of U, Y, diag(qe) dO, dO, S, dS' and V', and e_last
enum Scal { kScalU, kScalY, kScalO, kScalGl, kScalDo, kScalS, kScalD, kScalV };

// Workspace record of one (chunk slot, qk-head), in bytes.
template <int DK>
struct QkRec {
  static constexpr size_t kK = 0;                // image of K16 [C][DK], in panels, columns by swap32
  static constexpr size_t kQ = kK + 2 * C * DK;  // of Q16
  static constexpr size_t kF = kQ + 2 * C * DK;   // floats [4][C]: k_hat = kf K16, q_hat = qf Q16, and kf |k|, qf |q| inverted
  static constexpr size_t kBytes = kF + 16 * C;
};

// What the gradients kernel has to know of a slot.
struct SlotInfo {
  int64_t c0;     // first token
  int32_t rows;   // tokens, 0: an empty slot
  int32_t pad;
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
template <int DK, int DV>
__device__ __forceinline__ SlotInfo* slot_info(const BwdArgs& a, int64_t slot) {
  return reinterpret_cast<SlotInfo*>(qk_at<DK, DV>(a, slots_of<DK, DV>(a), 0)) + slot;
}

// ------------------------------------------------------------------ fragments
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

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// ------------------------------------------------------------------ 1. prepare
// One block per (slot, qk-head): K16, Q16 and their products once, then its v-heads in turn.

constexpr int kPrepThreads = 256;

template <int DK, int DV>
struct PrepSmem {
  static constexpr int DP = DK + 8, VP = DV + 8;
  static constexpr size_t kK = 0;                                       // fp16 [C][DP] K16
  static constexpr size_t kQ = kK + 2 * C * DP;                         // fp16 [C][DP] Q16, then T beta and P 2^8, [C][HP] each
  static constexpr size_t kQBytes = 2 * C * DP > 4 * C * HP ? 2 * C * DP : 4 * C * HP;
  static constexpr size_t kV = kQ + kQBytes;                            // fp16 [C][VP] V
  static constexpr size_t kO = kV + 2 * C * VP;                         // fp16 [C][VP] dO
  static constexpr size_t kA = kO + 2 * C * VP;                         // fp32 [C][TP] A, then T
  static constexpr size_t kY = kA + 4 * C * TP;                         // fp32 [C / 2][TP] scratch of the inverse
  static constexpr size_t kF = kY + 2 * C * TP;                         // fp32 [C] each: gc, beta, kf, qf, T's column and row factors of W
  static constexpr size_t kQe = kF + 24 * C;                            // fp32 [C] e qf
  static constexpr size_t kTop = kQe + 4 * C;                           // fp32 [3][8] largest |v|, |dO|, |diag(qe) dO| by warp, [2] beta
  static constexpr size_t kBytes = kTop + 112;
  static_assert(kBytes <= 113 * 1024, "two blocks per SM");
};

// Rows of q or k: to fp16 with a factor of two for each row, into a tile (pitch DK + 8) and the workspace,
// and the factors.  DK / 8 lanes per row.  Rows so small that the norm's eps decides are scaled by 2^17, so
// that kf and qf stay within a few powers of two of one another.
template <int DK>
__device__ __forceinline__ void load_rows(const bf16* x, int64_t c0, int64_t end, int heads, int head,
                                          uint4 (&w)[C * DK / 8 / kPrepThreads], int tid) {
  constexpr int L = DK / 8, R = kPrepThreads / L;
#pragma unroll
  for (int p = 0; p < C / R; ++p) {
    const int r = p * R + tid / L;
    w[p] = make_uint4(0u, 0u, 0u, 0u);
    if (c0 + r < end) w[p] = *reinterpret_cast<const uint4*>(x + ((size_t)(c0 + r) * heads + head) * DK + 8 * (tid % L));
  }
}
template <int DK>
__device__ __forceinline__ void store_qk(const uint4 (&vec)[C * DK / 8 / kPrepThreads], __half* tile, uint8_t* img,
                                         float* f, float* wf, float* wn, int tid) {
  constexpr int L = DK / 8, R = kPrepThreads / L, N = C / R;
  const int lr = tid % L;
  float ss[N], top[N], s[N], inv[N];
#pragma unroll
  for (int p = 0; p < N; ++p) {
    const uint32_t u[4] = {vec[p].x, vec[p].y, vec[p].z, vec[p].w};
    ss[p] = top[p] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = bf2(u[i]);
      ss[p] = fmaf(v.x, v.x, fmaf(v.y, v.y, ss[p]));
      top[p] = fmaxf(top[p], fmaxf(fabsf(v.x), fabsf(v.y)));
    }
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
    for (int p = 0; p < N; ++p) {
      ss[p] += __shfl_xor_sync(0xffffffffu, ss[p], o);
      top[p] = fmaxf(top[p], __shfl_xor_sync(0xffffffffu, top[p], o));
    }
#pragma unroll
  for (int p = 0; p < N; ++p) {
    const int r = p * R + tid / L;
    const uint32_t u[4] = {vec[p].x, vec[p].y, vec[p].z, vec[p].w};
    pow2_factor(fmaxf(top[p], 0x1p-10f), s[p], inv[p]);
    uint4 h;
    uint32_t* w = &h.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = bf2(u[i]);
      w[i] = pack2(v.x * s[p], v.y * s[p]);
    }
    *reinterpret_cast<uint4*>(tile + r * (DK + 8) + 8 * lr) = h;
    transpose4(h, lr);
    *reinterpret_cast<uint4*>(img + image<-C>(r, (8 * lr & ~31) + 8 * (lr & 3))) = h;
  }
  static_assert(N <= L, "a lane for every row");
  if (lr < N) {  // lane p has row p's factors: one square root and division for all
    float q = ss[0], a = s[0], b = inv[0];
#pragma unroll
    for (int p = 1; p < N; ++p)
      if (lr == p) {
        q = ss[p];
        a = s[p];
        b = inv[p];
      }
    const int r = lr * R + tid / L;
    b /= sqrtf(q + kNormEps);
    f[r] = b;
    wf[r] = b;
    wn[r] = a;
  }
}

// Brings [C x DV] of v or dout into L2, a line of 128 bytes a thread
template <int DV>
__device__ __forceinline__ void prefetch_v(const bf16* x, int64_t c0, int64_t end, int nv, int h, int tid) {
  constexpr int L = DV / 64;
  const int r = tid / L;
  if (r < C && c0 + r < end)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(x + ((size_t)(c0 + r) * nv + h) * DV + 64 * (tid % L)));
}

// [C x DV] of v or dout for this thread: NV vectors of 8, vector i at row i R + tid / L
template <int DV>
__device__ __forceinline__ void load_v(const bf16* x, int64_t c0, int64_t end, int nv, int h, uint4 (&w)[C * DV / 8 / kPrepThreads], int tid) {
  constexpr int L = DV / 8, R = kPrepThreads / L;
#pragma unroll
  for (int p = 0; p < C / R; ++p) {
    const int r = p * R + tid / L;
    w[p] = make_uint4(0u, 0u, 0u, 0u);
    if (c0 + r < end) w[p] = *reinterpret_cast<const uint4*>(x + ((size_t)(c0 + r) * nv + h) * DV + 8 * (tid % L));
  }
}
// The largest magnitudes of a vector's even and odd elements (a NaN does not count), and over a warp or its shares in `t`
__device__ __forceinline__ __nv_bfloat162 top_v(const uint4& w) {
  const __nv_bfloat162* u = reinterpret_cast<const __nv_bfloat162*>(&w);
  return __hmax2(__hmax2(__habs2(u[0]), __habs2(u[1])), __hmax2(__habs2(u[2]), __habs2(u[3])));
}
__device__ __forceinline__ float top_f(__nv_bfloat162 x) { return fmaxf(__bfloat162float(x.x), __bfloat162float(x.y)); }
__device__ __forceinline__ float warp_top(float x) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x))); }
__device__ __forceinline__ float top8(const float* t) {
  const float4 a = *reinterpret_cast<const float4*>(t), b = *reinterpret_cast<const float4*>(t + 4);
  return fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)), fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
}
template <int DV>
__device__ __forceinline__ void store_v(const uint4 (&w)[C * DV / 8 / kPrepThreads], float s, __half* tile, uint8_t* img, int tid) {
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
    const int r = p * R + tid / L, c = 8 * (tid % L);
    *reinterpret_cast<uint4*>(tile + r * (DV + 8) + c) = make_uint4(h[0], h[1], h[2], h[3]);
    if (img) *reinterpret_cast<uint4*>(img + image<2 * DV>(r, c)) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// Row g (e = 0) or g + 8 (e = 2) of a warp's accumulators, 32 columns from x on, times f: this lane's 8 columns in the
// order of swap32, where they are one vector
__device__ __forceinline__ uint4 swapped32(const float (*x)[4], int e, float f) {
  return make_uint4(pack2(x[0][e] * f, x[0][e + 1] * f), pack2(x[1][e] * f, x[1][e + 1] * f), pack2(x[2][e] * f, x[2][e + 1] * f),
                    pack2(x[3][e] * f, x[3][e + 1] * f));
}
// Rows 16 u .. of an image [DV][C] from accumulators, times f, columns by swap32
__device__ __forceinline__ void store_rows(uint8_t* img, int u, const float (&x)[8][4], float f, int g, int t) {
#pragma unroll
  for (int j = 0; j < 8; j += 4)
#pragma unroll
    for (int e = 0; e < 4; e += 2) *reinterpret_cast<uint4*>(img + image<2 * C>(16 * u + g + 4 * e, 8 * j + 8 * t)) = swapped32(x + j, e, f);
}

template <int DK, int DV>
__global__ void __launch_bounds__(kPrepThreads, 2) prepare_half_kernel(BwdArgs a) {
  let_next_begin();
  using L = PrepSmem<DK, DV>;
  using R = Rec<DK, DV>;
  using QR = QkRec<DK>;
  extern __shared__ __align__(128) uint8_t sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
  const int hq = blockIdx.x, group = a.nv / a.nqk;
  const int64_t slot = grid_slot();
  if (slot >= a.total_tokens / C + a.num_seqs) return;
  int64_t c0, end;
  const bool any = bwd::chunk_at(a, slot, c0, end);
  if (hq == 0 && tid == 0) *slot_info<DK, DV>(a, slot) = SlotInfo{c0, any ? (int32_t)min((int64_t)C, end - c0) : 0, 0};
  if (!any) return;
  __half *K = reinterpret_cast<__half*>(sm + L::kK), *Q = reinterpret_cast<__half*>(sm + L::kQ);
  __half *TB = Q, *P = Q + C * HP, *V = reinterpret_cast<__half*>(sm + L::kV), *O = reinterpret_cast<__half*>(sm + L::kO);
  float *A = reinterpret_cast<float*>(sm + L::kA), *Y = reinterpret_cast<float*>(sm + L::kY);
  float *gc = reinterpret_cast<float*>(sm + L::kF), *bt = gc + C, *kf = bt + C, *qf = kf + C, *wf = qf + C, *wr_f = wf + C;
  float* qe = reinterpret_cast<float*>(sm + L::kQe);
  float* tops = reinterpret_cast<float*>(sm + L::kTop);
  uint8_t* qrec = qk_at<DK, DV>(a, slot, hq);
  float* qfl = reinterpret_cast<float*>(qrec + QR::kF);

  {
    uint4 kw[C * DK / 8 / kPrepThreads], qw[C * DK / 8 / kPrepThreads];  // all loads before the first store
    load_rows<DK>(static_cast<const bf16*>(a.k), c0, end, a.nqk, hq, kw, tid);
    load_rows<DK>(static_cast<const bf16*>(a.q), c0, end, a.nqk, hq, qw, tid);
    for (int h = hq * group; h < (hq + 1) * group; ++h) {
      prefetch_v<DV>(static_cast<const bf16*>(a.v), c0, end, a.nv, h, tid);
      prefetch_v<DV>(static_cast<const bf16*>(a.dout), c0, end, a.nv, h, tid);
    }
    store_qk<DK>(kw, K, qrec + QR::kK, kf, qfl, qfl + 2 * C, tid);
    store_qk<DK>(qw, Q, qrec + QR::kQ, qf, qfl + C, qfl + 3 * C, tid);
  }
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

  uint4 vw[C * DV / 8 / kPrepThreads], ow[C * DV / 8 / kPrepThreads];  // of the next v-head, while this one's U and Y are formed
  load_v<DV>(static_cast<const bf16*>(a.v), c0, end, a.nv, hq * group, vw, tid);
  load_v<DV>(static_cast<const bf16*>(a.dout), c0, end, a.nv, hq * group, ow, tid);
  for (int h = hq * group; h < (hq + 1) * group; ++h) {
    uint8_t* rec = rec_at<DK, DV>(a, slot, h);
    float* rf = reinterpret_cast<float*>(rec + R::kF);
    constexpr int NV = C * DV / 8 / kPrepThreads;
    __nv_bfloat162 vt = __float2bfloat162_rn(0.f), orow[NV], ot = vt;  // orow: of this thread's part of a row of dO
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      vt = __hmax2(vt, top_v(vw[p]));
      orow[p] = top_v(ow[p]);
      ot = __hmax2(ot, orow[p]);
    }
    float vtop = warp_top(top_f(vt)), otop = warp_top(top_f(ot));
    float gv = 0.f, bv = 0.f;
    if (tid < C && c0 + tid < end) {
      load_gate(a, (size_t)(c0 + tid) * a.nv + h, h, gv, bv);
      if (!(gv <= 0.f) || !(bv >= 0.f && bv <= 2.f)) report_status(a.status, kStatusGate);
      gv = gv < kGateFloor ? kGateFloor : gv;
    }
    __syncthreads();  // the head before is done with the tiles
    if (lane == 0) {
      tops[warp] = vtop;
      tops[8 + warp] = otop;
    }
    if (tid < C) {
      gc[tid] = gv;
      bt[tid] = bv;
      const float top = warp_top(bv);
      if (lane == 0) tops[24 + warp] = top;
    }
    __syncthreads();
    if (warp == 0) bwd::cumsum_chunk(gc, lane);
    vtop = top8(tops);
    otop = top8(tops + 8);
    float vs, vinv, os, oinv;
    pow2_factor(vtop, vs, vinv);
    pow2_factor(otop, os, oinv);
    store_v<DV>(vw, vs, V, nullptr, tid);
    store_v<DV>(ow, os, O, rec + R::kO, tid);
    __syncthreads();
    float p[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int r = r0 + 4 * e, i = wc + 8 * j + 2 * t4;
        const float2 gi = *reinterpret_cast<const float2*>(gc + i);
        const float g0 = i <= r ? ptx::ex2_approx(1.44269504f * (gc[r] - gi.x)) : 0.f;  // masked before exp
        const float g1 = i + 1 <= r ? ptx::ex2_approx(1.44269504f * (gc[r] - gi.y)) : 0.f;
        *reinterpret_cast<float2*>(A + r * TP + i) =
            make_float2(i < r ? -bt[r] * (kk[j][e] * g0) : 0.f, i + 1 < r ? -bt[r] * (kk[j][e + 1] * g1) : 0.f);
        p[j][e] = qk[j][e] * g0 * 0x1p8f;
        p[j][e + 1] = qk[j][e + 1] * g1 * 0x1p8f;
      }
    __syncthreads();
    if (tid >= 128 && tid < 128 + C) {  // while warps 0-3 substitute
      const int i = tid - 128;
      const float e = expf(gc[i]);
      // Row r of W is b_r e_r k_r^T times a product of contractions, so b_r e_r bounds it, and T_ri b_i e_i is at most
      // 2 b_r e_r: a factor a row keeps the digits of rows that lie any number of binades below the first.
      // 2^7 kf <= 1 (kf is at most 2^-7: the largest element of a row is at most its norm)
      float wrow, winv;
      pow2_factor(bt[i] * e, wrow, winv);
      wr_f[i] = wrow;
      rf[R::fWr + i] = winv;
      wf[i] = bt[i] * e * kf[i] * 0x1p6f;
      qe[i] = e * qf[i];
      rf[R::fGc + i] = gc[i];
      rf[R::fBeta + i] = bt[i];
      rf[R::fKw + i] = expf(gc[C - 1] - gc[i]) * kf[i];
      if (i == C - 1) {
        float f, inv;
        pow2_factor(fmaxf(tops[24], tops[25]), f, inv);
        rf[R::fScal + kScalU] = 0x1p8f * inv * vinv;
        rf[R::fScal + kScalY] = a.scale * oinv;
        rf[R::fScal + kScalGl] = e;
        rf[R::fScal + kScalDo] = oinv;
      }
    }
    bwd::invert_chunk<true>(A, Y, warp, lane);
    float bs, binv;  // beta's factor: T beta is at most 2^8 times a half of it
    pow2_factor(fmaxf(tops[24], tops[25]), bs, binv);
    bs *= 0.5f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int r = r0 + 4 * e, i = wc + 8 * j + 2 * t4;
        const float2 t = *reinterpret_cast<const float2*>(A + r * TP + i);
        *reinterpret_cast<uint32_t*>(P + r * HP + i) = pack2(p[j][e], p[j][e + 1]);
        *reinterpret_cast<uint32_t*>(TB + r * HP + i) = pack2(t.x * (bt[i] * bs), t.y * (bt[i + 1] * bs));
        *reinterpret_cast<uint32_t*>(rec + R::kT + image<2 * C>(r, i)) = pack2(t.x * 0x1p7f, t.y * 0x1p7f);
      }
    float qtop = 0.f;
#pragma unroll
    for (int p = 0; p < NV; ++p) qtop = fmaxf(qtop, top_f(orow[p]) * qe[(p * kPrepThreads + tid) / (DV / 8)]);
    qtop = warp_top(qtop);
    if (lane == 0) tops[16 + warp] = qtop;
    __syncthreads();
    {  // W over its rows' factors = (those T diag(b e kf) 2^6) K16 2^-6: this warp's 16 rows, one half of the columns.  Where
       // keys repeat, the terms of a row cancel, so the first operand is a pair hi + lo (K16 is exact)
      constexpr int NT = DK / 16;
      float x[NT][4] = {};
      const int n0 = (DK / 2) * (warp >> 2);
      const float fr[2] = {wr_f[r0], wr_f[r0 + 8]};
#pragma unroll
      for (int k = 0; k < C; k += 16) {  // T's zeros above the diagonal are multiplied too: a branch would cost more
        uint32_t ah[4], al[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + 8 * (e & 1), i = k + 8 * (e >> 1) + 2 * t4;
          const float2 t = *reinterpret_cast<const float2*>(A + r * TP + i);
          const float p0 = t.x * fr[e & 1] * wf[i], p1 = t.y * fr[e & 1] * wf[i + 1];
          ah[e] = pack2(p0, p1);
          const float2 h = unpack2(ah[e]);
          al[e] = pack2(p0 - h.x, p1 - h.y);
        }
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          uint32_t b[4];
          frag_b_t<L::DP>(b, K, n0 + 8 * j, k, lane);
          mma_f16(x[j], al, b);
          mma_f16(x[j + 1], al, b + 2);
          mma_f16(x[j], ah, b);
          mma_f16(x[j + 1], ah, b + 2);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; j += 4)
#pragma unroll
        for (int e = 0; e < 4; e += 2)
          *reinterpret_cast<uint4*>(rec + R::kW + image<-C>(r0 + 4 * e, n0 + 8 * j + 8 * t4)) = swapped32(x + j, e, 0x1p-6f);
    }
    {  // diag(qe) dO: fp32 products, rounded once, under a factor that follows the largest of them.  e spans any number of
       // binades over a chunk and between chunks, so a factor that did not would lose the digits of dS behind a strong gate
      float f, inv;
      pow2_factor(top8(tops + 16), f, inv);
      if (tid == 0) rf[R::fScal + kScalO] = a.scale * inv;
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const int r = (p * kPrepThreads + tid) / (DV / 8), c = 8 * (tid % (DV / 8));
        uint4 w = *reinterpret_cast<const uint4*>(O + r * L::VP + c);
        uint32_t* u = &w.x;
        // dO16 oinv is dO.  A row that is not zero in dO16 (at least 2^-24) has a factor of at most 2^32
        const float q = fminf(qe[r] * f * oinv, 0x1p100f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 o = unpack2(u[i]);
          u[i] = pack2(o.x * q, o.y * q);
        }
        *reinterpret_cast<uint4*>(rec + R::kOq + image<-C>(r, c)) = w;
      }
    }
    if (h + 1 < (hq + 1) * group) {
      load_v<DV>(static_cast<const bf16*>(a.v), c0, end, a.nv, h + 1, vw, tid);
      load_v<DV>(static_cast<const bf16*>(a.dout), c0, end, a.nv, h + 1, ow, tid);
    }
    // U^T = V^T (T diag(b))^T and Y^T = dO^T P, 16 columns of Dv a unit
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
      store_rows(rec + R::kV, u, x, 0x1p-7f, g8, t4);
    }
    for (int u = kPrepThreads / 32 - 1 - warp; u < DV / 16; u += kPrepThreads / 32) {
      float x[8][4] = {};
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
      }
      store_rows(rec + R::kX, u, x, 0x1p-8f, g8, t4);
    }
  }
}

// ------------------------------------------------------------------ 2. states
// One block of 8 warps per (sequence, v-head, direction).  S^T (or dS^T) stays in registers in fp32, a row (a column of
// Dv) in two threads of warps w and w + 4, whose TMEM lanes it shares; a chunk is two products on the tensor cores with
// M = 128 (Dv = 64 leaves half of the lanes unread):
//   x^T = S^T W^T          then  S^T = e_last S^T + (V'^T diag(kw)) K                    forwards
//   x^T = dS'^T K^T        then  dS^T = e_last dS'^T + (diag(qe) dO)^T Q - (dV'^T diag(wr)) W   backwards
// Their A operands are written to shared memory: S^T once, as the gradients read it, and V' diag(kw) and dV' diag(wr)
// (wr: the factors of W's rows) over the U or Y that they were formed from.  Both vectors span any number of binades over
// a chunk, and so may V' and dV', so these products have factors of their own, a row.  The images leave by bulk copies.
// The tiles of a chunk come in two chunks ahead.  All columns of Dk are in the order of swap32, which no product sees.
// The state's image has one factor, joined over the block, and so has the image of V'; that of dV' has one a row.  Both
// are written while the second product runs.
// A chunk waits for the one before it, and a thread issues an MMA every 90 to 130 cycles: so N is all of Dk, x is
// two sums over half of Dk from two warps, and z = (diag(qe) dO)^T Q comes from a third (2 x 32768 tokens and 32
// heads of 128, while its operands had fixed factors: 1.15 ms; 1.54 with one warp and N = 64, 1.51 with a ninth warp for all
// of them; 2.11 with warp MMAs).

constexpr int kStateThreads = 256;

template <int DK, int DV>
struct StateSmem {  // from a 1024-byte boundary: tiles of the 128-byte swizzle
  static constexpr uint32_t kTile = 2 * C * DK, kRows = 2 * C * DV;
  static constexpr uint32_t oW = 0, oK = kTile, oU = 3 * kTile, oO = oU + kRows, oF = oO + kRows;  // a stage: W; K16, Q16; U or Y; Oq
  static constexpr uint32_t kStage = oF + 1024;         // and kw [C], wr [C], Scal [8]
  static constexpr uint32_t kS = 2 * kStage;            // S^T, panels of 128 rows
  static constexpr uint32_t kV = kS + 2 * 128 * DK;     // V'^T [128][C]
  static constexpr uint32_t kTop = kV + 2 * 128 * C;    // fp32 [2][8], [8] the warps' largest of the state and V'; [2][128] pairs of a row's halves
  static constexpr uint32_t kBar = kTop + 96 + 2048;    // five barriers
  static constexpr uint32_t kTmem = kBar + 48;
  static constexpr uint32_t kBytes = kTmem + 16 + 1024;
  static_assert(kBytes <= 232448, "shared memory budget");
};

__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 pack8(const float* x, float f) {
  return make_uint4(pack2(x[0] * f, x[1] * f), pack2(x[2] * f, x[3] * f), pack2(x[4] * f, x[5] * f), pack2(x[6] * f, x[7] * f));
}

// The largest magnitude of N values, four at a time: one after another, each fmaxf would wait for the one before
template <int N>
__device__ __forceinline__ float top_of(const float (&x)[N]) {
  float t[4] = {};
#pragma unroll
  for (int j = 0; j < N; ++j) t[j & 3] = fmaxf(t[j & 3], fabsf(x[j]));
  return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}

template <int DK, int DV, bool kBackward>
__device__ __forceinline__ void walk(const BwdArgs& a, uint8_t* sm, int n, int h) {
  using L = StateSmem<DK, DV>;
  using R = Rec<DK, DV>;
  using QR = QkRec<DK>;
  constexpr int NS = DK / 2;                                     // columns of Dk of a thread
  constexpr uint32_t kCols = kBackward && DK == 128 ? 512 : 256; // TMEM: x [2][64], y [DK], z [DK]
  constexpr uint32_t tY = 128, tZ = 128 + DK;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = warp >> 2;
  const int c = 32 * (warp & 3) + lane;                          // this thread's column of Dv
  const bool active = 32 * (warp & 3) < DV;
  const int hq = h / (a.nv / a.nqk);
  const uint32_t base = ptx::smem_u32(sm);
  float *tops = reinterpret_cast<float*>(sm + L::kTop), *vtops = tops + 16;
  float2* rtops = reinterpret_cast<float2*>(tops + 24);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::kBar);     // a stage's copies (two), x, y, z
  int64_t start, end;
  seq_bounds(a, n, start, end);
  const int64_t chunks = (end - start + C - 1) / C, slot0 = start / C + n;
  if (chunks == 0 && !(kBackward && a.ds0)) return;
  if (warp == 0) {
    ptx::tmem_alloc(reinterpret_cast<uint32_t*>(sm + L::kTmem), kCols);
    ptx::tmem_relinquish();
  }

  float s[NS];
  const float* init = kBackward ? a.ds_final : a.s0;
  const size_t state_off = ((size_t)n * a.nv + h) * (size_t)DK * DV;
#pragma unroll
  for (int j = 0; j < NS; ++j) s[j] = init && active ? init[state_off + (size_t)swap32(NS * half + j) * DV + c] : 0.f;

  auto slot_of = [&](int64_t i) { return slot0 + (kBackward ? chunks - 1 - i : i); };
  auto fetch = [&](int64_t i) {  // by one thread
    if (i >= chunks) return;
    uint8_t* st = sm + (i & 1) * L::kStage;
    uint64_t* b = bar + (i & 1);
    const uint8_t* rec = rec_at<DK, DV>(a, slot_of(i), h);
    constexpr uint32_t tiles = (kBackward ? 2 : 1) * L::kTile;
    ptx::mbar_arrive_expect_tx(b, L::kTile + tiles + (kBackward ? 2 : 1) * L::kRows + 8 * C + 32);
    bulk_copy(st + L::oW, rec + R::kW, L::kTile, b);
    bulk_copy(st + L::oK, qk_at<DK, DV>(a, slot_of(i), hq) + QR::kK, tiles, b);  // Q16 stands behind K16
    bulk_copy(st + L::oU, rec + (kBackward ? R::kX : R::kV), L::kRows, b);
    if (kBackward) bulk_copy(st + L::oO, rec + R::kOq, L::kRows, b);
    bulk_copy(st + L::oF, rec + R::kF + 4 * R::fKw, 8 * C, b);  // and the factors of W behind it
    bulk_copy(st + L::oF + 8 * C, rec + R::kF + 4 * R::fScal, 32, b);
  };
  // the largest element of the state over the block; also the barrier behind which a chunk's tiles are free
  auto join_top = [&](int64_t i, bool ok) {
    const float top = warp_top(top_of(s));
    if (lane == 0) tops[8 * (i & 1) + warp] = top;
    return __syncthreads_or(!ok);
  };
  if (tid == 0) {
    for (int i = 0; i < 5; ++i) ptx::mbar_init(bar + i, i == 2 ? 2 : 1);
    ptx::fence_mbar_init();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<const uint32_t*>(sm + L::kTmem);
  const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  if (tid == 0) {
    fetch(0);
    fetch(1);
  }
  join_top(1, true);
  const uint32_t S = base + L::kS, V = base + L::kV;
  // this thread's 16-byte vectors of a row of 128 bytes: v ^ (c & 7)
  const uint32_t row = (uint32_t)c * 128, sw = (uint32_t)(c & 7);
  bool quit = false;
  for (int64_t i = 0; i < chunks; ++i) {
    uint8_t* rec = rec_at<DK, DV>(a, slot_of(i), h);
    float* rf = reinterpret_cast<float*>(rec + R::kF);
    uint8_t* st = sm + (i & 1) * L::kStage;
    const uint32_t W = base + (uint32_t)(i & 1) * L::kStage + L::oW, K = W + L::oK, Q = K + L::kTile, Oq = W + L::oO;
    const float *kw = reinterpret_cast<const float*>(st + L::oF), *wr = kw + C, *scal = wr + C;
    float sfac, sinv;
    pow2_factor(top8(tops + 8 * ((i + 1) & 1)), sfac, sinv);
    if (active) {
#pragma unroll
      for (int v = 0; v < NS / 8; ++v) {
        const uint32_t p = (uint32_t)(NS / 8 * half + v);  // vector of the row
        *reinterpret_cast<uint4*>(sm + L::kS + (p >> 3) * (128 * 128) + row + (((p & 7) ^ sw) << 4)) = pack8(s + 8 * v, sfac);
      }
    }
    bool ok = ptx::mbar_wait_bounded(bar + (i & 1), (uint32_t)((i >> 1) & 1), kWaitLimitNs);
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    if (tid == 0 || tid == 128) {
      ptx::tc_fence_after();
      const uint32_t b = kBackward ? K : W;
#pragma unroll
      for (int j = 0; j < DK / 32; ++j) {
        const int k = DK / 32 * half + j;  // step of 16 columns of Dk
        ptx::mma_bf16(tmem + 64 * half, ptx::sdesc_sw128(S + (k >> 2) * (128 * 128) + 32 * (k & 3), 16, 1024),
                      ptx::sdesc_sw128(b + (k >> 2) * (128 * C) + 32 * (k & 3), 16, 1024), idesc_f16_f32(128, 64, false, false), j > 0);
      }
      ptx::mma_commit(bar + 2);
    } else if (kBackward && tid == 64) {
      ptx::tc_fence_after();
#pragma unroll
      for (int k = 0; k < 4; ++k)
        ptx::mma_bf16(tmem + tZ, ptx::sdesc_sw128(Oq + 2048 * k, 128 * C, 1024), ptx::sdesc_sw128(Q + 2048 * k, 128 * C, 1024),
                      idesc_f16_f32(128, DK, true, true), k > 0);
      ptx::mma_commit(bar + 4);
    } else if (tid == 32) {
#pragma unroll
      for (int m = 0; m < DK / 64; ++m) bulk_store(rec + (kBackward ? R::kD : R::kS) + m * (128 * DV), S + m * (128 * 128), 128 * DV);
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      rf[R::fScal + (kBackward ? kScalD : kScalS)] = sinv;
    }
    const float us = scal[kBackward ? kScalY : kScalU], os = scal[kScalO], gl = scal[kScalGl];
    // forwards V'^T = U^T - x diag(wr), backwards dV'^T = Y^T + x diag(kw); then times the other of the two
    float x[32], w[32], vtop = 0.f, pinv = 0.f;
    uint4 u[4];
#pragma unroll
    for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4*>(w + j) = *reinterpret_cast<const float4*>((kBackward ? kw : wr) + 32 * half + j);
    if (active) {
#pragma unroll
      for (int t = 0; t < 4; ++t) u[t] = *reinterpret_cast<const uint4*>(st + L::oU + row + (((uint32_t)(4 * half + t) ^ sw) << 4));
    }
    ok = ptx::mbar_wait_bounded(bar + 2, (uint32_t)(i & 1), kWaitLimitNs) && ok;
    ptx::tc_fence_after();
    if (active) {
      float y[32];
      ptx::tmem_ld32(tl + 32 * half, x);
      ptx::tmem_ld32(tl + 64 + 32 * half, y);
      ptx::tmem_ld_wait();
      float pfac;
      const float fx = kBackward ? sinv : -sinv;
#pragma unroll
      for (int j = 0; j < 32; ++j) {  // columns j, j ^ 1 of this half stand in vector (j / 2) % 4, word j / 8
        const uint4& v = u[(j >> 1) & 3];
        const float2 u2 = unpack2(j < 8 ? v.x : j < 16 ? v.y : j < 24 ? v.z : v.w);
        x[j] = fmaf(x[j] + y[j], fx * w[j], us * (j & 1 ? u2.y : u2.x));
      }
#pragma unroll
      for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4*>(w + j) = *reinterpret_cast<const float4*>((kBackward ? wr : kw) + 32 * half + j);
#pragma unroll
      for (int j = 0; j < 32; ++j) w[j] *= x[j];
      const float ptop = top_of(w), xtop = top_of(x);
      rtops[128 * half + c] = make_float2(ptop, xtop);
      asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory");  // warps w and w + 4
      const float2 other = rtops[128 * (half ^ 1) + c];
      pow2_factor(fmaxf(ptop, other.x), pfac, pinv);
      if constexpr (kBackward) {
        vtop = fmaxf(xtop, other.y);
      } else {
        const float top = warp_top(xtop);
        if (lane == 0) vtops[warp] = top;
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) *reinterpret_cast<uint4*>(st + L::oU + row + (((uint32_t)(4 * half + t) ^ sw) << 4)) = pack8(w + 8 * t, pfac);
    } else if (!kBackward && lane == 0) {
      vtops[warp] = 0.f;
    }
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    if (tid == 32) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // S, and the last chunk's V' or dV', have left
    __syncthreads();
    if (tid == 0) {
      ptx::tc_fence_after();
      const uint32_t b = kBackward ? W : K;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        ptx::mma_bf16(tmem + tY, ptx::sdesc_sw128(W + L::oU + 32 * k, 16, 1024), ptx::sdesc_sw128(b + 2048 * k, 128 * C, 1024),
                      idesc_f16_f32(128, DK, false, true), k > 0);
      ptx::mma_commit(bar + 3);
    }
    // what does not need y, meanwhile: the image of V' or dV'
    float vfac, vinv;
    pow2_factor(kBackward ? vtop : top8(vtops), vfac, vinv);
    if (!kBackward && tid == 32) rf[R::fScal + kScalV] = vinv;
    if (active) {
      if (kBackward && half == 0) rf[R::fDV + c] = vinv;
#pragma unroll
      for (int t = 0; t < 4; ++t)
        *reinterpret_cast<uint4*>(sm + L::kV + row + (((uint32_t)(4 * half + t) ^ sw) << 4)) = pack8(x + 8 * t, vfac);
    }
    ptx::fence_proxy_async_smem();
    if constexpr (kBackward) {
      ok = ptx::mbar_wait_bounded(bar + 4, (uint32_t)(i & 1), kWaitLimitNs) && ok;
      ptx::tc_fence_after();
      if (active) {
#pragma unroll
        for (int m = 0; m < NS; m += 32) {
          ptx::tmem_ld32(tl + tZ + NS * half + m, x);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) s[m + j] = fmaf(os, x[j], gl * s[m + j]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NS; ++j) s[j] *= gl;
    }
    const float fy = kBackward ? -pinv : pinv;
    ok = ptx::mbar_wait_bounded(bar + 3, (uint32_t)(i & 1), kWaitLimitNs) && ok;
    ptx::tc_fence_after();
    if (active) {
#pragma unroll
      for (int m = 0; m < NS; m += 32) {
        ptx::tmem_ld32(tl + tY + NS * half + m, x);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) s[m + j] = fmaf(fy, x[j], s[m + j]);
      }
    }
    ptx::tc_fence_before();
    quit = join_top(i, ok);
    if (tid == 32) {
      bulk_store(rec + (kBackward ? R::kX : R::kV), V, L::kRows);
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    if (quit) {  // a copy or a product never came: report it, wait once more for what is in flight, and leave
      if (tid == 0) {
        report_status(a.status, kStatusTimeout);
        ptx::mbar_wait_bounded(bar + (i & 1), (uint32_t)((i >> 1) & 1), kWaitLimitNs);
        if (i + 1 < chunks) ptx::mbar_wait_bounded(bar + ((i + 1) & 1), (uint32_t)(((i + 1) >> 1) & 1), kWaitLimitNs);
        ptx::mbar_wait_bounded(bar + 2, (uint32_t)(i & 1), kWaitLimitNs);
        ptx::mbar_wait_bounded(bar + 3, (uint32_t)(i & 1), kWaitLimitNs);
        if (kBackward) ptx::mbar_wait_bounded(bar + 4, (uint32_t)(i & 1), kWaitLimitNs);
      }
      break;
    }
    if (tid == 0) fetch(i + 2);
  }
  if (kBackward && a.ds0 && active && !quit) {
#pragma unroll
    for (int j = 0; j < NS; ++j) a.ds0[state_off + (size_t)swap32(NS * half + j) * DV + c] = s[j];
  }
  if (tid == 32) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 0) ptx::tmem_dealloc(tmem, kCols);
}

// blockIdx.x: direction, y: v-head, z: sequence
template <int DK, int DV>
__global__ void __launch_bounds__(kStateThreads) states_half_kernel(BwdArgs a) {
  let_next_begin();
  wait_for_previous();
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (ptx::smem_u32(raw) & 1023u)) & 1023u);
  if (blockIdx.x == 0)
    walk<DK, DV, true>(a, sm, blockIdx.z, blockIdx.y);
  else
    walk<DK, DV, false>(a, sm, blockIdx.z, blockIdx.y);
}

// ------------------------------------------------------------------ 3. gradients
// One block of 16 warps per SM takes (slot, qk-head) items, and their v-heads in turn.  The tiles of the next
// v-head (of the next item, after an item's last one) are fetched by bulk copies as soon as this one's are used:
//   1. all warps: dX^T = dV'^T T
//   2. warps 0-7: dO S^T, then dA and dP; warps 8-15: V' dS'^T, then dX S^T; all: <S, dS'>
//   3. warps 0-7: N and B; warps 8-15: dV
//   4. warps 0-7: N K, and keep dq; warps 8-15: N^T Q + (B + B^T) K, and keep dk
// with a block barrier after 1 and after 3.

constexpr int kGradThreads = 512;
constexpr int kSms = 148;  // one block on each

template <int DK, int DV>
struct GradSmem {
  using R = Rec<DK, DV>;
  static constexpr size_t kX = 0;                             // dV'^T and T
  static constexpr size_t kXBytes = R::kV - R::kX;
  static constexpr size_t kV = kX + kXBytes;                  // V'^T
  static constexpr size_t kVBytes = R::kS - R::kV;
  static constexpr size_t kS = kV + kVBytes;                  // S^T, dO and dS'^T
  static constexpr size_t kSBytes = R::kW - R::kS;
  static constexpr size_t kDx = kS + kSBytes;                 // dX^T, an image [DV][C]
  static constexpr size_t kN = kDx + 2 * C * DV;              // N and B, images [C][C]
  static constexpr size_t kB = kN + 2 * C * C;
  static constexpr size_t kK = kB + 2 * C * C;                // two of: K16, Q16 (columns by swap32) and their floats
  static constexpr size_t kKBytes = QkRec<DK>::kBytes;
  static constexpr size_t kF = kK + 2 * kKBytes;              // two of: the record's floats up to fWr
  static constexpr size_t kFBytes = 4 * R::fWr;
  static constexpr size_t kE = kF + 2 * kFBytes;              // fp32 [C] e
  static constexpr size_t kRed = kE + 4 * C;                  // fp32 [3][4][C] rows' dots by column block
  static constexpr size_t kRedA = kRed + 48 * C;              // fp32 [7][C] row sums: through A and P (two halves: dgc, dbeta), dX V (two); dX V'
  static constexpr size_t kCol = kRedA + 28 * C;              // fp32 [4][C] column sums by row block
  static constexpr size_t kDot = kCol + 16 * C;               // fp32 [16] <S, dS'> by warp
  static constexpr size_t kBar = kDot + 64;                   // barriers: X, V, S, K16 and Q16 (two)
  static constexpr size_t kBytes = kBar + 40;
  static_assert(kXBytes % 128 == 0 && kK % 128 == 0 && kF % 16 == 0 && kFBytes % 16 == 0, "images and bulk copies");
  static_assert(kBytes <= 232448, "shared memory budget");
};

// The largest of n factors (powers of two), by a warp
__device__ __forceinline__ float top_factor(const float* f, int n, int lane) {
  uint32_t top = 0u;
  for (int i = lane; i < n; i += 32) top = max(top, __float_as_uint(f[i]));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, top));
}

// x[2][NT] (32 rows from m0, 8 NT columns from n0) += A B over k in [16 K0, 16 K1).
// A: an image [m][k], or [k][m]; B: an image [k][n].
template <int NT, int K0, int K1, int RA, bool kAT, int RBB>
__device__ __forceinline__ void gemm32(float (&x)[2][NT][4], uint32_t A, int m0, uint32_t B, int n0, const Lane& l) {
#pragma unroll 2
  for (int k = K0; k < K1; ++k) {
    uint32_t a0[4], a1[4];
    if (kAT) {
      img_a_t<RA>(a0, A, m0, 16 * k, l);
      img_a_t<RA>(a1, A, m0 + 16, 16 * k, l);
    } else {
      img_a<RA>(a0, A, m0, 16 * k, l);
      img_a<RA>(a1, A, m0 + 16, 16 * k, l);
    }
#pragma unroll
    for (int j = 0; j < NT; j += 2) {
      uint32_t b[4];
      img_b_t<RBB>(b, B, n0 + 8 * j, 16 * k, l);
      mma_f16(x[0][j], a0, b);
      mma_f16(x[0][j + 1], a0, b + 2);
      mma_f16(x[1][j], a1, b);
      mma_f16(x[1][j + 1], a1, b + 2);
    }
  }
}

// Rows' dots of x (as gemm32 leaves it) with an image Y, this thread's part of row m0 + 16 m + 8 e + g in dot[m][e];
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
        const float2 y = unpack2(lds32(img_word<RB>(Y, r, n0 + 8 * j + 2 * l.t, l.g)));
        dot[m][e] = fmaf(x[m][j][2 * e], y.x, fmaf(x[m][j][2 * e + 1], y.y, dot[m][e]));
        sum[m][j][2 * e] = fmaf(f[m][e], x[m][j][2 * e], sum[m][j][2 * e]);
        sum[m][j][2 * e + 1] = fmaf(f[m][e], x[m][j][2 * e + 1], sum[m][j][2 * e + 1]);
      }
    }
}

// A row's sum over the quad of lanes, to dst[row] by one of them
__device__ __forceinline__ void put_row(float v, float* dst, int t) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  if (t == 0) *dst = v;
}

template <int DK, int DV>
__global__ void __launch_bounds__(kGradThreads, 1) grads_half_kernel(BwdArgs a) {
  wait_for_previous();
  using L = GradSmem<DK, DV>;
  using R = Rec<DK, DV>;
  using QR = QkRec<DK>;
  extern __shared__ __align__(128) uint8_t sm[];
  constexpr int NT = DK / 32;        // 8-column tiles of a warp's quarter of Dk
  constexpr int KV = DV / 16;        // steps over the columns of Dv
  constexpr int RK = -C, RS = -DV, RV = 2 * DV, RC = 2 * C;  // layouts of K and Q, S and dS, dO, the rest
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Lane ln(lane);
  const bool first = warp < 8;       // warps 0-7, which keep dq
  const int w8 = warp & 7;
  const int group = a.nv / a.nqk;
  const int64_t items = slots_of<DK, DV>(a) * a.nqk;
  const uint32_t base = ptx::smem_u32(sm);
  const uint32_t X = base + L::kX, T = X + 2 * C * DV, V = base + L::kV, S = base + L::kS, O = S + 2 * DK * DV, D = O + 2 * C * DV;
  const uint32_t Dx = base + L::kDx, N = base + L::kN, B = base + L::kB;
  float* eg = reinterpret_cast<float*>(sm + L::kE);
  float *red = reinterpret_cast<float*>(sm + L::kRed), *reda = reinterpret_cast<float*>(sm + L::kRedA);
  float *col = reinterpret_cast<float*>(sm + L::kCol), *dots = reinterpret_cast<float*>(sm + L::kDot);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::kBar);

  // The next item from `w` on whose slot is not empty, its first token and tokens
  int64_t c0 = 0;
  int rows = 0;
  auto seek = [&](int64_t w, int64_t& first_token, int& tokens) {
    for (; w < items; w += gridDim.x) {
      const SlotInfo s = *slot_info<DK, DV>(a, w / a.nqk);
      first_token = s.c0;
      tokens = s.rows;
      if (s.rows > 0) break;
    }
    return w;
  };
  int64_t item = seek(blockIdx.x, c0, rows);
  if (item >= items) return;
  // by one thread; nh: v-heads taken so far, ni: items
  auto fetch_x = [&](int64_t w, int h, uint32_t nh) {
    const uint8_t* rec = rec_at<DK, DV>(a, w / a.nqk, h);
    ptx::mbar_arrive_expect_tx(bar, (uint32_t)(L::kXBytes + L::kFBytes));
    bulk_copy(sm + L::kX, rec + R::kX, L::kXBytes, bar);
    bulk_copy(sm + L::kF + (nh & 1) * L::kFBytes, rec + R::kF, L::kFBytes, bar);
  };
  auto fetch_rest = [&](int64_t w, int h) {
    const uint8_t* rec = rec_at<DK, DV>(a, w / a.nqk, h);
    ptx::mbar_arrive_expect_tx(bar + 1, (uint32_t)L::kVBytes);
    bulk_copy(sm + L::kV, rec + R::kV, L::kVBytes, bar + 1);
    ptx::mbar_arrive_expect_tx(bar + 2, (uint32_t)L::kSBytes);
    bulk_copy(sm + L::kS, rec + R::kS, L::kSBytes, bar + 2);
  };
  auto fetch_k = [&](int64_t w, uint32_t ni) {
    const uint8_t* qrec = qk_at<DK, DV>(a, w / a.nqk, (int)(w % a.nqk));
    ptx::mbar_arrive_expect_tx(bar + 3 + (ni & 1), (uint32_t)L::kKBytes);
    bulk_copy(sm + L::kK + (ni & 1) * L::kKBytes, qrec + QR::kK, L::kKBytes, bar + 3 + (ni & 1));
  };
  if (tid == 0) {
    for (int i = 0; i < 5; ++i) ptx::mbar_init(bar + i, 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();
  if (tid == 0) {
    fetch_k(item, 0);
    fetch_x(item, (int)(item % a.nqk) * group, 0);
    fetch_rest(item, (int)(item % a.nqk) * group);
  }
  // a warp's 32 rows and quarter of the columns of Dk for products with the state, its 16 rows and 32 columns of
  // the [C][C] products (warps 0-7), and its 16 rows and half of the columns of Dv for dV (warps 8-15)
  const int m0 = 32 * (w8 & 1), n0 = (DK / 4) * (w8 >> 1);
  const bool above = w8 == 4 || w8 == 5;  // rows 0..31 and columns 32..63: all above the diagonal, and never read
  if (first && above) {
    col[(w8 & 3) * C + 32 + lane] = 0.f;
    if (lane < 16) reda[2 * C + 16 * (w8 & 3) + lane] = reda[3 * C + 16 * (w8 & 3) + lane] = 0.f;
  }
  bool ok = true, quit = false;
  uint32_t nh = 0, ni = 0;
  while (item < items) {
    const int hq = (int)(item % a.nqk), h0 = hq * group;
    int64_t next = item + gridDim.x, next_c0 = 0;
    int next_rows = 0;
    if (next < items) {  // looked at when it has arrived
      const SlotInfo s = *slot_info<DK, DV>(a, next / a.nqk);
      next_c0 = s.c0;
      next_rows = s.rows;
    }
    const uint32_t K = base + L::kK + (ni & 1) * (uint32_t)L::kKBytes, Q = K + 2 * C * DK;
    const float *kf = reinterpret_cast<const float*>(sm + L::kK + (ni & 1) * L::kKBytes + 4 * C * DK), *qf = kf + C, *kn = qf + C, *qn = kn + C;
    ok &= ptx::mbar_wait_bounded(bar + 3 + (ni & 1), (ni >> 1) & 1, kWaitLimitNs);
    ln.again();
    uint32_t kk[4][2], qk[4][2];  // warps 0-7: k_r . k_i and q_r . k_i, pairs of columns in fp16 (at most 1)
    if (first && !above) {
      const int r0 = 16 * (w8 & 3) + ln.g, i0 = 32 * (w8 >> 2) + 2 * ln.t;
      float xk[4][4] = {}, xq[4][4] = {};
#pragma unroll
      for (int k = 0; k < DK; k += 16) {
        uint32_t ak[4], aq[4], b[8];
        img_a<RK>(ak, K, 16 * (w8 & 3), k, ln);
        img_a<RK>(aq, Q, 16 * (w8 & 3), k, ln);
        img_b<RK>(b, K, 32 * (w8 >> 2), k, ln);
        img_b<RK>(b + 4, K, 32 * (w8 >> 2) + 16, k, ln);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mma_f16(xk[j], ak, b + 2 * j);
          mma_f16(xq[j], aq, b + 2 * j);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = r0 + 8 * e, i = i0 + 8 * j;
          kk[j][e] = pack2(xk[j][2 * e] * kf[r] * kf[i], xk[j][2 * e + 1] * kf[r] * kf[i + 1]);
          qk[j][e] = pack2(xq[j][2 * e] * qf[r] * kf[i], xq[j][2 * e + 1] * qf[r] * kf[i + 1]);
        }
    }
    float sum[2][NT][4] = {};  // qf dq_hat (warps 0-7) or kf dk_hat (warps 8-15), over the group's v-heads

    for (int h = h0; h < h0 + group; ++h, ++nh) {
      const float* rf = reinterpret_cast<const float*>(sm + L::kF + (nh & 1) * L::kFBytes);
      const bool last = h + 1 == h0 + group;
      // ---- 1.
      ln.again();
      ok &= ptx::mbar_wait_bounded(bar, nh & 1, kWaitLimitNs);
      const float mV = rf[R::fScal + kScalV], mX = top_factor(rf + R::fDV, DV, lane);
      if (tid < C) eg[tid] = expf(rf[R::fGc + tid]);
      {  // times 2^7 for T and 2^-7: 16 columns of Dv by 16 or 32 tokens (T's zeros above the diagonal included)
        constexpr int NB = DV / 64;  // blocks of 16 tokens
        const int cb = 16 * (warp % KV), ib = 16 * NB * (warp / KV);
        const float f0 = __fdividef(rf[R::fDV + cb + ln.g], mX) * 0x1p-7f, f1 = __fdividef(rf[R::fDV + cb + ln.g + 8], mX) * 0x1p-7f;
        float x[2 * NB][4] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t af[4];
          img_a<RC>(af, X, cb, 16 * k, ln);
#pragma unroll
          for (int u = 0; u < NB; ++u) {
            uint32_t b[4];
            img_b_t<RC>(b, T, ib + 16 * u, 16 * k, ln);
            mma_f16(x[2 * u], af, b);
            mma_f16(x[2 * u + 1], af, b + 2);
          }
        }
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j) {
          sts32(img_word<RC>(Dx, cb + ln.g, ib + 8 * j + 2 * ln.t, ln.g), pack2(x[j][0] * f0, x[j][1] * f0));
          sts32(img_word<RC>(Dx, cb + ln.g + 8, ib + 8 * j + 2 * ln.t, ln.g), pack2(x[j][2] * f1, x[j][3] * f1));
        }
      }
      quit = __syncthreads_or(!ok);
      if (quit) break;
      if (h == h0) {
        if (next < items && next_rows == 0) next = seek(next + gridDim.x, next_c0, next_rows);
        if (tid == 0 && next < items) fetch_k(next, ni + 1);  // its buffer was last read before the item before ended
      }
      if (tid == 0 && (!last || next < items))
        fetch_x(last ? next : item, last ? (int)(next % a.nqk) * group : h + 1, nh + 1);
      // ---- 2.
      ln.again();
      ok &= ptx::mbar_wait_bounded(bar + 1, nh & 1, kWaitLimitNs);
      ok &= ptx::mbar_wait_bounded(bar + 2, nh & 1, kWaitLimitNs);
      const float mS = rf[R::fScal + kScalS], mD = rf[R::fScal + kScalD], oinv = rf[R::fScal + kScalDo];
      {  // <S, dS'>: the diagonal of S^T dS', 16 columns of Dv and a share of Dk a warp
        constexpr int KS = DK * KV / 256;  // steps of a share
        const int cb = 16 * (warp % KV), k0 = KS * (warp / KV);
        float x[2][4] = {};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t af[4], b[4];
          img_a<RS>(af, S, cb, 16 * (k0 + k), ln);
          img_b<RS>(b, D, cb, 16 * (k0 + k), ln);
          mma_f16(x[0], af, b);
          mma_f16(x[1], af, b + 2);
        }
        const float d = warp_sum((2 * ln.t == ln.g ? x[0][0] + x[1][2] : 0.f) + (2 * ln.t + 1 == ln.g ? x[0][1] + x[1][3] : 0.f));
        if (lane == 0) dots[warp] = d * mS * mD;
      }
      const float sP = oinv * mV, sA = mX * mV;
      if (first) {
        float f[2][2], dot[2][2];
        {
          float x[2][NT][4] = {};
          gemm32<NT, 0, KV, RV, false, RS>(x, O, m0, S, n0, ln);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = m0 + 16 * m + 8 * e + ln.g;
              f[m][e] = a.scale * eg[r] * qf[r] * oinv * mS;
            }
          take<NT, RK>(x, Q, m0, n0, f, sum, dot, ln);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) put_row(f[m][e] * dot[m][e], red + (w8 >> 1) * C + m0 + 16 * m + 8 * e + ln.g, ln.t);
        if (!above) {
          ln.again();
          const int r0 = 16 * (w8 & 3) + ln.g, i0 = 32 * (w8 >> 2) + 2 * ln.t;
          float dA[4][4] = {}, dP[4][4] = {};
#pragma unroll
          for (int k = 0; k < KV; ++k) {
            uint32_t ax[4], ao[4], b[8];
            img_a_t<RC>(ax, Dx, 16 * (w8 & 3), 16 * k, ln);
            img_a<RV>(ao, O, 16 * (w8 & 3), 16 * k, ln);
            img_b_t<RC>(b, V, 32 * (w8 >> 2), 16 * k, ln);
            img_b_t<RC>(b + 4, V, 32 * (w8 >> 2) + 16, 16 * k, ln);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              mma_f16(dA[j], ax, b + 2 * j);
              mma_f16(dP[j], ao, b + 2 * j);
            }
          }
          if ((w8 & 3) >> 1 == w8 >> 2 && ln.t == ln.g >> 1) {  // the diagonal: dX_r . V'_r of rows r0 and r0 + 8
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x0 = w8 & 1 ? dA[2 + e][2 * e] : dA[e][2 * e], x1 = w8 & 1 ? dA[2 + e][2 * e + 1] : dA[e][2 * e + 1];
              reda[6 * C + r0 + 8 * e] = sA * (ln.g & 1 ? x1 : x0);
            }
          }
          // ---- 3. what goes through A and P
          const float *gc = rf + R::fGc, *bt = rf + R::fBeta;
          float s_gc[2] = {0.f, 0.f}, s_bt[2] = {0.f, 0.f}, gr[2], br[2], qr[2], kr[2], cs[8];
          float2 gi[4], ki[4];
          constexpr float kLog2e = 1.44269504f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            gi[j] = *reinterpret_cast<const float2*>(gc + i0 + 8 * j);
            ki[j] = *reinterpret_cast<const float2*>(kf + i0 + 8 * j);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            gr[e] = gc[r0 + 8 * e];
            br[e] = -bt[r0 + 8 * e];
            qr[e] = qf[r0 + 8 * e] * 0x1p6f;    // 2^14 for the factors, 2^-8
            kr[e] = kf[r0 + 8 * e] * 0x1p-2f;   // 2^14, 2^-16
          }
          const float sQ = a.scale * sP;
#pragma unroll
          for (int j = 0; j < 4; ++j)  // hidden as in Lane::again, or they would be kept unpacked
#pragma unroll
            for (int e = 0; e < 2; ++e) asm volatile("" : "+r"(kk[j][e]), "+r"(qk[j][e]));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = i0 + 8 * j;
            cs[2 * j] = cs[2 * j + 1] = 0.f;
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
              const int r = r0 + 8 * e2;
              const float2 kd2 = unpack2(kk[j][e2]), qk2 = unpack2(qk[j][e2]);
              float nn[2], bb[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // masked before exp, and the difference before the factor: 1 on the diagonal; the strict triangle for A
                const float gamma = i + e <= r ? ptx::ex2_approx(kLog2e * (gr[e2] - (e ? gi[j].y : gi[j].x))) : 0.f;
                const float strict = i + e < r ? gamma : 0.f, kc = e ? ki[j].y : ki[j].x;
                const float dp = dP[j][2 * e2 + e], da = dA[j][2 * e2 + e];
                const float akd = sA * da * ((e ? kd2.y : kd2.x) * strict);
                const float both = fmaf(br[e2], akd, sQ * dp * strict * (e ? qk2.y : qk2.x));
                s_bt[e2] -= akd;
                s_gc[e2] += both;
                cs[2 * j + e] += both;
                nn[e] = dp * gamma * (qr[e2] * kc);
                bb[e] = da * br[e2] * strict * (kr[e2] * kc);
              }
              sts32(img_word<RC>(N, r, i, ln.g), pack2(nn[0], nn[1]));
              sts32(img_word<RC>(B, r, i, ln.g), pack2(bb[0], bb[1]));
            }
          }
          // eight columns over eight rows of lanes: a lane passes on half of what it has, and ends with one column
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) {
            const bool upper = ln.g & o;
#pragma unroll
            for (int m = 0; m < o; ++m) {
              const float give = upper ? cs[m] : cs[m + o], keep = upper ? cs[m + o] : cs[m];
              cs[m] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * o);
            }
          }
          col[(w8 & 3) * C + i0 + 8 * (ln.g >> 1) + (ln.g & 1)] = cs[0];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            put_row(s_gc[e], reda + (2 * (w8 >> 2)) * C + r0 + 8 * e, ln.t);
            put_row(s_bt[e], reda + (2 * (w8 >> 2) + 1) * C + r0 + 8 * e, ln.t);
          }
        }
      } else {
        float f[2][2], dot[2][2];
        {
          float x[2][NT][4] = {};
          gemm32<NT, 0, KV, RC, true, RS>(x, V, m0, D, n0, ln);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = m0 + 16 * m + 8 * e + ln.g;
              f[m][e] = rf[R::fKw + r] * mV * mD;
            }
          take<NT, RK>(x, K, m0, n0, f, sum, dot, ln);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) put_row(f[m][e] * dot[m][e], red + (4 + (w8 >> 1)) * C + m0 + 16 * m + 8 * e + ln.g, ln.t);
        ln.again();
        const int r0 = 16 * (w8 & 3) + ln.g;
        // this thread's share of V: rows r0, r0 + 8, columns 16 k + 2 t, + 8 of its half of the steps
        const int k0 = (KV / 2) * (w8 >> 2);
        uint32_t vraw[KV / 2][4];
#pragma unroll
        for (int k = 0; k < KV / 2; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = r0 + 8 * (e & 1), c = 16 * (k0 + k) + 8 * (e >> 1) + 2 * ln.t;
            vraw[k][e] = r < rows ? *reinterpret_cast<const uint32_t*>(static_cast<const bf16*>(a.v) + ((size_t)(c0 + r) * a.nv + h) * DV + c) : 0u;
          }
        {
          float x[2][NT][4] = {};
          gemm32<NT, 0, KV, RC, true, RS>(x, Dx, m0, S, n0, ln);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = m0 + 16 * m + 8 * e + ln.g;
              f[m][e] = -rf[R::fBeta + r] * eg[r] * kf[r] * mX * mS;
            }
          take<NT, RK>(x, K, m0, n0, f, sum, dot, ln);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = m0 + 16 * m + 8 * e + ln.g;
            put_row(-eg[r] * kf[r] * mX * mS * dot[m][e], red + (8 + (w8 >> 1)) * C + r, ln.t);
          }
        ln.again();
        // ---- 3. dV = diag(b) dX and its part of dbeta
        float s_v[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KV / 2; ++k) {
          uint32_t w[4];
          img_a_t<RC>(w, Dx, 16 * (w8 & 3), 16 * (k0 + k), ln);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 d = unpack2(w[e]);
            d.x *= mX;
            d.y *= mX;
            const float2 v = bf2(vraw[k][e]);
            s_v[e & 1] = fmaf(d.x, v.x, fmaf(d.y, v.y, s_v[e & 1]));
            const float b = rf[R::fBeta + r0 + 8 * (e & 1)];
            w[e] = ptx::pack_bf16x2(b * d.x, b * d.y);
          }
          // lane t of a quad takes all four pairs of word t: a vector of 8 columns
          const bool odd = ln.t & 1, up = ln.t & 2;
          const uint32_t p0 = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1), p1 = __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
          const uint32_t a0 = odd ? p0 : w[0], a1 = odd ? w[1] : p0, b0 = odd ? p1 : w[2], b1 = odd ? w[3] : p1;
          const uint32_t q0 = __shfl_xor_sync(0xffffffffu, up ? a0 : b0, 2), q1 = __shfl_xor_sync(0xffffffffu, up ? a1 : b1, 2);
          const int r = r0 + 8 * (ln.t & 1), c = 16 * (k0 + k) + 8 * (ln.t >> 1);
          if (r < rows)
            *reinterpret_cast<uint4*>(static_cast<bf16*>(a.dv_out) + ((size_t)(c0 + r) * a.nv + h) * DV + c) =
                up ? make_uint4(q0, q1, b0, b1) : make_uint4(a0, a1, q0, q1);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) put_row(s_v[e], reda + (4 + (w8 >> 2)) * C + r0 + 8 * e, ln.t);
      }
      ptx::fence_proxy_async_smem();  // the tiles' generic reads come before the copies over them
      __syncthreads();
      if (tid == 0 && (!last || next < items)) fetch_rest(last ? next : item, last ? (int)(next % a.nqk) * group : h + 1);
      // ---- 4.
      ln.again();
      if (first) {
        float x[2][NT][4] = {};
        if (m0 == 0)
          gemm32<NT, 0, 2, RC, false, RK>(x, N, m0, K, n0, ln);
        else
          gemm32<NT, 0, 4, RC, false, RK>(x, N, m0, K, n0, ln);
        const float sN = a.scale * sP * 0x1p-6f;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[m][j][e] = fmaf(sN, x[m][j][e], sum[m][j][e]);
      } else {
        float x[2][NT][4] = {};
        if (m0 == 0)
          gemm32<NT, 0, 4, RC, true, RK>(x, N, m0, Q, n0, ln);
        else
          gemm32<NT, 2, 4, RC, true, RK>(x, N, m0, Q, n0, ln);
        const float sN = a.scale * sP * 0x1p-6f, sB = sA * 0x1p2f;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              sum[m][j][e] = fmaf(sN, x[m][j][e], sum[m][j][e]);
              x[m][j][e] = 0.f;
            }
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
      if (warp == 0 || warp == 2) {  // two of the warps whose product above was the shorter: rows 2 lane, 2 lane + 1 of dg and dbeta
        auto add = [](float2 x, float2 y) { return make_float2(x.x + y.x, x.y + y.y); };
        auto pair = [&](const float* x) { return *reinterpret_cast<const float2*>(x + 2 * lane); };
        auto four = [&](const float* x) { return add(add(pair(x), pair(x + C)), add(pair(x + 2 * C), pair(x + 3 * C))); };
        const float2 b = pair(rf + R::fBeta), u = four(red + 8 * C);
        float2 out;
        if (warp == 0) {
          // dgc; then the suffix sums.  l_r k_r . (V' dS'^T)_r is taken from dgc_r and added to the last row: in dg_t only
          // the rows before t are left of it, and are added as such, since the difference of the two sums would have no
          // digits where a chunk's own decay is small beside it (one token behind a strong gate).
          const float2 th = four(red + 4 * C), cols = four(col), r0 = four(red), ra = add(pair(reda), pair(reda + 2 * C));
          const float d[2] = {ra.x + r0.x + b.x * u.x - cols.x, ra.y + r0.y + b.y * u.y - cols.y};
          const float dsum = warp_sum(lane < 16 ? dots[lane] : 0.f) * rf[R::fScal + kScalGl];
          float suf = d[0] + d[1], pre = th.x + th.y;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_down_sync(0xffffffffu, suf, o), z = __shfl_up_sync(0xffffffffu, pre, o);
            if (lane + o < 32) suf += y;
            if (lane >= o) pre += z;
          }
          float beyond = __shfl_down_sync(0xffffffffu, suf, 1), before = __shfl_up_sync(0xffffffffu, pre, 1);
          if (lane == 31) beyond = 0.f;
          if (lane == 0) before = 0.f;
          out = make_float2(suf + (before + dsum), beyond + d[1] + (before + th.x + dsum));
        } else {
          // V' = diag(b) (V - diag(e) K S - Kd V'), so dbeta_r = dX_r . V'_r / b_r: no difference of large terms where keys
          // repeat.  A small b_r leaves V'_r few digits beside the tile's largest: there, and for 0, the terms one by one
          const float2 xv = pair(reda + 6 * C), sum = add(add(add(pair(reda + C), pair(reda + 3 * C)), add(pair(reda + 4 * C), pair(reda + 5 * C))), u);
          out = make_float2(b.x >= 0x1p-10f ? __fdividef(xv.x, b.x) : sum.x, b.y >= 0x1p-10f ? __fdividef(xv.y, b.y) : sum.y);
        }
        bf16* dst = static_cast<bf16*>(warp == 0 ? a.dg : a.dbeta) + (size_t)(c0 + 2 * lane) * a.nv + h;
        if (2 * lane < rows) dst[0] = __float2bfloat16_rn(out.x);
        if (2 * lane + 1 < rows) dst[a.nv] = __float2bfloat16_rn(out.y);
      }
    }
    if (quit) break;
    __syncthreads();  // the last v-head's sums are read
    ln.again();
    // the norms: with y = qf dq_hat, dq = (y - qf^2 Q16 (Q16 . y)) / (qf |q|), and dk alike
    {
      const uint32_t Y = first ? Q : K;
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
            const float2 y = unpack2(lds32(img_word<RK>(Y, r, n0 + 8 * j + 2 * ln.t, ln.g)));
            dot = fmaf(sum[m][j][2 * e], y.x, fmaf(sum[m][j][2 * e + 1], y.y, dot));
          }
          put_row(dot, part + (w8 >> 1) * C + r, ln.t);
        }
      __syncthreads();
      bf16* out = static_cast<bf16*>(first ? a.dq : a.dk);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = m0 + 16 * m + 8 * e + ln.g;
          const float p = yf[r] * yf[r] * ((part[r] + part[C + r]) + (part[2 * C + r] + part[3 * C + r])), fn = yn[r];
          uint32_t w[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const float2 y = unpack2(lds32(img_word<RK>(Y, r, n0 + 8 * j + 2 * ln.t, ln.g)));
            w[j] = ptx::pack_bf16x2(fn * (sum[m][j][2 * e] - y.x * p), fn * (sum[m][j][2 * e + 1] - y.y * p));
          }
          // by swap32 this thread's pairs are neighbours: 8 columns (Dk = 128) or 4 (Dk = 64)
          if (r < rows) {
            bf16* dst = out + ((size_t)(c0 + r) * a.nqk + hq) * DK + swap32(n0 + 2 * ln.t);
            if constexpr (NT == 4)
              *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            else
              *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
          }
        }
    }
    item = next;
    c0 = next_c0;
    rows = next_rows;
    ++ni;
    __syncthreads();  // the sums and the floats of this item's last v-head are read
  }
  if (quit && tid == 0) {  // a copy never came: report it, wait once more for what is in flight, and leave
    report_status(a.status, kStatusTimeout);
    for (int i = 0; i < 3; ++i) ptx::mbar_wait_bounded(bar + i, nh & 1, kWaitLimitNs);
    for (uint32_t i = ni; i < ni + 2; ++i) ptx::mbar_wait_bounded(bar + 3 + (i & 1), (i >> 1) & 1, kWaitLimitNs);
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
    prepare_half_kernel<DK, DV><<<slot_grid(slots, a.nqk), kPrepThreads, PrepSmem<DK, DV>::kBytes, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = set_smem(states_half_kernel<DK, DV>, StateSmem<DK, DV>::kBytes)) != cudaSuccess) return e;
  e = launch_next(states_half_kernel<DK, DV>, dim3(2, a.nv, a.num_seqs), kStateThreads, StateSmem<DK, DV>::kBytes, stream, a);
  if (e != cudaSuccess || a.total_tokens == 0) return e;
  if ((e = set_smem(grads_half_kernel<DK, DV>, GradSmem<DK, DV>::kBytes)) != cudaSuccess) return e;
  const int64_t items = (int64_t)slots * a.nqk;
  const unsigned int grid = (unsigned int)(items < kSms ? items : kSms);
  return launch_next(grads_half_kernel<DK, DV>, grid, kGradThreads, GradSmem<DK, DV>::kBytes, stream, a);
}

}  // namespace bwdh

int64_t chunk_bwd_half_workspace(int64_t total_tokens, int num_seqs, int nqk, int nv, int dk, int dv) {
  if (total_tokens == 0) return 0;
  const int64_t c = bwdh::C, slots = total_tokens / c + num_seqs;
  const int64_t rec = 2 * (c * (c + dk + 4 * dv) + 2 * (int64_t)dk * dv) + 4 * (4 * c + 8 + dv);
  return slots * (nv * rec + nqk * (4 * c * dk + 16 * c) + (int64_t)sizeof(bwdh::SlotInfo));
}

cudaError_t launch_chunk_bwd_half(const BwdArgs& a, int dk, int dv, cudaStream_t s) {
  static_assert(bwdh::Rec<128, 64>::kBytes == 2 * (64 * (64 + 128 + 4 * 64) + 2 * 128 * 64) + 4 * (4 * 64 + 8 + 64), "workspace size");
  static_assert(bwdh::QkRec<128>::kBytes == 4 * 64 * 128 + 16 * 64, "workspace size");
  if (dk == 64 && dv == 64) return bwdh::launch_one<64, 64>(a, s);
  if (dk == 64 && dv == 128) return bwdh::launch_one<64, 128>(a, s);
  if (dk == 128 && dv == 64) return bwdh::launch_one<128, 64>(a, s);
  if (dk == 128 && dv == 128) return bwdh::launch_one<128, 128>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace gdn
