// chunk_bwd.cuh -- what the two kernel families of gdn_chunk_bwd share: chunk
// slots, the split-TF32 warp product, the in-chunk cumsum, the inverse, and fp16
// products of tiles that bulk copies bring in.
#pragma once

#include <cuda_fp16.h>

#include "train_common.cuh"
#include "sm100_ptx.cuh"

namespace gdn {
namespace bwd {

constexpr int C = 64;           // tokens per chunk
constexpr int TP = C + 4;       // pitch of fp32 [C][C] tiles

// Chunks are numbered by slots: chunk c of sequence n has slot cu[n] / C + n + c.
// Slots of different sequences never meet (cu[n] / C + ceil(len / C) <= cu[n + 1] / C + 1),
// and there are at most T / C + N of them.
// The chunk at a slot: its sequence's end and its first token; false where the slot is empty.  By whole warps: 32
// sequences are looked at together, so that a block waits for two or three loads and not for log2 of the sequences.
template <class Args>
__device__ __forceinline__ bool chunk_at(const Args& a, int64_t slot, int64_t& c0, int64_t& end) {
  const int lane = threadIdx.x & 31;
  int lo = 0, count = a.num_seqs;  // the last sequence of [lo, lo + count) whose first slot is not beyond `slot`
  int64_t s, e;
  while (true) {
    const int step = (count + 31) / 32, n = lo + lane * step;
    const bool in = lane * step < count;
    s = e = 0;
    if (in) seq_bounds_quiet(a, n, s, e);
    const unsigned int before = __ballot_sync(0xffffffffu, in && s / C + n <= slot);
    const int last = before ? 31 - __clz(before) : 0;
    lo += last * step;
    if (step == 1) {
      s = __shfl_sync(0xffffffffu, s, last);
      e = __shfl_sync(0xffffffffu, e, last);
      break;
    }
    count = min(step, count - last * step);
  }
  end = e;
  c0 = s + (slot - (s / C + lo)) * C;
  return c0 >= s && c0 < end;
}

// Slots and qk-heads of a grid whose blocks of one chunk follow one another, so that they share DRAM pages
__device__ __forceinline__ int64_t grid_slot() { return (int64_t)blockIdx.z * 65535 + blockIdx.y; }
static inline dim3 slot_grid(int64_t slots, int nqk) {
  return dim3((unsigned int)nqk, (unsigned int)(slots < 65535 ? slots : 65535), (unsigned int)((slots + 65534) / 65535));
}

// x as hi + lo of TF32: rounded, within 2^-22 of x, or (kCut) cut off by masks, within 2^-21 and always towards zero.
// Cutting is what the kernels with fp16 operands do, which keep 11 bits of what comes of it: prepare takes 5 % less there.
// For those with pairs it is too little: where keys repeat, the gradients' errors were three to eight times as large.
template <bool kCut>
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  if constexpr (kCut) {
    hi = __float_as_uint(x) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
  } else {
    hi = ptx::to_tf32(x);
    lo = ptx::to_tf32(x - __uint_as_float(hi));
  }
}

// acc (a 16 x 8 tile) += A[16 x K] B[K x 8] over k in [k0, k1), one warp; a(m, k) and b(k, n) read the operands'
// elements, which are split into hi + lo: three MMAs, whose 8 terms are added in fp32, since an MMA truncates as it adds.
template <bool kCut, typename FA, typename FB>
__device__ __forceinline__ void warp_gemm(float (&acc)[4], int k0, int k1, FA a, FB b, int g, int t) {
#pragma unroll 2
  for (int kk = k0; kk < k1; kk += 8) {
    uint32_t ah[4], al[4], bh[2], bl[2];
    split_tf32<kCut>(a(g, kk + t), ah[0], al[0]);
    split_tf32<kCut>(a(g + 8, kk + t), ah[1], al[1]);
    split_tf32<kCut>(a(g, kk + t + 4), ah[2], al[2]);
    split_tf32<kCut>(a(g + 8, kk + t + 4), ah[3], al[3]);
    split_tf32<kCut>(b(kk + t, g), bh[0], bl[0]);
    split_tf32<kCut>(b(kk + t + 4, g), bh[1], bl[1]);
    float d[4] = {}, e[4] = {};
    ptx::mma_tf32_16x8x8(e, al, bh);
    ptx::mma_tf32_16x8x8(d, ah, bh);
    ptx::mma_tf32_16x8x8(e, ah, bl);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += d[i] + e[i];
  }
}

// A gate below this decays to 0 in fp32, as this one does (exp(-105) < 2^-150).  It is raised to it, so that sums of gates
// stay where their differences keep digits: a token's decay from the ones behind a reset must not depend on the reset.
constexpr float kGateFloor = -105.f;

// In-chunk inclusive cumsum of x[0..C) by one warp.
__device__ __forceinline__ void cumsum_chunk(float* x, int lane) {
  const float x0 = x[2 * lane], x1 = x[2 * lane + 1];
  float incl = x0 + x1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  float excl = __shfl_up_sync(0xffffffffu, incl, 1);
  if (lane == 0) excl = 0.f;
  x[2 * lane] = excl + x0;
  x[2 * lane + 1] = excl + x0 + x1;
}
// hi + lo += x + y, without a rounding but lo's
__device__ __forceinline__ void add_pair(float& hi, float& lo, float x, float y) {
  const float s = hi + x, b = s - hi;
  lo += y + ((hi - (s - b)) + (x - b));
  hi = s;
}
// The same as a pair hi + lo, so that differences are exact to fp32 however large the sums; gates of either sign: what the
// chunk's positive ones add up to lowers the floor.
__device__ __forceinline__ void cumsum_chunk(float* x, float* low, int lane) {
  float x0 = x[2 * lane], x1 = x[2 * lane + 1];
  const float least = kGateFloor - warp_sum(fmaxf(x0, 0.f) + fmaxf(x1, 0.f));
  x0 = x0 < least ? least : x0;
  x1 = x1 < least ? least : x1;
  float hi = x0, lo = 0.f;
  add_pair(hi, lo, x1, 0.f);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_up_sync(0xffffffffu, hi, o), z = __shfl_up_sync(0xffffffffu, lo, o);
    if (lane >= o) add_pair(hi, lo, y, z);
  }
  float eh = __shfl_up_sync(0xffffffffu, hi, 1), el = __shfl_up_sync(0xffffffffu, lo, 1);
  if (lane == 0) eh = el = 0.f;
  add_pair(eh, el, x0, 0.f);
  x[2 * lane] = eh;
  low[2 * lane] = el;
  x[2 * lane + 1] = hi;
  low[2 * lane + 1] = lo;
}

// T = (I - A)^-1 over A (strictly lower, pitch TP), as in chunk_simt.cu: 16 x 16
// diagonal blocks by forward substitution in fp32 (a warp per block, a column
// per lane), then T10 = T11 A10 T00 for blocks of 16 and of 32.  Y: [C / 2][TP]
// scratch.  Zeros above the diagonal are written; the unit diagonal is stored.
template <bool kCut>
__device__ __forceinline__ void invert_chunk(float* A, float* Y, int warp, int lane) {
  if (warp < C / 16 && lane < 16) {
    float* blk = A + (16 * warp) * TP + 16 * warp;
    const int jc = lane;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float acc = (jc < i) ? blk[i * TP + jc] : 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m)
        if (m > jc) acc = fmaf(blk[i * TP + m], x[m], acc);
      x[i] = acc;
    }
    __syncwarp(0x0000ffffu);
#pragma unroll
    for (int i = 0; i < 16; ++i) blk[i * TP + jc] = jc < i ? x[i] : (jc == i ? 1.f : 0.f);
  }
  __syncthreads();
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int s = 16; s < C; s *= 2) {
    const int nb = s / 16, nunit = (C / (2 * s)) * nb * nb * 2;  // 16 x 8 blocks of all T10 of this size
    const int u = warp / 2, p = u / (nb * nb), rb = (u / nb) % nb, c0 = 16 * (u % nb) + 8 * (warp & 1), base = 2 * s * p;
    if (warp < nunit) {  // Y = A10 T00
      const float* a10 = A + (base + s + 16 * rb) * TP + base;
      const float* t00 = A + base * TP + base + c0;
      float acc[4] = {};
      warp_gemm<kCut>(acc, c0, s, [&](int m, int k) { return a10[m * TP + k]; }, [&](int k, int n) { return t00[k * TP + n]; }, g, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) Y[(p * s + 16 * rb + g + 8 * (e >> 1)) * TP + c0 + 2 * t + (e & 1)] = acc[e];
    }
    __syncthreads();
    if (warp < nunit) {  // T10 = T11 Y
      const float* t11 = A + (base + s + 16 * rb) * TP + base + s;
      const float* yp = Y + p * s * TP + c0;
      float acc[4] = {};
      warp_gemm<kCut>(acc, 0, 16 * rb + 16, [&](int m, int k) { return t11[m * TP + k]; }, [&](int k, int n) { return yp[k * TP + n]; }, g, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) A[(base + s + 16 * rb + g + 8 * (e >> 1)) * TP + base + c0 + 2 * t + (e & 1)] = acc[e];
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ fp16 products from images
// An image is a tile of fp16 as it stands in shared memory, so that one bulk copy brings it in: rows of 128 or 256
// bytes whose 16-byte vectors are swapped by their row (vector v of row r at v ^ (r & 7)), which keeps ldmatrix free
// of bank conflicts without padding.

// Layout RB > 0: rows of RB bytes; -RB > 0: panels of 64 columns, -RB rows of 128 bytes each, the 128-byte swizzle
// of the tcgen05 operand descriptors (sm100_ptx.cuh).
template <int RB> constexpr int kRowBytes = RB > 0 ? RB : 128;
template <int RB> constexpr int kPanel = RB > 0 ? 128 : -RB * 128;  // from one 64 columns to the next
// Where element (r, col) of an image stands, in bytes.
template <int RB> __device__ __forceinline__ int image(int r, int col) {
  return r * kRowBytes<RB> + (col >> 6) * kPanel<RB> + (((((col >> 3) & 7) ^ (r & 7)) << 4) | ((col & 7) * 2));
}
// Column d of a row of 32 stands at swap32(d): lane t's columns 8 b + 2 t, + 1 of the states' accumulators
// (b = 0..3) are next to one another, so that they are stored as one vector.  Pairs stay pairs, and the swap is its
// own inverse.
__device__ __forceinline__ int swap32(int d) { return (d & ~31) | (((d >> 1) & 3) << 3) | (((d >> 3) & 3) << 1) | (d & 1); }

// Four lanes' vectors of four words each: lane m gets word m of all
__device__ __forceinline__ void transpose4(uint4& v, int lane) {
  const bool odd = lane & 1, high = lane & 2;
  const uint32_t a = __shfl_xor_sync(0xffffffffu, odd ? v.x : v.y, 1), b = __shfl_xor_sync(0xffffffffu, odd ? v.z : v.w, 1);
  if (odd) { v.x = a; v.z = b; } else { v.y = a; v.w = b; }
  const uint32_t c = __shfl_xor_sync(0xffffffffu, high ? v.x : v.z, 2), d = __shfl_xor_sync(0xffffffffu, high ? v.y : v.w, 2);
  if (high) { v.x = c; v.y = d; } else { v.z = c; v.w = d; }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
// f = 2^k with top f in [2^7, 2^8), and 1 / f.  Magnitudes below 2^-119 count as 2^-119; an infinite or
// NaN `top` gives a finite factor, so such values stay what they are.
__device__ __forceinline__ void pow2_factor(float top, float& f, float& inv) {
  const uint32_t e = max((__float_as_uint(top) >> 23) & 255u, 8u);
  f = __uint_as_float((261u - e) << 23);
  inv = __uint_as_float((e - 7u) << 23);
}

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
// What a lane adds to the address of a fragment in an image: its row and the swap of the 16-byte vectors (m0, n0 and
// k0 are multiples of 16, so a lane's row is lane & 7 mod 8).  `again` hides the values from the compiler, which
// would otherwise form the addresses of every product ahead of the loop around them, and spill them.
struct Lane {
  uint32_t ra, rb, sa, sb;   // rows of kind a (lane & 15) and b, and their swaps
  int g, t;
  __device__ __forceinline__ explicit Lane(int lane)
      : ra(lane & 15), rb((lane & 7) + 8 * (lane >> 4)), sa(((lane >> 4) ^ (lane & 7)) << 4),
        sb((((lane >> 3) & 1) ^ (lane & 7)) << 4), g(lane >> 2), t(lane & 3) {}
  __device__ __forceinline__ void again() {
    asm volatile("" : "+r"(ra), "+r"(rb), "+r"(sa), "+r"(sb), "+r"(g), "+r"(t));
  }
};
// kPair: the image is a pair hi, lo, in blocks of 16 rows, hi then lo (see chunk_bwd.cu); `row` is a multiple of 16.
template <int RB, bool kPair = false>
__device__ __forceinline__ uint32_t img_addr(uint32_t img, int row, int col, uint32_t r, uint32_t s) {
  return img + (uint32_t)(row * kRowBytes<RB> * (kPair ? 2 : 1)) + r * kRowBytes<RB> + (((((uint32_t)col >> 3) & 7u) << 4) ^ s) +
         ((uint32_t)col >> 6) * kPanel<RB>;
}
// By address, without a memory clobber: volatile statements and barriers keep their order, and images are written
// and read by such statements only, or on two sides of a barrier.
__device__ __forceinline__ void ldsm(uint32_t* r, uint32_t p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(p));
}
__device__ __forceinline__ void ldsm_t(uint32_t* r, uint32_t p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(p));
}
template <int RB> __device__ __forceinline__ void img_a(uint32_t* r, uint32_t img, int m0, int k0, const Lane& l) {
  ldsm(r, img_addr<RB>(img, m0, k0, l.ra, l.sa));
}
template <int RB> __device__ __forceinline__ void img_a_t(uint32_t* r, uint32_t img, int m0, int k0, const Lane& l) {
  ldsm_t(r, img_addr<RB>(img, k0, m0, l.rb, l.sb));
}
template <int RB> __device__ __forceinline__ void img_b(uint32_t* r, uint32_t img, int n0, int k0, const Lane& l) {
  ldsm(r, img_addr<RB>(img, n0, k0, l.rb, l.sb));
}
template <int RB> __device__ __forceinline__ void img_b_t(uint32_t* r, uint32_t img, int n0, int k0, const Lane& l) {
  ldsm_t(r, img_addr<RB>(img, k0, n0, l.ra, l.sa));
}
// Words of an image in shared memory: row r (r & 7 = g), columns col, col + 1
template <int RB> __device__ __forceinline__ uint32_t img_word(uint32_t img, int r, int col, int g) {
  return img + (uint32_t)(r * kRowBytes<RB> + ((((((col >> 3) & 7) ^ (g & 7)) << 4) | ((col & 7) * 2)) + (col >> 6) * kPanel<RB>));
}
__device__ __forceinline__ uint32_t lds32(uint32_t p) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(p));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t p, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(p), "r"(v)); }

// A bulk copy from global to shared memory that completes on `bar` (sizes and addresses: multiples of 16 bytes).
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   ptx::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
               : "memory");
}
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // as in chunk_tc.cu

}  // namespace bwd
}  // namespace gdn
