// train_common.cuh -- arguments of the training kernels, and what they share beyond gdn_common.cuh.
#pragma once

#include <cuda_runtime.h>

#include "gdn_common.cuh"
#include "sm100_ptx.cuh"

namespace gdn {

// Arguments of the gradients of the chunked forward (gdn_chunk_bwd).
struct BwdArgs {
  const void* q;             // [T, Nqk, Dk]
  const void* k;             // [T, Nqk, Dk]
  const void* v;             // [T, Nv, Dv]
  const float* g;            // [T, Nv]: g, or the raw projection a when A_log != nullptr
  const float* beta;         // [T, Nv]: beta, or the raw projection b when A_log != nullptr
  const float* A_log;        // [Nv] or nullptr (g and beta given)
  const float* dt_bias;      // [Nv] (used with A_log)
  const void* dout;          // [T, Nv, Dv]
  const float* s0;           // [N, Nv, Dk, Dv] or nullptr
  const float* ds_final;     // [N, Nv, Dk, Dv] or nullptr
  const int32_t* cu;         // [N + 1] or nullptr (equal lengths)
  void* dq;                  // [T, Nqk, Dk] outputs
  void* dk;
  void* dv_out;              // [T, Nv, Dv]
  void* dg;                  // [T, Nv] in the io dtype
  void* dbeta;               // [T, Nv] in the io dtype
  float* ds0;                // [N, Nv, Dk, Dv] or nullptr
  float* ws;                 // workspace (chunk_bwd_workspace bytes)
  int32_t uniform_len;       // sequence length when cu == nullptr
  int32_t num_seqs;
  int64_t total_tokens;
  unsigned int* status;      // device status word (kStatus* bits)
  int32_t nqk, nv;
  int32_t qk_l2norm;
  float scale;
};

// Arguments of the gradients of the gated RMSNorm (gdn_gated_rmsnorm_bwd).
struct NormBwdArgs {
  const void* dy;            // [rows, dim] io dtype
  const void* o;             // [rows, dim] io dtype, or e4m3 codes
  const uint8_t* o_scales;   // [rows, dim / 32] when o holds codes, or nullptr
  const void* z;             // as o
  const uint8_t* z_scales;
  const float* w;            // [dim]
  float eps;
  void* d_o;                 // [rows, dim] io dtype
  void* d_z;
  float* dw;                 // [dim]
  int64_t rows;
};

// Arguments of the gradients of the gate (gdn_gate_bwd).
struct GateBwdArgs {
  const void* dg;            // [tokens, nv] io dtype
  const void* dbeta;
  const float* a;            // [tokens, nv]
  const float* b;
  const float* A_log;        // [nv]
  const float* dt_bias;
  void* da;                  // [tokens, nv] io dtype
  void* db;
  float* dA_log;             // [nv]
  float* ddt_bias;
  int64_t tokens;
  int32_t nv;
};

// Arguments of the gradients of the causal conv1d + SiLU (gdn_qkv_conv_bwd).
struct ConvBwdArgs {
  const void* dq;            // [T, nqk, dk] io dtype
  const void* dk_;
  const void* dv_;           // [T, nv, dv]
  const void* x;             // [T, channels] io dtype, or e4m3 codes
  const uint8_t* x_scales;   // [T, channels / 32] when x holds codes, or nullptr
  const float* weight;       // [channels, ksize]
  const float* bias;         // [channels] or nullptr
  const void* state_in;      // [N, channels, ksize] io dtype or nullptr (zeros)
  const void* dstate_out;    // [N, channels, ksize] io dtype or nullptr
  const int32_t* cu;         // [N + 1] or nullptr (equal lengths)
  void* dx;                  // [T, channels] io dtype
  float* dw;                 // [channels, ksize]
  float* db;                 // [channels] or nullptr
  void* dstate_in;           // [N, channels, ksize] io dtype or nullptr
  int32_t uniform_len;       // sequence length when cu == nullptr
  int32_t num_seqs;
  int64_t total_tokens;
  int32_t channels, ksize;   // channels = 2 nqk dk + nv dv
  int32_t nqk, nv, dk, dv;
  unsigned int* status;      // device status word (kStatus* bits)
};

// The bounds of sequence n as seq_bounds clamps them, without a report: for kernels that look bounds up again
// after another kernel of the same call has reported.
template <class Args>
__device__ __forceinline__ void seq_bounds_quiet(const Args& a, int n, int64_t& start, int64_t& end) {
  if (!a.cu) {
    start = (int64_t)n * a.uniform_len;
    end = start + a.uniform_len;
    return;
  }
  const int64_t s = a.cu[n], e = a.cu[n + 1], T = a.total_tokens;
  start = s < 0 ? 0 : (s > T ? T : s);
  end = e < start ? start : (e > T ? T : e);
}

// A call's kernels follow one another closely: each lets the next one be launched as soon as all its blocks have begun
// (let_next_begin), and that one's blocks wait for its end before they do anything (wait_for_previous).  Launched by
// launch_next; only the first kernel of a call is launched as usual, behind everything before it on the stream.
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
static inline cudaError_t launch_next(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

// Instruction descriptor of a tcgen05 MMA of kind::f16 with fp16 A/B and fp32 D (the type fields of the bf16 one are 1).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn_major, bool b_mn_major) {
  return ptx::idesc_bf16_f32(M, N, a_mn_major, b_mn_major) & ~((1u << 7) | (1u << 10));
}

}  // namespace gdn
