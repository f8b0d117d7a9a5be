// gdn_launch.h -- launchers of the libgdn.so kernels (host side, internal).
#pragma once

#include <cuda_runtime.h>

#include "train_common.cuh"

namespace gdn {

// fp32 CUDA-core chunked forward; dk in {64,128}, chunk in {64,128}, dv % 32 == 0.
cudaError_t launch_chunk_simt(const ChunkArgs& a, int dk, int chunk, int io_bf16, cudaStream_t s);

// Tensor-core chunked forward (tcgen05 + TMA): bf16 io, Dk = Dv = 128, chunk 64.
bool chunk_tc_supported(int dk, int dv, int chunk, int io_bf16);
cudaError_t launch_chunk_tc(const ChunkArgs& a, int64_t total_tokens, cudaStream_t s);
// One CTA whose bounded wait on a barrier nothing arrives on expires after
// limit_ns and records kStatusTimeout in *status.
cudaError_t launch_selftest_wait(uint64_t limit_ns, unsigned int* status, cudaStream_t s);

// One-token decode step; dk, dv in {64,128}.
cudaError_t launch_recurrent_step(const StepArgs& a, int dk, int dv, int io_bf16, cudaStream_t s);

// Gated RMSNorm rows: y = o / sqrt(mean(o^2) + eps) * w * silu(z); dim in {64,128}; y may be o.
cudaError_t launch_gated_rmsnorm(const void* o, const void* z, const float* w, float eps, void* y,
                                 int64_t rows, int dim, int io_bf16, cudaStream_t s);

// Causal depthwise conv1d + SiLU of q|k|v: prefill (with the final conv_state
// when state_out is set) and the one-token decode update; ksize in [1, 4].
cudaError_t launch_conv_fwd(const ConvArgs& a, int io_bf16, cudaStream_t s);
cudaError_t launch_conv_update(const ConvArgs& a, int io_bf16, cudaStream_t s);

// Gradients of the chunked forward; dk, dv in {64,128}.  Workspace bytes and launch.
int64_t chunk_bwd_workspace(int64_t total_tokens, int num_seqs, int nqk, int nv, int dk, int dv);
cudaError_t launch_chunk_bwd(const BwdArgs& a, int dk, int dv, int io_bf16, cudaStream_t s);
// The same for bf16 io with normalised q, k, and fp16 operands.
int64_t chunk_bwd_half_workspace(int64_t total_tokens, int num_seqs, int nqk, int nv, int dk, int dv);
cudaError_t launch_chunk_bwd_half(const BwdArgs& a, int dk, int dv, cudaStream_t s);

// Activations in 8 bits: n values (a multiple of 32), codes [n], scale bytes [n / 32].
cudaError_t launch_act_quantize(const void* x, uint8_t* codes, uint8_t* scales, int64_t n, int io_bf16, cudaStream_t s);
cudaError_t launch_act_dequantize(const uint8_t* codes, const uint8_t* scales, void* y, int64_t n, int io_bf16, cudaStream_t s);

// Gradients of the gated RMSNorm, of the conv and of the gate; `part`: workspace of the bytes that go before.
int64_t gated_rmsnorm_bwd_workspace(int64_t rows, int dim, int io_bf16);
cudaError_t launch_gated_rmsnorm_bwd(const NormBwdArgs& p, int dim, int io_bf16, float* part, cudaStream_t s);
int64_t conv_bwd_workspace(int64_t tokens, int channels, int ksize, int io_bf16);
cudaError_t launch_conv_bwd(const ConvBwdArgs& a, int io_bf16, float* part, cudaStream_t s);
int64_t gate_bwd_workspace(int64_t tokens, int nv);
cudaError_t launch_gate_bwd(const GateBwdArgs& p, int io_bf16, float* part, cudaStream_t s);

}  // namespace gdn
