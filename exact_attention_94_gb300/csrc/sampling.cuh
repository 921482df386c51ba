// What the kernels of a sampling step (norms of query and key heads with their
// rotation, attention of requests that share a prefix) take, beyond serving.cuh.
#pragma once

#include "serving.cuh"

namespace fa {

// Norms of heads with the rotation (see fa_qk_norm_rope in fa.h).
struct NormRopeParams {
  const void* q;             // inputs of the forward
  const void* k;
  const void* dyq;           // gradients of its outputs (backward)
  const void* dyk;
  void* q_out;               // outputs, or the gradients of the inputs
  void* k_out;
  const void* wq;            // [d] bf16, or fp32 with w_fp32
  const void* wk;
  const int* positions;      // [n_axes, T]
  float* dw_part;            // backward: [blocks, d] sums of each block, q's blocks first
  long long q_stride, k_stride, dyq_stride, dyk_stride, q_out_stride, k_out_stride;  // elements between rows
  int T, Hq, Hkv;
  int w_fp32;
  float eps;
  int heads_per_thread;      // set by the launch
  int q_chunks, k_chunks;    //   thread chunks of a token's query and of its key heads
  int q_blocks;              //   blocks that work on query heads (backward)
  signed char axis[64];      // axis of pair p, -1: not rotated
  uint64_t turn[64];         // its frequency: fraction of a turn per position, in 2^-64
};
cudaError_t launch_norm_rope(NormRopeParams& p, int D, bool neighbours, cudaStream_t stream);
int norm_rope_bwd_blocks(int T, int Hq, int Hkv, int D, int* q_blocks);  // blocks of the backward, those of q's heads
cudaError_t launch_norm_rope_bwd(NormRopeParams& p, int D, bool neighbours, float* dwq, float* dwk, cudaStream_t stream);

}  // namespace fa
