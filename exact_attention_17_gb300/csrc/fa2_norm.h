// Internal: the normed rotary kernels' launch (fa2_norm.cu).
#pragma once

#include "fa2_rope.h"

namespace fa2dev {

struct NormParams {
  RopeParams r;            // x, y and the rest of the rotary call, or the append's
  // [d] of the rows' type or fp32 (weight32); of x, or of the append's queries and keys (null: these are not normed)
  const void *weight, *k_weight;
  int weight32;
  float eps;
  // gradient: r.x is x, r.y is dX; dY [B, H, N, d] and the blocks' sums of dweight
  const void* dy;
  long long dy_batch, dy_token, dy_head;
  float* partial;          // [blocks][d]
  long long places;        // token tiles times heads (set by the launch)
};

}  // namespace fa2dev

namespace fa2host {

// Most blocks that the gradient's first kernel has (each leaves d sums).
constexpr int kNormGradBlocksPerSm = 2;

cudaError_t prepare_norm();
// wide: every row start, stride and weight allows 16-byte vectors, and whole vectors hold the rotated columns.
cudaError_t launch_norm_rope(fa2dev::NormParams p, bool append, int dtype, bool wide, int sms, cudaStream_t s);
cudaError_t launch_norm_rope_grad(fa2dev::NormParams p, float* dweight, int dtype, bool wide, int sms, cudaStream_t s);

}  // namespace fa2host
