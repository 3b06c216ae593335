// Internal: the rotary and append kernels' launch (fa2_rope.cu).
#pragma once

#include <cuda_runtime.h>

#include "fa2.h"
#include "fa2_paged_sm103.cuh"

namespace fa2dev {

struct RopeParams {
  // rotary alone: x and y [B, H, N, d] with element strides
  const void* x;
  void* y;
  const void* positions;   // int32 or int64 (pos64), [N] or [B, N] (pos_batch = N)
  int pos64;
  long long pos_batch;
  long long N;
  long long x_batch, x_token, x_head, y_batch, y_token, y_head;
  // append: packed q [T, Hq, d], k and v [T, Hkv, d]; pages [P, Hkv, S, d]
  const void *q, *k, *v;
  void *q_out, *k_pages, *v_pages;
  long long q_token, q_head, qo_token, qo_head, k_token, k_head, v_token, v_head;
  long long page_stride, page_head, slot_stride;
  const int* page_table;
  const int* kv_lens;
  const int* cu_q;         // [B + 1], or null: one token per sequence
  long long table_stride;
  int B, Hq, Hkv, page_log2, num_pages, max_len;
  int* status;
  // both
  const double* inv_freq;  // [r / 2] radians per position
  int d, r, interleaved, transposed;
  float mscale;
  long long total_tokens;
  int total_rows;          // head rows of a token
  // set by the launch
  int tokens, rows;        // of a block
  int units;               // of a head row
  FastDiv div_units, div_n;
};

}  // namespace fa2dev

namespace fa2host {

// Elements of a vector: four pairs to a unit (interleaved 16-bit: 16 bytes; in
// halves 8 bytes twice; fp32: two pairs in 16 bytes, or four in 16 bytes twice).
constexpr int rope_width(int elem_bytes, bool interleaved) { return interleaved && elem_bytes == 2 ? 8 : 4; }

// dtype: FA2_DTYPE_*; wide: every row start and stride allows vectors of
// rope_width elements, and the rotated columns (their half, unless
// interleaved) fill them.
cudaError_t launch_rope(fa2dev::RopeParams p, bool append, int dtype, bool wide, int sms, cudaStream_t s);

}  // namespace fa2host
