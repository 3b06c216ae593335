// Internal: host helpers shared by the entry-point units (defined in fa2_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>

#include "fa2_fwd_sm103.cuh"

namespace fa2host {

int require_device();                                  // fa2_status of the current device
int device_sms();                                      // after require_device succeeded
bool device_memory_ok(const void* p, size_t bytes);    // [p, p + bytes) is device memory of one allocation
int* device_status_word();                             // nullptr on failure
unsigned long long wait_timeout_ns();
// Tensor map of 16-bit elements, 128-byte swizzle (box[0] = 64 elements);
// strides in bytes of dimensions 1 .. rank-1.
bool encode_tiled(CUtensorMap* map, bool f16, int rank, const void* base, const unsigned long long* dims,
                  const unsigned long long* strides, const unsigned* box);
fa2dev::FastDiv make_fast_div(int d);
// Maps of dense [Z][N][d] arrays, 128-byte swizzle: 16-bit (64 columns x 128 rows), fp32 dQ (32 x 128), the forward's
// output (elem_bytes 2 or 4).
bool encode_heads(CUtensorMap* map, const void* base, int d, int N, int Z, bool f16);
bool encode_heads_f32(CUtensorMap* map, const void* base, int d, int N, int Z);
bool encode_heads_out(CUtensorMap* map, const void* base, int d, int N, long long Z, int elem_bytes, bool f16);

}  // namespace fa2host
