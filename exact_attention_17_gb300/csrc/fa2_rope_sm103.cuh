// Device code that the rotary kernels (fa2_rope.cu) and the normed ones
// (fa2_norm.cu) share: angles, vectors of elements, where a cache's new tokens go.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa2_rope.h"

namespace fa2dev {

constexpr int kRopeThreads = 256;

// 2^64 times the fraction of a turn that f radians are, modulo 2^64.
// |f| = mant 2^(e-1075); kTurn = 2^66 / (2 pi) rounded, so |f| / (2 pi) 2^64 =
// mant kTurn 2^(e-1077).
__device__ __forceinline__ unsigned long long turns_of(double f) {
  constexpr unsigned long long kTurn = 11743562013128004906ull;
  const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(f));
  const int e = static_cast<int>((bits >> 52) & 0x7ff);
  if (e == 0) return 0;   // zero or below 2^-1022
  const unsigned long long mant = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
  const unsigned long long hi = __umul64hi(mant, kTurn), lo = mant * kTurn;
  const int s = 1077 - e;   // right shift of hi:lo
  unsigned long long t;
  if (s >= 128) t = 0;
  else if (s >= 64) t = hi >> (s - 64);
  else if (s > 0) t = (lo >> s) | (hi << (64 - s));
  else t = s > -64 ? lo << -s : 0;
  return (bits >> 63) ? 0ull - t : t;
}

// (cos, sin) times m of `pos` steps of f radians
__device__ __forceinline__ float2 rotation(double f, long long pos, float m, bool transposed) {
  const unsigned long long t = turns_of(f) * static_cast<unsigned long long>(pos);
  const uint32_t top = static_cast<uint32_t>(t >> 32);   // turns * 2^32
  const uint32_t quadrant = (top + 0x20000000u) >> 30;
  const float y = static_cast<float>(static_cast<int>(top - (quadrant << 30))) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  const float z = y * y;
  float s = 2.7557319e-6f, c = -2.7557319e-7f;   // 1 / 9!, -1 / 10!
  s = fmaf(s, z, -1.9841270e-4f);                // 1 / 7!
  s = fmaf(s, z, 8.3333333e-3f);
  s = fmaf(s, z, -1.6666667e-1f);
  s = fmaf(s * z, y, y);
  c = fmaf(c, z, 2.4801587e-5f);                 // 1 / 8!
  c = fmaf(c, z, -1.3888889e-3f);
  c = fmaf(c, z, 4.1666667e-2f);
  c = fmaf(c, z, -0.5f);
  c = fmaf(c, z, 1.0f);
  const float a = (quadrant & 1) ? s : c, b = (quadrant & 1) ? c : s;
  const float mc = (quadrant == 1 || quadrant == 2) ? -m : m;
  const float ms = ((quadrant >= 2) != transposed) ? -m : m;
  return make_float2(a * mc, b * ms);
}

// W elements moved at once.
template <typename T, int W>
struct alignas(sizeof(T) * W) Vec {
  T v[W];
};

// Two neighbouring elements as fp32, and back (rounded to nearest even).
__device__ __forceinline__ float2 widen(const float* v) { return make_float2(v[0], v[1]); }
__device__ __forceinline__ float2 widen(const __nv_bfloat16* v) {
  const uint32_t x = *reinterpret_cast<const uint32_t*>(v);
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
__device__ __forceinline__ float2 widen(const __half* v) { return __half22float2(*reinterpret_cast<const __half2*>(v)); }
__device__ __forceinline__ void narrow(float* v, float x, float y) {
  v[0] = x;
  v[1] = y;
}
__device__ __forceinline__ void narrow(__nv_bfloat16* v, float x, float y) {
  *reinterpret_cast<uint32_t*>(v) = pack_bf16x2(x, y);
}
__device__ __forceinline__ void narrow(__half* v, float x, float y) { *reinterpret_cast<uint32_t*>(v) = pack_f16x2(x, y); }
__device__ __forceinline__ float widen1(float x) { return x; }
__device__ __forceinline__ float widen1(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen1(__half x) { return __half2float(x); }
__device__ __forceinline__ void narrow1(float& v, float x) { v = x; }
__device__ __forceinline__ void narrow1(__nv_bfloat16& v, float x) { v = __float2bfloat16_rn(x); }
__device__ __forceinline__ void narrow1(__half& v, float x) { v = __float2half_rn(x); }

// Where a new token of a cache goes.
struct RopeToken {
  long long dst;     // element offset of its slot in the pages, -1: not written
  long long pos;
  int live;          // 0: nothing is written for this token
};

// A sequence's length and the rows of its new tokens lie within the table and the call's tokens.
__device__ __forceinline__ bool append_in_order(const RopeParams& p, int begin, int end, int len) {
  return (begin >= 0) & (begin <= end) & (end <= p.total_tokens) & (len >= 0) & (len <= p.max_len);
}

// Whole block: positions and slots of `n_tok` tokens from tok0 on, a warp per
// token.  Where a sequence's numbers are not in order, its tokens are not
// written: a slot taken from them could be an older token's.  (Their queries turn
// at the positions that attention gives them, from the numbers cut to their range.)
// Sequences without a token in the call are looked at and reported too, by the
// first block's first warp, which reads all offsets for its token anyway.
__device__ __forceinline__ void append_tokens(const RopeParams& p, int tok0, int n_tok, RopeToken* toks) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int k = warp; k < n_tok; k += kRopeThreads / 32) {
    const int t = tok0 + k;
    int b = t, begin = t, end = t + 1;
    if (p.cu_q != nullptr) {
      const bool all = blockIdx.x == 0 && blockIdx.y == 0 && k == 0;
      bool good = true;
      int c = 0;   // sequences that end at or before t
      for (int i = lane + 1; i <= p.B; i += 32) {
        const int e = p.cu_q[i], a = all ? p.cu_q[i - 1] : e, n = all ? p.kv_lens[i - 1] : 0;   // (loads side by side)
        c += e <= t ? 1 : 0;
        good &= !all | append_in_order(p, a, e, n);
      }
      if (!good) atomicOr(p.status, kDevErrPage);
      b = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(c)));
      begin = b < p.B ? p.cu_q[b] : 0;
      end = b < p.B ? p.cu_q[b + 1] : 0;
    }
    if (lane == 0) {
      RopeToken o;
      o.dst = -1;
      o.pos = 0;
      o.live = b < p.B && begin <= t && t < end;
      if (o.live) {
        const int len = p.kv_lens[b];
        const long long pos = min(max(len, 0), p.max_len) - min(static_cast<long long>(end), p.total_tokens) + t;
        o.pos = pos;
        if (!append_in_order(p, begin, end, len)) {
          atomicOr(p.status, kDevErrPage);
        } else if (pos >= 0) {
          const int page = p.page_table[b * p.table_stride + (pos >> p.page_log2)];
          if (page < 0 || page >= p.num_pages)
            atomicOr(p.status, kDevErrPage);
          else
            o.dst = page * p.page_stride + (pos & ((1 << p.page_log2) - 1)) * p.slot_stride;
        }
      }
      toks[k] = o;
    }
  }
}

}  // namespace fa2dev
