// Rotary positions, alone (fa2_rope) and on the way into a paged key/value
// cache (fa2_append_paged).
//
// For pair i of the first r columns of a head row at position t:
//   (a, b) -> m (a cos(t f_i) - b sin(t f_i),  b cos(t f_i) + a sin(t f_i))
// with f_i radians per position (64-bit, given by the caller: long-context
// scaling lives there), m a magnitude factor and the pair either columns
// (i, i + r/2) or (2i, 2i + 1).  The gradient is the transposed rotation: the
// same with -sin.  Columns r..d-1 are copied.
//
// Angles.  t f in 32 bits is off by whole turns at far positions, and 64-bit
// floating point is slow here.  f / (2 pi) is turned into a 64-bit fixed-point
// fraction of a turn with one 64 x 64-bit multiplication; times t modulo 2^64 it
// is the exact angle of the rounded frequency (error below |t| 2^-63 turns), and
// its top 32 bits, rounded to fp32, go to sincospif: the angle is within 2^-25
// turns for every 32-bit position.
//
// Bound: bytes (each row read and written once).  A block takes `tokens` x
// `rows` head rows; each thread first loads its vectors (up to four pairs of 16
// bytes), then the block computes the sines of its tokens once for all heads in
// shared memory, then rotates and stores: the arithmetic overlaps the loads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa2_host.h"
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
  const int top = static_cast<int>(static_cast<long long>(t) >> 32);   // turns * 2^32, in [-1/2, 1/2)
  float s, c;
  sincospif(static_cast<float>(top) * 0x1p-31f, &s, &c);
  return make_float2(c * m, transposed ? -s * m : s * m);
}

template <typename T> __device__ __forceinline__ float to_float(T x);
template <> __device__ __forceinline__ float to_float(float x) { return x; }
template <> __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }

// W elements moved at once (16 bytes, or one element)
template <typename T, int W>
struct alignas(sizeof(T) * W) Vec {
  T v[W];
};

// Where a block's tokens go.
struct RopeToken {
  long long src;     // element offset of the token in x (or its index in the packed tensors)
  long long dst;     // the same in the output (append: offset of its slot in the pages, -1: not written)
  long long pos;
  int live;          // 0: nothing is written for this token
};

// A block's rows: `tokens` consecutive tokens times `rows` consecutive head
// rows.  Work is numbered (token, row, unit); unit u of a row is the pair of
// vectors (u, u + half) when HALF, else the vector u.  Rows of W elements:
// the rotated vectors first, then the copied ones two at a time (HALF) or one.
template <typename T, int W, bool HALF, bool APPEND, int ITEMS>
__global__ void __launch_bounds__(kRopeThreads) fa2_rope_kernel(const RopeParams p) {
  extern __shared__ float2 cs[];   // [tokens][r / 2]
  __shared__ RopeToken toks[kRopeMaxTokens];
  using V = Vec<T, W>;
  const int tile = fast_div(static_cast<int>(blockIdx.x), p.div_row_tiles);
  const int row0 = (static_cast<int>(blockIdx.x) - tile * p.row_tiles) * p.rows;
  const long long tok0 = static_cast<long long>(tile) * p.tokens;
  const int n_tok = static_cast<int>(min(static_cast<long long>(p.tokens), p.total_tokens - tok0));
  const int n_row = min(p.rows, p.total_rows - row0);
  const int half = p.r / 2;

  // ---- the block's tokens
  if constexpr (APPEND) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int k = warp; k < n_tok; k += kRopeThreads / 32) {
      const int t = static_cast<int>(tok0) + k;
      int b = t, begin = t, end = t + 1;
      if (p.cu_q != nullptr) {
        int c = 0;   // sequences that end at or before t
        for (int i = lane + 1; i <= p.B; i += 32) c += p.cu_q[i] <= t ? 1 : 0;
        b = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(c)));
        begin = b < p.B ? p.cu_q[b] : 0;
        end = b < p.B ? p.cu_q[b + 1] : 0;
      }
      if (lane == 0) {
        RopeToken& o = toks[k];
        o.src = t;
        o.dst = -1;
        o.live = b < p.B && begin <= t && t < end;
        o.pos = 0;
        if (o.live) {
          const int len = p.kv_lens[b];
          const long long pos = static_cast<long long>(len) - end + t;
          o.pos = pos;
          if (len > p.max_len) {
            atomicOr(p.status, kDevErrPage);
          } else if (pos >= 0) {
            const int page = p.page_table[b * p.table_stride + (pos >> p.page_log2)];
            if (page < 0 || page >= p.num_pages)
              atomicOr(p.status, kDevErrPage);
            else
              o.dst = page * p.page_stride + (pos & ((1 << p.page_log2) - 1)) * p.slot_stride;
          }
        }
      }
    }
  } else {
    for (int k = threadIdx.x; k < n_tok; k += kRopeThreads) {
      const long long t = tok0 + k;
      const long long b = t / p.N, n = t - b * p.N;
      RopeToken& o = toks[k];
      o.src = b * p.x_batch + n * p.x_token;
      o.dst = b * p.y_batch + n * p.y_token;
      const long long at = b * p.pos_batch + n;
      o.pos = p.pos64 ? static_cast<const long long*>(p.positions)[at] : static_cast<const int*>(p.positions)[at];
      o.live = 1;
    }
  }
  __syncthreads();

  // ---- loads
  constexpr int PAIR = HALF ? 2 : 1;                 // vectors per unit
  const int rot_units = p.r / (W * PAIR);            // units that rotate
  const int units = p.units;
  const int total = n_tok * n_row * units;
  V a[ITEMS], b2[ITEMS];
  T* to[ITEMS];
  T* to2[ITEMS];
  int how[ITEMS];   // index of the token's first sine of this unit, or -1: copy, -2: nothing
  for (int base = 0; base < total; base += kRopeThreads * ITEMS) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int item = base + i * kRopeThreads + threadIdx.x;
      how[i] = -2;
      to[i] = to2[i] = nullptr;
      if (item >= total) continue;
      const int rr = fast_div(item, p.div_units);
      const int u = item - rr * units;
      const int k = n_row == p.rows ? fast_div(rr, p.div_rows) : rr / n_row;
      int row = row0 + (rr - k * n_row);
      const RopeToken tk = toks[k];
      if (!tk.live) continue;
      const T* x;
      T* y;
      bool rotate = u < rot_units;
      if constexpr (APPEND) {
        if (row < p.Hq) {
          x = static_cast<const T*>(p.q) + tk.src * p.q_token + row * p.q_head;
          y = static_cast<T*>(p.q_out) + tk.src * p.qo_token + row * p.qo_head;
        } else {
          if (tk.dst < 0) continue;
          row -= p.Hq;
          const bool value = row >= p.Hkv;
          if (value) row -= p.Hkv;
          x = value ? static_cast<const T*>(p.v) + tk.src * p.v_token + row * p.v_head
                    : static_cast<const T*>(p.k) + tk.src * p.k_token + row * p.k_head;
          y = static_cast<T*>(value ? p.v_pages : p.k_pages) + tk.dst + row * p.page_head;
          if (value) rotate = false;
        }
      } else {
        x = static_cast<const T*>(p.x) + tk.src + row * p.x_head;
        y = static_cast<T*>(p.y) + tk.dst + row * p.y_head;
      }
      // columns of the unit's vectors: (c, c2), c2 < 0: one vector
      int c, c2 = -1;
      if constexpr (HALF) {
        if (u < rot_units) {
          c = u * W;
          c2 = c + half;
        } else {
          c = p.r + (u - rot_units) * 2 * W;
          c2 = c + W < p.d ? c + W : -1;
        }
      } else {
        c = u * W;
      }
      a[i] = *reinterpret_cast<const V*>(x + c);
      to[i] = y + c;
      if (HALF && c2 >= 0) {
        b2[i] = *reinterpret_cast<const V*>(x + c2);
        to2[i] = y + c2;
      }
      how[i] = rotate ? k * half + (HALF ? u * W : u * W / 2) : -1;
    }
    // ---- sines, once per block, while the first loads are in flight
    if (base == 0 && half > 0) {
      for (int e = threadIdx.x; e < n_tok * half; e += kRopeThreads) {
        const int k = fast_div(e, p.div_half);
        cs[e] = rotation(p.inv_freq[e - k * half], toks[k].pos, p.mscale, p.transposed != 0);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (how[i] >= 0) {
        const float2* t = cs + how[i];
        if constexpr (HALF) {
#pragma unroll
          for (int e = 0; e < W; ++e) {
            const float x0 = to_float(a[i].v[e]), x1 = to_float(b2[i].v[e]);
            const float2 w = t[e];
            a[i].v[e] = from_float<T>(x0 * w.x - x1 * w.y);
            b2[i].v[e] = from_float<T>(x1 * w.x + x0 * w.y);
          }
        } else {
#pragma unroll
          for (int e = 0; e < W; e += 2) {
            const float x0 = to_float(a[i].v[e]), x1 = to_float(a[i].v[e + 1]);
            const float2 w = t[e / 2];
            a[i].v[e] = from_float<T>(x0 * w.x - x1 * w.y);
            a[i].v[e + 1] = from_float<T>(x1 * w.x + x0 * w.y);
          }
        }
      }
      if (to[i] != nullptr) *reinterpret_cast<V*>(to[i]) = a[i];
      if (HALF && to2[i] != nullptr) *reinterpret_cast<V*>(to2[i]) = b2[i];
    }
  }
}

}  // namespace fa2dev

namespace fa2host {
namespace {

using fa2dev::RopeParams;

template <typename T, int W, bool HALF, bool APPEND, int ITEMS>
cudaError_t run(const RopeParams& p, unsigned grid, size_t smem, cudaStream_t s) {
  fa2dev::fa2_rope_kernel<T, W, HALF, APPEND, ITEMS><<<grid, fa2dev::kRopeThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int W, bool APPEND>
cudaError_t by_layout(const RopeParams& p, unsigned grid, size_t smem, int items, cudaStream_t s) {
  constexpr int WI = W > 1 ? W : 2;   // an interleaved pair is two neighbours at least
  if (p.interleaved)
    return items == 1 ? run<T, WI, false, APPEND, 1>(p, grid, smem, s) : run<T, WI, false, APPEND, 4>(p, grid, smem, s);
  return items == 1 ? run<T, W, true, APPEND, 1>(p, grid, smem, s) : run<T, W, true, APPEND, 4>(p, grid, smem, s);
}

template <typename T, bool APPEND>
cudaError_t by_width(const RopeParams& p, unsigned grid, size_t smem, int items, bool wide, cudaStream_t s) {
  return wide ? by_layout<T, 16 / sizeof(T), APPEND>(p, grid, smem, items, s)
              : by_layout<T, 1, APPEND>(p, grid, smem, items, s);
}

template <bool APPEND>
cudaError_t by_type(const RopeParams& p, int dtype, unsigned grid, size_t smem, int items, bool wide, cudaStream_t s) {
  if (dtype == FA2_DTYPE_BF16) return by_width<__nv_bfloat16, APPEND>(p, grid, smem, items, wide, s);
  if (dtype == FA2_DTYPE_FP16) return by_width<__half, APPEND>(p, grid, smem, items, wide, s);
  if constexpr (!APPEND) return by_width<float, APPEND>(p, grid, smem, items, wide, s);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope(RopeParams p, bool append, int dtype, bool wide, int sms, cudaStream_t s) {
  const int size = dtype == FA2_DTYPE_FP32 ? 4 : 2;
  const int w = wide ? 16 / size : (p.interleaved ? 2 : 1);
  const int pair = p.interleaved ? 1 : 2;
  const int rot_units = p.r / (w * pair);
  p.units = rot_units + ((p.d - p.r) / w + pair - 1) / pair;
  // Head rows of a block: four units a thread (the loads of one thread in
  // flight together) when that leaves four blocks an SM, else one.
  const long long all = p.total_tokens * p.total_rows * p.units;
  int items = 4;
  if (all < 4ll * sms * 4 * fa2dev::kRopeThreads) items = 1;
  int rows_per_block = items * fa2dev::kRopeThreads / p.units;
  if (rows_per_block < 1) rows_per_block = 1;
  p.rows = p.total_rows < 8 ? p.total_rows : 8;
  if (items == 1 && p.rows > rows_per_block) p.rows = rows_per_block;
  p.tokens = rows_per_block / p.rows;
  if (p.tokens < 1) p.tokens = 1;
  if (p.tokens > fa2dev::kRopeMaxTokens) p.tokens = fa2dev::kRopeMaxTokens;
  // the sines of a block stay within the default 48 KB of shared memory
  const int half = p.r / 2;
  while (p.tokens > 1 && static_cast<size_t>(p.tokens) * half * sizeof(float2) > (32u << 10)) p.tokens /= 2;
  p.row_tiles = (p.total_rows + p.rows - 1) / p.rows;
  const long long blocks = (p.total_tokens + p.tokens - 1) / p.tokens * p.row_tiles;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  p.div_row_tiles = make_fast_div(p.row_tiles);
  p.div_rows = make_fast_div(p.rows);
  p.div_units = make_fast_div(p.units);
  p.div_half = make_fast_div(half > 0 ? half : 1);
  const size_t smem = static_cast<size_t>(p.tokens) * half * sizeof(float2);
  return append ? by_type<true>(p, dtype, static_cast<unsigned>(blocks), smem, items, wide, s)
                : by_type<false>(p, dtype, static_cast<unsigned>(blocks), smem, items, wide, s);
}

}  // namespace fa2host
