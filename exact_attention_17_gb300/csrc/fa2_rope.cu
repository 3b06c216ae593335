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
// is the exact angle of the rounded frequency (error below |t| 2^-63 turns).  Its
// top 32 bits give the quadrant and a remainder of at most an eighth turn, whose
// sine and cosine are Taylor polynomials (degree 9 and 10: remainders below
// 2e-9 and 2e-10): about 30 instructions a pair, a third of a library call.
//
// Bound: bytes (each row read and written once); 16 heads of 128 columns at 4 x
// 4096 positions in bf16, 134 MB, take 23 us, 5.8 TB/s (24.5-25.2 us from one call
// to the next), a chunk append of 10,500 tokens (32 + 4 + 4 heads of 64, 32 columns
// rotated) 23.1-24.3 us, one token of 64 sequences 5.5-6.3 us (latency).  A thread keeps one unit of the
// head (two 8-byte vectors of 16-bit elements whose columns are rotated against
// each other, or one 16-byte vector of neighbouring pairs) at one token: it
// computes the unit's four sines once, in registers, and then runs over the
// heads, four at a time.  Nothing goes through shared memory but, for the cache,
// where the block's tokens lie.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa2_host.h"
#include "fa2_launch.h"
#include "fa2_rope.h"

namespace fa2dev {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;   // heads whose loads a thread has in flight

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

// Rotates a unit: vectors a and b against each other (HALF), or a's neighbours.
template <typename T, int W, bool HALF, int PAIRS>
__device__ __forceinline__ void turn(Vec<T, W>& a, Vec<T, W>& b, const float2 (&w)[PAIRS]) {
  if constexpr (!HALF) {
#pragma unroll
    for (int e = 0; e < PAIRS; ++e) {
      const float2 x = widen(&a.v[2 * e]);
      narrow(&a.v[2 * e], x.x * w[e].x - x.y * w[e].y, x.y * w[e].x + x.x * w[e].y);
    }
  } else if constexpr (W % 2 == 0) {
#pragma unroll
    for (int e = 0; e < W; e += 2) {
      const float2 x = widen(&a.v[e]), y = widen(&b.v[e]);
      narrow(&a.v[e], x.x * w[e].x - y.x * w[e].y, x.y * w[e + 1].x - y.y * w[e + 1].y);
      narrow(&b.v[e], y.x * w[e].x + x.x * w[e].y, y.y * w[e + 1].x + x.y * w[e + 1].y);
    }
  } else {
    const float x = widen1(a.v[0]), y = widen1(b.v[0]);
    narrow1(a.v[0], x * w[0].x - y * w[0].y);
    narrow1(b.v[0], y * w[0].x + x * w[0].y);
  }
}

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

// Unit u of a head row is the pair of vectors (u, u + half) when HALF, else the
// vector u; behind the rotated units come the copied ones, two vectors at a
// time (HALF) or one.
template <typename T, int W, bool HALF, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads, 3) fa2_rope_kernel(const __grid_constant__ RopeParams p) {
  using V = Vec<T, W>;
  constexpr int PAIRS = HALF ? W : W / 2;
  constexpr int U = HALF && sizeof(V) == 16 ? kRopeUnroll / 2 : kRopeUnroll;   // (registers)
  __shared__ RopeToken toks[APPEND ? kRopeThreads : 1];
  const long long tok0 = static_cast<long long>(blockIdx.x) * p.tokens;
  const int n_tok = static_cast<int>(min(static_cast<long long>(p.tokens), p.total_tokens - tok0));
  const int row0 = blockIdx.y * p.rows, row1 = min(row0 + p.rows, p.total_rows);
  const int rot_units = p.r / (HALF ? 2 * W : W);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  for (int base = 0; base < n_tok * p.units; base += kRopeThreads) {   // once, but for rows of more than 256 units
    const int id = base + threadIdx.x;
    const bool active = id < n_tok * p.units;
    const int k = active ? fast_div(id, p.div_units) : 0;
    const int u = active ? id - k * p.units : 0;
    const long long t = tok0 + k;
    // columns of the unit's vectors: c and, when `two`, c + second
    const bool rotate = u < rot_units;
    int c = u * W, second = p.r / 2;
    bool two = HALF;
    if (HALF && !rotate) {
      c = p.r + (u - rot_units) * 2 * W;
      second = W;
      two = c + W < p.d;
    }
    double f[PAIRS];
    if (rotate) {
#pragma unroll
      for (int e = 0; e < PAIRS; ++e) f[e] = p.inv_freq[HALF ? c + e : c / 2 + e];
    }
    long long pos, batch = 0, n = t, slot = -1;
    bool live = active;
    if constexpr (APPEND) {
      if (base == 0) {
        append_tokens(p, static_cast<int>(tok0), n_tok, toks);
        __syncthreads();
      }
      pos = toks[k].pos;
      slot = toks[k].dst;
      live = active && toks[k].live;
    } else {
      if (p.N < p.total_tokens) {
        batch = t < 0x7fffffff ? static_cast<long long>(fast_div(static_cast<int>(t), p.div_n)) : t / p.N;
        n = t - batch * p.N;
      }
      const long long at = batch * p.pos_batch + n;
      pos = p.pos64 ? static_cast<const long long*>(p.positions)[at] : static_cast<const int*>(p.positions)[at];
    }
    if (!live) continue;   // (no barrier follows but in rows of more than 256 units, which are of one token)
    float2 w[PAIRS];
    // the queries' heads, the keys' and the values' of a new token, or all heads of one array
#pragma unroll 1
    for (int part = 0; part < (APPEND ? 3 : 1); ++part) {
      const T* x;
      T* y;
      long long xs, ys;
      int from = row0, to = row1;
      if constexpr (APPEND) {
        const int first = part == 0 ? 0 : p.Hq + (part - 1) * p.Hkv;
        from = max(row0, first) - first;
        to = min(row1, first + (part == 0 ? p.Hq : p.Hkv)) - first;
        if (part > 0 && slot < 0) to = from;
        xs = part == 0 ? p.q_head : part == 1 ? p.k_head : p.v_head;
        ys = part == 0 ? p.qo_head : p.page_head;
        x = static_cast<const T*>(part == 0 ? p.q : part == 1 ? p.k : p.v) +
            t * (part == 0 ? p.q_token : part == 1 ? p.k_token : p.v_token);
        y = static_cast<T*>(part == 0 ? p.q_out : part == 1 ? p.k_pages : p.v_pages) +
            (part == 0 ? t * p.qo_token : slot);
      } else {
        xs = p.x_head;
        ys = p.y_head;
        x = static_cast<const T*>(p.x) + batch * p.x_batch + n * p.x_token;
        y = static_cast<T*>(p.y) + batch * p.y_batch + n * p.y_token;
      }
      int left = to - from;
      if (left <= 0) continue;
      x += from * xs + c;
      y += from * ys + c;
      const bool turns = rotate && part < 2;
      // U heads on their way while the U before them are rotated and stored
      V a[U], b[U], a2[U], b2[U];
      auto load = [&](V (&va)[U], V (&vb)[U], int count) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          if (i < count) {
            va[i] = *reinterpret_cast<const V*>(x);
            if (HALF && two) vb[i] = *reinterpret_cast<const V*>(x + second);
          }
          x += xs;
        }
      };
      load(a, b, left);
      if (part == 0 || (part == 1 && row0 >= p.Hq)) {   // the first part that turns
        if (rotate) {
#pragma unroll
          for (int e = 0; e < PAIRS; ++e) w[e] = rotation(f[e], pos, p.mscale, p.transposed != 0);
        }
      }
      for (;;) {
        if (left > U) load(a2, b2, left - U);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          if (i < left) {
            if (turns) turn<T, W, HALF>(a[i], b[i], w);
            *reinterpret_cast<V*>(y) = a[i];
            if (HALF && two) *reinterpret_cast<V*>(y + second) = b[i];
          }
          y += ys;
        }
        left -= U;
        if (left <= 0) break;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          a[i] = a2[i];
          if (HALF) b[i] = b2[i];
        }
      }
    }
  }
}

}  // namespace fa2dev

namespace fa2host {
namespace {

using fa2dev::RopeParams;

template <typename T, int W, bool HALF, bool APPEND>
cudaError_t run(const RopeParams& p, dim3 grid, cudaStream_t s) {
  return launch_behind(fa2dev::fa2_rope_kernel<T, W, HALF, APPEND>, grid, fa2dev::kRopeThreads, 0, s, p);
}

template <typename T, bool APPEND>
cudaError_t by_layout(const RopeParams& p, dim3 grid, bool wide, cudaStream_t s) {
  if (p.interleaved)   // a pair is two neighbours at least
    return wide ? run<T, rope_width(sizeof(T), true), false, APPEND>(p, grid, s) : run<T, 2, false, APPEND>(p, grid, s);
  return wide ? run<T, rope_width(sizeof(T), false), true, APPEND>(p, grid, s) : run<T, 1, true, APPEND>(p, grid, s);
}

template <bool APPEND>
cudaError_t by_type(const RopeParams& p, int dtype, dim3 grid, bool wide, cudaStream_t s) {
  if (dtype == FA2_DTYPE_BF16) return by_layout<__nv_bfloat16, APPEND>(p, grid, wide, s);
  if (dtype == FA2_DTYPE_FP16) return by_layout<__half, APPEND>(p, grid, wide, s);
  if constexpr (!APPEND) return by_layout<float, APPEND>(p, grid, wide, s);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope(RopeParams p, bool append, int dtype, bool wide, int sms, cudaStream_t s) {
  const int size = dtype == FA2_DTYPE_FP32 ? 4 : 2;
  const int w = wide ? rope_width(size, p.interleaved) : (p.interleaved ? 2 : 1);
  const int pair = p.interleaved ? 1 : 2;
  p.units = p.r / (w * pair) + ((p.d - p.r) / w + pair - 1) / pair;
  p.tokens = fa2dev::kRopeThreads / p.units;
  if (p.tokens < 1) p.tokens = 1;
  const long long tiles = (p.total_tokens + p.tokens - 1) / p.tokens;
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  // Heads of a block: all of them, so that the sines are computed once, unless
  // that leaves fewer than two blocks an SM; then as few as it takes, at least one
  // unrolled step.  (10460 tokens of 40 rows in 327 blocks: 24.6 us; two, four and
  // eight times the blocks: 27.4, 30.7 and 45.1.)
  long long chunks = (2ll * sms + tiles - 1) / tiles;
  const long long most = (p.total_rows + fa2dev::kRopeUnroll - 1) / fa2dev::kRopeUnroll;
  if (chunks > most) chunks = most;
  if (chunks > 65535) chunks = 65535;
  p.rows = static_cast<int>((p.total_rows + chunks - 1) / chunks);
  chunks = (p.total_rows + p.rows - 1) / p.rows;
  p.div_units = make_fast_div(p.units);
  p.div_n = make_fast_div(static_cast<int>(p.N > 0 ? p.N : 1));
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(chunks));
  return append ? by_type<true>(p, dtype, grid, wide, s) : by_type<false>(p, dtype, grid, wide, s);
}

}  // namespace fa2host
