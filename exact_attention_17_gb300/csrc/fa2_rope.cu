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
#include "fa2_host.h"
#include "fa2_launch.h"
#include "fa2_rope_sm103.cuh"

namespace fa2dev {

constexpr int kRopeUnroll = 4;   // heads whose loads a thread has in flight

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
