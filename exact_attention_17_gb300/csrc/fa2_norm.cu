// Each head's row normed and rotated in one pass (fa2_norm_rope), on the way into
// a paged key/value cache too (fa2_append_paged_norm), and the gradients.
//
// A row x of d columns with weight w, at position t:
//   r = 1 / sqrt(sum_c x_c^2 / d + eps),   y = R(t) (w x r)
// R(t) being the rotation of fa2_rope.cu.  With g = R(t)^T dy, h = w g:
//   dw = sum over the rows of g x r
//   dx = r (h - x r (sum_c h_c x_c r) / d)
// r is computed again from x, which is read anyway; no statistics are kept.
//
// Bound: bytes, each row read and written once (x and dy read, dx written).  A
// row belongs to neighbouring lanes of one warp, so that its sums are a few
// shuffles; a lane holds pairs of vectors whose columns are rotated against each
// other, computes the sines (and, forward, their products with the weights) of its
// columns once for a token and then runs over the token's heads.  Sums are fp32.
// The gradient's blocks keep their columns' sums over all the rows they see in
// registers, add up their lanes in shared memory, and leave d numbers each; a
// second kernel adds those up in one order, so that the result does not depend on
// timing.
#include "fa2_host.h"
#include "fa2_launch.h"
#include "fa2_norm.h"
#include "fa2_rope_sm103.cuh"

namespace fa2dev {

// Which columns a lane holds: NV pairs of vectors of W elements.
template <typename T, int D, int W, bool HALF>
struct NormShape {
  static constexpr int kUnits = D / (2 * W);                // pairs of vectors in a row
  static constexpr int kLanes = kUnits < 32 ? kUnits : 32;  // lanes of a row
  static constexpr int NV = kUnits / kLanes;
  static constexpr int E = 2 * W * NV;                      // elements of a lane
  static constexpr int PAIRS = W * NV;
  static constexpr bool kAcross = HALF || W == 1;           // a pair lies in both vectors (else in neighbours of one)
  using V = Vec<T, W>;

  // column of vector `half` (0, 1) of the lane's pair v; r rotated columns
  static __device__ __forceinline__ int column(int lane, int v, int half, int r) {
    const int u = lane + v * kLanes;
    if (HALF) {
      const int turned = r / (2 * W);
      return u < turned ? u * W + half * (r / 2) : r + 2 * (u - turned) * W + half * W;
    }
    return W == 1 ? 2 * u + half : u * W + half * (D / 2);
  }
  // elements (first, second) of pair e of a lane
  static __device__ __forceinline__ int first(int e) { return kAcross ? e / W * 2 * W + e % W : 2 * e; }
  static __device__ __forceinline__ int second(int e) { return kAcross ? first(e) + W : 2 * e + 1; }
};

template <typename T, int W>
__device__ __forceinline__ void widen_all(const Vec<T, W>& a, float* out) {
  if constexpr (W % 2 == 0) {
#pragma unroll
    for (int e = 0; e < W; e += 2) {
      const float2 x = widen(&a.v[e]);
      out[e] = x.x;
      out[e + 1] = x.y;
    }
  } else {
    out[0] = widen1(a.v[0]);
  }
}

template <typename T, int W>
__device__ __forceinline__ void narrow_all(Vec<T, W>& a, const float* in) {
  if constexpr (W % 2 == 0) {
#pragma unroll
    for (int e = 0; e < W; e += 2) narrow(&a.v[e], in[e], in[e + 1]);
  } else {
    narrow1(a.v[0], in[0]);
  }
}

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The lane's weights.
template <typename S>
__device__ __forceinline__ void load_weights(const void* weight, int weight32, int lane, int r, float* w) {
  constexpr int W = sizeof(typename S::V) / sizeof(typename S::V{}.v[0]);
  using T = std::remove_reference_t<decltype(typename S::V{}.v[0])>;
#pragma unroll
  for (int v = 0; v < S::NV; ++v)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = S::column(lane, v, h, r);
#pragma unroll
      for (int e = 0; e < W; ++e)
        w[(2 * v + h) * W + e] = weight32 ? static_cast<const float*>(weight)[c + e]
                                          : widen1(static_cast<const T*>(weight)[c + e]);
    }
}

// (cos, sin) of the lane's pairs at a position, (1, 0) where a pair is not rotated; bit e: pair e is rotated
template <typename S, int W, bool HALF>
__device__ __forceinline__ unsigned load_turns(const RopeParams& p, int lane, long long pos, float2* t) {
  unsigned turned = 0;
#pragma unroll
  for (int e = 0; e < S::PAIRS; ++e) {
    int c, i;   // a column of the pair, the pair's number
    if (S::kAcross) {
      c = S::column(lane, e / W, 0, p.r) + (HALF ? e % W : 0);
      i = HALF ? c : c / 2;
    } else {
      const int at = 2 * e;   // of the lane's elements
      c = S::column(lane, at / (2 * W), at / W % 2, p.r) + at % W;
      i = c / 2;
    }
    t[e] = make_float2(1.f, 0.f);
    if (HALF ? c < p.r / 2 : c < p.r) {
      t[e] = rotation(p.inv_freq[i], pos, p.mscale, p.transposed != 0);
      turned |= 1u << e;
    }
  }
  return turned;
}

__device__ __forceinline__ long long position_of(const RopeParams& p, long long t, long long* batch, long long* n) {
  *batch = 0;
  *n = t;
  if (p.N < p.total_tokens) {
    *batch = t < 0x7fffffff ? static_cast<long long>(fast_div(static_cast<int>(t), p.div_n)) : t / p.N;
    *n = t - *batch * p.N;
  }
  const long long at = *batch * p.pos_batch + *n;
  return p.pos64 ? static_cast<const long long*>(p.positions)[at] : static_cast<const int*>(p.positions)[at];
}

constexpr int kNormUnroll = 2;   // heads whose rows are normed side by side (and as many on their way)

template <typename T, int D, int W, bool HALF, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads, 2) fa2_norm_rope_kernel(const __grid_constant__ NormParams np) {
  using S = NormShape<T, D, W, HALF>;
  using V = typename S::V;
  constexpr int U = kNormUnroll, NV = S::NV, E = S::E;
  constexpr int kTokens = kRopeThreads / S::kLanes;
  const RopeParams& p = np.r;
  __shared__ RopeToken toks[APPEND ? kTokens : 1];
  const long long tok0 = static_cast<long long>(blockIdx.x) * kTokens;
  const int n_tok = static_cast<int>(min(static_cast<long long>(kTokens), p.total_tokens - tok0));
  const int row0 = blockIdx.y * p.rows, row1 = min(row0 + p.rows, p.total_rows);
  const int k = threadIdx.x / S::kLanes, lane = threadIdx.x % S::kLanes;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // Every lane runs along to the end (the sums are the warp's); one without a token neither reads nor writes.
  bool live = k < n_tok;
  const long long t = tok0 + (live ? k : 0);
  long long pos, batch = 0, n = t, slot = -1;
  if constexpr (APPEND) {
    append_tokens(p, static_cast<int>(tok0), n_tok, toks);
    __syncthreads();
    const RopeToken o = toks[live ? k : 0];
    pos = o.pos;
    slot = o.dst;
    live = live && o.live;
  } else {
    pos = position_of(p, t, &batch, &n);
  }
  float2 turns[S::PAIRS];
  unsigned turned = 0;
  bool have_turns = false;
  int at[2 * NV];
#pragma unroll
  for (int v = 0; v < 2 * NV; ++v) at[v] = S::column(lane, v / 2, v % 2, p.r);

  // the queries' heads, the keys' and the values' of a new token, or all heads of one array
#pragma unroll 1
  for (int part = 0; part < (APPEND ? 3 : 1); ++part) {
    const T* x;
    T* y;
    long long xs, ys;
    int from = row0, to = row1;
    bool mine = live;
    const void* weight = np.weight;
    if constexpr (APPEND) {
      const int first = part == 0 ? 0 : p.Hq + (part - 1) * p.Hkv;
      from = max(row0, first) - first;
      to = min(row1, first + (part == 0 ? p.Hq : p.Hkv)) - first;
      mine = live && (part == 0 || slot >= 0);
      weight = part == 0 ? np.weight : part == 1 ? np.k_weight : nullptr;
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
    int left = to - from;   // the same for the whole block
    if (left <= 0) continue;
    x += from * xs;
    y += from * ys;
    V a[U][2 * NV], next[U][2 * NV];
    auto load = [&](V (&to_)[U][2 * NV], int count) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (mine && i < count) {
#pragma unroll
          for (int v = 0; v < 2 * NV; ++v) to_[i][v] = *reinterpret_cast<const V*>(x + at[v]);
        } else {
#pragma unroll
          for (int v = 0; v < 2 * NV; ++v) to_[i][v] = V{};
        }
        x += xs;
      }
    };
    load(a, left);
    const bool plain = APPEND && part == 2;   // values are copied
    float w[E];
    if (!plain) {
      if (weight != nullptr) {
        load_weights<S>(weight, np.weight32, lane, p.r, w);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = 1.f;
      }
      if (!have_turns) turned = load_turns<S, W, HALF>(p, lane, pos, turns);
      have_turns = true;
    }
    for (;;) {
      if (left > U) load(next, left - U);
      if (!plain) {
        float scale[U];
#pragma unroll
        for (int i = 0; i < U; ++i) scale[i] = 1.f;
        if (weight != nullptr) {
          float sum[U];
#pragma unroll
          for (int i = 0; i < U; ++i) {
            float f[E], s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int v = 0; v < 2 * NV; ++v) widen_all(a[i][v], f + v * W);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              s0 = fmaf(f[e], f[e], s0);
              s1 = fmaf(f[e + 1], f[e + 1], s1);
            }
            sum[i] = s0 + s1;
          }
#pragma unroll
          for (int o = S::kLanes / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < U; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
#pragma unroll
          for (int i = 0; i < U; ++i) scale[i] = rsqrtf(fmaf(sum[i], 1.f / D, np.eps));
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float f[E];
#pragma unroll
          for (int v = 0; v < 2 * NV; ++v) widen_all(a[i][v], f + v * W);
#pragma unroll
          for (int e = 0; e < E; ++e) f[e] *= scale[i] * w[e];
#pragma unroll
          for (int e = 0; e < S::PAIRS; ++e) {
            const int i0 = S::first(e), i1 = S::second(e);
            const float u0 = f[i0] * turns[e].x - f[i1] * turns[e].y, u1 = f[i1] * turns[e].x + f[i0] * turns[e].y;
            if (turned >> e & 1) {   // (a column that is not rotated takes nothing from another)
              f[i0] = u0;
              f[i1] = u1;
            }
          }
#pragma unroll
          for (int v = 0; v < 2 * NV; ++v) narrow_all(a[i][v], f + v * W);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (mine && i < left) {
#pragma unroll
          for (int v = 0; v < 2 * NV; ++v) *reinterpret_cast<V*>(y + at[v]) = a[i][v];
        }
        y += ys;
      }
      left -= U;
      if (left <= 0) break;
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int v = 0; v < 2 * NV; ++v) a[i][v] = next[i][v];
    }
  }
}

// Blocks take (token tile, range of heads) items one after the other, tiles innermost.
template <typename T, int D, int W, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, 2) fa2_norm_rope_grad_kernel(const __grid_constant__ NormParams np) {
  using S = NormShape<T, D, W, HALF>;
  using V = typename S::V;
  constexpr int NV = S::NV, E = S::E;
  constexpr int kTokens = kRopeThreads / S::kLanes;
  const RopeParams& p = np.r;
  __shared__ float sums[kRopeThreads / 32][D];
  const int k = threadIdx.x / S::kLanes, lane = threadIdx.x % S::kLanes;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float w[E], dw[E];
  load_weights<S>(np.weight, np.weight32, lane, p.r, w);
#pragma unroll
  for (int e = 0; e < E; ++e) dw[e] = 0.f;
  int at[2 * NV];
#pragma unroll
  for (int v = 0; v < 2 * NV; ++v) at[v] = S::column(lane, v / 2, v % 2, p.r);

#pragma unroll 1
  for (int item = blockIdx.x; item < np.items; item += gridDim.x) {
    const int range = fast_div(item, np.div_tiles), tile = item - range * np.tiles;
    const long long tok0 = static_cast<long long>(tile) * kTokens;
    const bool live = k < p.total_tokens - tok0;
    const long long t = tok0 + (live ? k : 0);
    long long batch, n;
    const long long pos = position_of(p, t, &batch, &n);
    const int row0 = range * p.rows;
    int left = min(p.rows, p.total_rows - row0);
    const T* x = static_cast<const T*>(p.x) + batch * p.x_batch + n * p.x_token + row0 * p.x_head;
    const T* g = static_cast<const T*>(np.dy) + batch * np.dy_batch + n * np.dy_token + row0 * np.dy_head;
    T* y = static_cast<T*>(p.y) + batch * p.y_batch + n * p.y_token + row0 * p.y_head;
    V xa[2 * NV], ga[2 * NV], xn[2 * NV], gn[2 * NV];
    auto load = [&](V (&vx)[2 * NV], V (&vg)[2 * NV]) {
#pragma unroll
      for (int v = 0; v < 2 * NV; ++v) {
        vx[v] = live ? *reinterpret_cast<const V*>(x + at[v]) : V{};
        vg[v] = live ? *reinterpret_cast<const V*>(g + at[v]) : V{};
      }
      x += p.x_head;
      g += np.dy_head;
    };
    load(xa, ga);
    float2 turns[S::PAIRS];
    const unsigned turned = load_turns<S, W, HALF>(p, lane, pos, turns);
    for (; left > 0; --left) {
      if (left > 1) load(xn, gn);
      float fx[E], fg[E];
#pragma unroll
      for (int v = 0; v < 2 * NV; ++v) {
        widen_all(xa[v], fx + v * W);
        widen_all(ga[v], fg + v * W);
      }
      float square = 0.f, dot = 0.f;
#pragma unroll
      for (int e = 0; e < S::PAIRS; ++e) {
        const int i0 = S::first(e), i1 = S::second(e);
        const float u0 = fg[i0] * turns[e].x - fg[i1] * turns[e].y, u1 = fg[i1] * turns[e].x + fg[i0] * turns[e].y;
        if (turned >> e & 1) {
          fg[i0] = u0;
          fg[i1] = u1;
        }
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        square = fmaf(fx[e], fx[e], square);
        dot = fmaf(fx[e], fg[e] * w[e], dot);
      }
#pragma unroll
      for (int o = S::kLanes / 2; o > 0; o >>= 1) {
        square += __shfl_xor_sync(0xffffffffu, square, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
      }
      const float r = rsqrtf(fmaf(square, 1.f / D, np.eps));
      const float along = dot * (1.f / D) * r * r;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        dw[e] = fmaf(fg[e], fx[e] * r, dw[e]);   // (rows that are not there are zeros)
        fg[e] = r * (fg[e] * w[e] - fx[e] * along);
      }
      if (live) {
#pragma unroll
        for (int v = 0; v < 2 * NV; ++v) {
          V out;
          narrow_all(out, fg + v * W);
          *reinterpret_cast<V*>(y + at[v]) = out;
        }
      }
      y += p.y_head;
#pragma unroll
      for (int v = 0; v < 2 * NV; ++v) {
        xa[v] = xn[v];
        ga[v] = gn[v];
      }
    }
  }
  // the warp's rows, then the block's warps
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int o = S::kLanes; o < 32; o <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], o);
  if ((threadIdx.x & 31) < S::kLanes) {
#pragma unroll
    for (int v = 0; v < 2 * NV; ++v)
#pragma unroll
      for (int e = 0; e < W; ++e) sums[threadIdx.x >> 5][at[v] + e] = dw[v * W + e];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kRopeThreads / 32; ++i) s += sums[i][threadIdx.x];
    np.partial[static_cast<long long>(blockIdx.x) * D + threadIdx.x] = s;
  }
}

// dweight: eight columns a block, the blocks' sums in 32 strips.
__global__ void __launch_bounds__(kRopeThreads) fa2_norm_sum_kernel(const float* __restrict__ partial, int blocks, int d,
                                                                    float* __restrict__ out) {
  __shared__ float sums[32][8];
  const int c = blockIdx.x * 8 + (threadIdx.x & 7), strip = threadIdx.x >> 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = 0.f;
#pragma unroll 4
  for (int i = strip; i < blocks; i += 32) s += partial[static_cast<long long>(i) * d + c];
  sums[strip][threadIdx.x & 7] = s;
  __syncthreads();
  if (threadIdx.x < 8) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += sums[i][threadIdx.x];
    out[c] = s;
  }
}

}  // namespace fa2dev

namespace fa2host {
namespace {

using fa2dev::NormParams;

// Vectors of 16 bytes where the call allows them.
template <typename T>
constexpr int kWide = 16 / sizeof(T);

template <typename T, int D, int W, bool HALF>
constexpr int kBlockTokens = fa2dev::kRopeThreads / fa2dev::NormShape<T, D, W, HALF>::kLanes;

template <typename T, int D, int W, bool HALF, bool APPEND>
cudaError_t run(NormParams p, int sms, cudaStream_t s) {
  constexpr int tokens = kBlockTokens<T, D, W, HALF>;
  const long long tiles = (p.r.total_tokens + tokens - 1) / tokens;
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  // heads of a block: as for the rotation alone (fa2_rope.cu)
  long long chunks = (2ll * sms + tiles - 1) / tiles;
  const long long most = (p.r.total_rows + fa2dev::kNormUnroll - 1) / fa2dev::kNormUnroll;
  if (chunks > most) chunks = most;
  if (chunks > 65535) chunks = 65535;
  p.r.rows = static_cast<int>((p.r.total_rows + chunks - 1) / chunks);
  chunks = (p.r.total_rows + p.r.rows - 1) / p.r.rows;
  p.r.div_n = make_fast_div(static_cast<int>(p.r.N > 0 ? p.r.N : 1));
  return launch_behind(fa2dev::fa2_norm_rope_kernel<T, D, W, HALF, APPEND>,
                       dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(chunks)), fa2dev::kRopeThreads, 0, s, p);
}

template <typename T, int D, int W, bool HALF>
cudaError_t run_grad(NormParams p, float* dweight, int sms, cudaStream_t s) {
  constexpr int tokens = kBlockTokens<T, D, W, HALF>;
  const long long tiles = (p.r.total_tokens + tokens - 1) / tokens;
  const long long most = static_cast<long long>(sms) * kNormGradBlocksPerSm;
  // heads of an item: at least four, and items for eight rounds of the blocks
  long long chunks = (8 * most + tiles - 1) / tiles;
  if (chunks > (p.r.total_rows + 3) / 4) chunks = (p.r.total_rows + 3) / 4;
  p.r.rows = static_cast<int>((p.r.total_rows + chunks - 1) / chunks);
  chunks = (p.r.total_rows + p.r.rows - 1) / p.r.rows;
  if (tiles * chunks > 0x7fffffffLL - most) return cudaErrorInvalidValue;
  p.items = static_cast<int>(tiles * chunks);
  p.tiles = static_cast<int>(tiles);
  p.div_tiles = make_fast_div(p.tiles);
  p.r.div_n = make_fast_div(static_cast<int>(p.r.N > 0 ? p.r.N : 1));
  const int grid = static_cast<int>(p.items < most ? p.items : most);
  const cudaError_t e = launch_behind(fa2dev::fa2_norm_rope_grad_kernel<T, D, W, HALF>, dim3(static_cast<unsigned>(grid)),
                                      fa2dev::kRopeThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  return launch_behind(fa2dev::fa2_norm_sum_kernel, dim3(D / 8), fa2dev::kRopeThreads, 0, s,
                       static_cast<const float*>(p.partial), grid, D, dweight);
}

// f(type, head dimension, vector width, halves)
template <typename F>
cudaError_t by_shape(int dtype, int d, bool wide, bool interleaved, const F& f) {
  const auto layout = [&](auto t, auto dim) {
    using T = decltype(t);
    using fa2dev::Int;
    if (interleaved) return wide ? f(t, dim, Int<kWide<T>>{}, std::false_type{}) : f(t, dim, Int<1>{}, std::false_type{});
    return wide ? f(t, dim, Int<kWide<T>>{}, std::true_type{}) : f(t, dim, Int<1>{}, std::true_type{});
  };
  const auto size = [&](auto t) {
    using fa2dev::Int;
    return d == 64 ? layout(t, Int<64>{}) : d == 128 ? layout(t, Int<128>{}) : layout(t, Int<256>{});
  };
  if (dtype == FA2_DTYPE_BF16) return size(__nv_bfloat16{});
  if (dtype == FA2_DTYPE_FP16) return size(__half{});
  return size(float{});
}

}  // namespace

cudaError_t launch_norm_rope(NormParams p, bool append, int dtype, bool wide, int sms, cudaStream_t s) {
  return by_shape(dtype, p.r.d, wide, p.r.interleaved != 0, [&](auto t, auto dim, auto w, auto half) {
    using T = decltype(t);
    if constexpr (!std::is_same_v<T, float>) {   // (a cache holds 16-bit elements)
      if (append) return run<T, decltype(dim)::value, decltype(w)::value, decltype(half)::value, true>(p, sms, s);
    }
    return run<T, decltype(dim)::value, decltype(w)::value, decltype(half)::value, false>(p, sms, s);
  });
}

cudaError_t launch_norm_rope_grad(NormParams p, float* dweight, int dtype, bool wide, int sms, cudaStream_t s) {
  return by_shape(dtype, p.r.d, wide, p.r.interleaved != 0, [&](auto t, auto dim, auto w, auto half) {
    return run_grad<decltype(t), decltype(dim)::value, decltype(w)::value, decltype(half)::value>(p, dweight, sms, s);
  });
}

}  // namespace fa2host
