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
//
// Measured: 4 x 16 heads x 4096 rows of 128 columns in bf16: forward (134 MB) 28.7-29.4 us
// a call, 4.6 TB/s; gradients (201 MB) 45-46 us, 4.4 TB/s; the warps' issue slots are 55 to
// 60% busy, a third of that with the sines.  The same rows in fp32 (twice the bytes): 45.7 and
// 67.4 us, 5.9 and 6.0 TB/s.  Rows off 16-byte boundaries, or 20 rotated columns (W = 1, an element a
// load): 99 and 125 us, in fp32 103 and 127.  One token of 64 sequences appended (32 + 8
// heads normed): 7.1-9 us, latency; 8192 tokens of a prompt (201 MB): 43.4 us, 41.1 without the norm.
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

// Every pair of a lane.
template <typename S>
__host__ __device__ constexpr unsigned all_pairs() {
  return S::PAIRS == 32 ? 0xffffffffu : (1u << (S::PAIRS & 31)) - 1u;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// The partner of element pair i: the same place of the other vector where a rotated pair lies across both, else the
// pair itself the other way round.
template <int W, bool HALF, int E2>
__device__ __forceinline__ float2 partner(const float2 (&f)[E2], int i) {
  return HALF && W > 1 ? f[i % W < W / 2 ? i + W / 2 : i - W / 2] : make_float2(f[i].y, f[i].x);
}

// A lane's elements two by two: neighbours of a vector, or (vectors of one element) the pair itself.  The
// arithmetic of a row is done on both at once (packed fp32 instructions).
template <typename T, int W, int NV>
__device__ __forceinline__ void widen_pairs(const Vec<T, W> (&a)[2 * NV], float2 (&out)[W * NV]) {
#pragma unroll
  for (int i = 0; i < W * NV; ++i) {
    if constexpr (W == 1)
      out[i] = make_float2(widen1(a[2 * i].v[0]), widen1(a[2 * i + 1].v[0]));
    else
      out[i] = widen(&a[i / (W / 2)].v[2 * (i % (W / 2))]);
  }
}

template <typename T, int W, int NV>
__device__ __forceinline__ void narrow_pairs(Vec<T, W> (&a)[2 * NV], const float2 (&in)[W * NV]) {
#pragma unroll
  for (int i = 0; i < W * NV; ++i) {
    if constexpr (W == 1) {
      narrow1(a[2 * i].v[0], in[i].x);
      narrow1(a[2 * i + 1].v[0], in[i].y);
    } else {
      narrow(&a[i / (W / 2)].v[2 * (i % (W / 2))], in[i].x, in[i].y);
    }
  }
}

// y = r (own x + cross x'), x' the partner: weight and rotation of a lane's columns in one.
template <typename S, typename T, int W, bool HALF>
struct Turn {
  static constexpr int E = S::E, E2 = S::E / 2;
  float2 own[E2], cross[E2];
  unsigned turned;

  __device__ __forceinline__ void set(const void* weight, int weight32, int lane, int r, const float2 (&turns)[S::PAIRS],
                                      unsigned which) {
    float w[E], o[E], c[E];
    if (weight != nullptr) {
      load_weights<S>(weight, weight32, lane, r, w);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] = 1.f;
    }
#pragma unroll
    for (int e = 0; e < S::PAIRS; ++e) {
      const int i0 = S::first(e), i1 = S::second(e);
      o[i0] = w[i0] * turns[e].x;
      o[i1] = w[i1] * turns[e].x;
      c[i0] = -w[i1] * turns[e].y;
      c[i1] = w[i0] * turns[e].y;
    }
#pragma unroll
    for (int i = 0; i < E2; ++i) {
      own[i] = make_float2(o[2 * i], o[2 * i + 1]);
      cross[i] = make_float2(c[2 * i], c[2 * i + 1]);
    }
    turned = which;
  }
  __device__ __forceinline__ void apply(const float2 (&f)[E2], float2 r, float2 (&u)[E2]) const {
    if (turned == all_pairs<S>()) {
#pragma unroll
      for (int e = 0; e < E2; ++e) u[e] = mul2(r, fma2(partner<W, HALF>(f, e), cross[e], mul2(f[e], own[e])));
      return;
    }
    // element by element: a column that is not rotated takes nothing from another, whatever that holds
    float flat[E], o[E], c[E];
#pragma unroll
    for (int e = 0; e < E2; ++e) {
      flat[2 * e] = f[e].x;
      flat[2 * e + 1] = f[e].y;
      o[2 * e] = own[e].x;
      o[2 * e + 1] = own[e].y;
      c[2 * e] = cross[e].x;
      c[2 * e + 1] = cross[e].y;
    }
#pragma unroll
    for (int e = 0; e < S::PAIRS; ++e) {
      const int i0 = S::first(e), i1 = S::second(e);
      float u0 = flat[i0] * o[i0], u1 = flat[i1] * o[i1];
      if (turned >> e & 1) {
        u0 = fmaf(flat[i1], c[i0], u0);
        u1 = fmaf(flat[i0], c[i1], u1);
      }
      flat[i0] = u0;
      flat[i1] = u1;
    }
#pragma unroll
    for (int e = 0; e < E2; ++e) u[e] = mul2(r, make_float2(flat[2 * e], flat[2 * e + 1]));
  }
};

constexpr int kNormUnroll = 2;   // append: heads whose rows are normed side by side (and as many on their way)

template <typename T, int D, int W, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, 2) fa2_norm_append_kernel(const __grid_constant__ NormParams np) {
  using S = NormShape<T, D, W, HALF>;
  using V = typename S::V;
  constexpr int U = kNormUnroll, NV = S::NV, E = S::E;
  constexpr int kTokens = kRopeThreads / S::kLanes;
  const RopeParams& p = np.r;
  __shared__ RopeToken toks[kTokens];
  const int k = threadIdx.x / S::kLanes, lane = threadIdx.x % S::kLanes;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int at[2 * NV];
#pragma unroll
  for (int v = 0; v < 2 * NV; ++v) at[v] = S::column(lane, v / 2, v % 2, p.r);

  const int row0 = blockIdx.y * p.rows, row1 = min(row0 + p.rows, p.total_rows);
  const long long tok0 = static_cast<long long>(blockIdx.x) * kTokens;
  const int n_tok = static_cast<int>(min(static_cast<long long>(kTokens), p.total_tokens - tok0));

  // Every lane runs along to the end (the sums are the warp's); one without a token neither reads nor writes.
  bool live = k < n_tok;
  const long long t = tok0 + (live ? k : 0);
  append_tokens(p, static_cast<int>(tok0), n_tok, toks);
  __syncthreads();
  const RopeToken token = toks[live ? k : 0];
  const long long pos = token.pos, slot = token.dst;
  live = live && token.live;
  float2 turns[S::PAIRS];   // (kept from the queries' heads to the keys')
  unsigned turned = 0;
  bool have_turns = false;

  // the queries' heads, the keys' and the values' of a new token
#pragma unroll 1
  for (int part = 0; part < 3; ++part) {
    const int first = part == 0 ? 0 : p.Hq + (part - 1) * p.Hkv;
    const int from = max(row0, first) - first, to = min(row1, first + (part == 0 ? p.Hq : p.Hkv)) - first;
    const bool mine = live && (part == 0 || slot >= 0);
    const void* weight = part == 0 ? np.weight : part == 1 ? np.k_weight : nullptr;
    const long long xs = part == 0 ? p.q_head : part == 1 ? p.k_head : p.v_head;
    const long long ys = part == 0 ? p.qo_head : p.page_head;
    const T* x = static_cast<const T*>(part == 0 ? p.q : part == 1 ? p.k : p.v) +
                 t * (part == 0 ? p.q_token : part == 1 ? p.k_token : p.v_token);
    T* y = static_cast<T*>(part == 0 ? p.q_out : part == 1 ? p.k_pages : p.v_pages) +
           (part == 0 ? t * p.qo_token : slot);
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
    const bool plain = part == 2;   // values are copied
    Turn<S, T, W, HALF> turn;
    if (!plain) {
      if (!have_turns) turned = load_turns<S, W, HALF>(p, lane, pos, turns);
      have_turns = true;
      turn.set(weight, np.weight32, lane, p.r, turns, turned);
    }
    constexpr int E2 = E / 2;
    auto work = [&](V (&row)[U][2 * NV]) {
      float2 f[U][E2];
      float scale[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        widen_pairs<T, W, NV>(row[i], f[i]);
        scale[i] = 1.f;
      }
      if (weight != nullptr) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float2 sum = mul2(f[i][0], f[i][0]);
#pragma unroll
          for (int e = 1; e < E2; ++e) sum = fma2(f[i][e], f[i][e], sum);
          scale[i] = sum.x + sum.y;
        }
#pragma unroll
        for (int o = S::kLanes / 2; o > 0; o >>= 1)
#pragma unroll
          for (int i = 0; i < U; ++i) scale[i] += __shfl_xor_sync(0xffffffffu, scale[i], o);
#pragma unroll
        for (int i = 0; i < U; ++i) scale[i] = rsqrtf(fmaf(scale[i], 1.f / D, np.eps));
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const float2 r = make_float2(scale[i], scale[i]);
        float2 u[E2];
        turn.apply(f[i], r, u);
        narrow_pairs<T, W, NV>(row[i], u);
      }
    };
    auto store = [&](const V (&row)[U][2 * NV], int count) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (mine && i < count) {
#pragma unroll
          for (int v = 0; v < 2 * NV; ++v) *reinterpret_cast<V*>(y + at[v]) = row[i][v];
        }
        y += ys;
      }
    };
    // two sets of rows in turn
    for (;;) {
      if (left > U) load(next, left - U);
      if (!plain) work(a);
      store(a, left);
      left -= U;
      if (left <= 0) break;
      if (left > U) load(a, left - U);
      if (!plain) work(next);
      store(next, left);
      left -= U;
      if (left <= 0) break;
    }
  }
}

// Block b's places are norm_range(b) .. norm_range(b + 1) - 1: all (token tile, head)
// places in equal shares, tiles outermost.  (With a block for each tile and all its heads, 512 of them on 304
// slots, the 134 MB took 32 us instead of 29.)
__device__ __forceinline__ long long norm_range(long long places, long long b) { return places * b / gridDim.x; }

// A block's walk over its places.
template <int TOKENS>
struct NormWalk {
  long long place, end;
  long long t, batch, n;   // this lane's token
  int head;
  bool live;

  __device__ __forceinline__ NormWalk(const NormParams& np) {
    place = norm_range(np.places, blockIdx.x);
    end = norm_range(np.places, blockIdx.x + 1ll);
    if (place < end) seek(np.r, place / np.r.total_rows);
  }
  __device__ __forceinline__ bool more() const { return place < end; }
  // to a tile, at the head that `place` says
  __device__ __forceinline__ void seek(const RopeParams& p, long long tile) {
    head = static_cast<int>(place - tile * p.total_rows);
    const long long tok0 = tile * TOKENS;
    const int k = threadIdx.x / (kRopeThreads / TOKENS);
    live = k < p.total_tokens - tok0;
    t = tok0 + (live ? k : 0);
    batch = 0;
    n = t;
    if (p.N < p.total_tokens) {
      batch = t < 0x7fffffff ? static_cast<long long>(fast_div(static_cast<int>(t), p.div_n)) : t / p.N;
      n = t - batch * p.N;
    }
    tile_ = tile;
  }
  // the next place; true when it is of another tile
  __device__ __forceinline__ bool next(const RopeParams& p) {
    ++place;
    if (++head < p.total_rows) return false;
    if (place < end) seek(p, tile_ + 1);
    return true;
  }

 private:
  long long tile_;
};

// Rows on their way to a block: each lane copies its own vectors asynchronously into
// its own slots of a ring in shared memory, kNormStages - 1 rows ahead of the one
// that it works on, over the ends of tiles too.  Nothing there is another thread's, so
// that waiting for one's own copies is all the order it takes.  (Rows ahead in
// registers: the gradients took 54 us instead of 45.5, the forward pass 29.2 as now.  Five
// stages instead of three: 50 us and 28.7; three blocks per SM, which spill: 36 forward.)
// Rows off 16-byte boundaries (W = 1) are loaded when it is their turn.
constexpr int kNormStages = 3;
constexpr int kNormBlocksPerSm = 2;

template <typename T, int W, int VECTORS>
struct NormFeed {
  static constexpr bool kAsync = sizeof(Vec<T, W>) == 16;
  static constexpr int kBytes = kAsync ? kNormStages * kRopeThreads * VECTORS * 16 : 16;
  uint8_t* slots;

  __device__ __forceinline__ uint8_t* slot(int stage, int v) const {
    return slots + ((stage * VECTORS + v) * kRopeThreads + threadIdx.x) * 16;
  }
  // vector v of a row into the stage, zeros where it is not `live`
  __device__ __forceinline__ void copy(int stage, int v, const T* from, bool live) const {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(slot(stage, v))), "l"(from),
                 "r"(live ? 16 : 0)
                 : "memory");
  }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  static __device__ __forceinline__ void wait() {   // for all rows but the last kNormStages - 2
    asm volatile("cp.async.wait_group %0;" ::"n"(kNormStages - 2) : "memory");
  }
};

template <typename T, int D, int W, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, kNormBlocksPerSm) fa2_norm_rope_kernel(const __grid_constant__ NormParams np) {
  using S = NormShape<T, D, W, HALF>;
  using V = typename S::V;
  constexpr int NV = S::NV, E2 = S::E / 2;
  using Feed = NormFeed<T, W, 2 * NV>;
  extern __shared__ __align__(16) uint8_t norm_smem[];
  const Feed feed = {norm_smem};
  const RopeParams& p = np.r;
  const int lane = threadIdx.x % S::kLanes;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int at[2 * NV];
#pragma unroll
  for (int v = 0; v < 2 * NV; ++v) at[v] = S::column(lane, v / 2, v % 2, p.r);

  // Every lane runs along to the end (the sums are the warp's); one without a token neither reads nor writes.
  NormWalk<kRopeThreads / S::kLanes> work(np), ahead = work;
  auto row_of = [&](const decltype(work)& w) {
    return static_cast<const T*>(p.x) + w.batch * p.x_batch + w.n * p.x_token + w.head * p.x_head;
  };
  auto send = [&](int stage) {
    if (ahead.more()) {
      const T* x = row_of(ahead);
#pragma unroll
      for (int v = 0; v < 2 * NV; ++v) feed.copy(stage, v, x + at[v], ahead.live);
      ahead.next(p);
    }
    Feed::commit();
  };
  if constexpr (Feed::kAsync) {
    for (int i = 0; i < kNormStages - 1; ++i) send(i);
  }
  Turn<S, T, W, HALF> turn;
  bool fresh = true;
  int stage = 0;
  while (work.more()) {
    if (fresh) {
      float2 turns[S::PAIRS];
      const long long i = work.batch * p.pos_batch + work.n;
      const long long pos = p.pos64 ? static_cast<const long long*>(p.positions)[i] : static_cast<const int*>(p.positions)[i];
      const unsigned turned = load_turns<S, W, HALF>(p, lane, pos, turns);
      turn.set(np.weight, np.weight32, lane, p.r, turns, turned);
    }
    V row[2 * NV];
    if constexpr (Feed::kAsync) {
      Feed::wait();
#pragma unroll
      for (int v = 0; v < 2 * NV; ++v) row[v] = *reinterpret_cast<const V*>(feed.slot(stage, v));
      send(stage == 0 ? kNormStages - 1 : stage - 1);   // (the row before this one's slots)
      stage = stage == kNormStages - 1 ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int v = 0; v < 2 * NV; ++v) row[v] = work.live ? *reinterpret_cast<const V*>(row_of(work) + at[v]) : V{};
    }
    float2 f[E2], u[E2];
    widen_pairs<T, W, NV>(row, f);
    float2 square = mul2(f[0], f[0]);
#pragma unroll
    for (int e = 1; e < E2; ++e) square = fma2(f[e], f[e], square);
    const float r = rsqrtf(fmaf(row_sum<S::kLanes>(square.x + square.y), 1.f / D, np.eps));
    turn.apply(f, make_float2(r, r), u);
    narrow_pairs<T, W, NV>(row, u);
    if (work.live) {
      T* y = static_cast<T*>(p.y) + work.batch * p.y_batch + work.n * p.y_token + work.head * p.y_head;
#pragma unroll
      for (int v = 0; v < 2 * NV; ++v) *reinterpret_cast<V*>(y + at[v]) = row[v];
    }
    fresh = work.next(p);
  }
}

// The gradients.
template <typename T, int D, int W, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, fa2host::kNormGradBlocksPerSm)
    fa2_norm_rope_grad_kernel(const __grid_constant__ NormParams np) {
  using S = NormShape<T, D, W, HALF>;
  using V = typename S::V;
  constexpr int NV = S::NV, E = S::E, E2 = E / 2;
  constexpr bool kOther = HALF && W > 1;   // the partner is in the other vector
  using Feed = NormFeed<T, W, 4 * NV>;
  extern __shared__ __align__(16) uint8_t norm_smem[];
  const Feed feed = {norm_smem};
  const RopeParams& p = np.r;
  __shared__ float sums[kRopeThreads / 32][D];
  const int lane = threadIdx.x % S::kLanes;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int at[2 * NV];
#pragma unroll
  for (int v = 0; v < 2 * NV; ++v) at[v] = S::column(lane, v / 2, v % 2, p.r);
  NormWalk<kRopeThreads / S::kLanes> work(np), ahead = work;
  auto row_of = [&](const decltype(work)& w) {
    return static_cast<const T*>(p.x) + w.batch * p.x_batch + w.n * p.x_token + w.head * p.x_head;
  };
  auto grad_of = [&](const decltype(work)& w) {
    return static_cast<const T*>(np.dy) + w.batch * np.dy_batch + w.n * np.dy_token + w.head * np.dy_head;
  };
  auto send = [&](int stage) {
    if (ahead.more()) {
      const T *x = row_of(ahead), *g = grad_of(ahead);
#pragma unroll
      for (int v = 0; v < 2 * NV; ++v) {
        feed.copy(stage, v, x + at[v], ahead.live);
        feed.copy(stage, 2 * NV + v, g + at[v], ahead.live);
      }
      ahead.next(p);
    }
    Feed::commit();
  };
  if constexpr (Feed::kAsync) {
    for (int i = 0; i < kNormStages - 1; ++i) send(i);
  }
  float2 w[E2], dw[E2];
  {
    float one[E];
    load_weights<S>(np.weight, np.weight32, lane, p.r, one);
#pragma unroll
    for (int i = 0; i < E2; ++i) {
      w[i] = make_float2(one[2 * i], one[2 * i + 1]);
      dw[i] = make_float2(0.f, 0.f);
    }
  }
  // Pairs that lie across two vectors share their coefficients but for the sign of `cross`.
  constexpr int C = kOther ? E2 / 2 : E2;
  float2 own[C], cross[C];
  unsigned turned = 0;
  // A row that is not there is zeros, whose r would be infinite with eps = 0, and 0 r no number: 1 takes the place of
  // eps.  (W = 1 keeps it for a tile: with the choice at every row the compiler orders the loads so that rows off
  // 16-byte boundaries take 150 us instead of 125.  The vectors' kernel has no register left for it.)
  float eps = np.eps;
  bool fresh = true;
  int stage = 0;
  while (work.more()) {
    if (fresh) {
      eps = work.live ? np.eps : 1.f;
      float2 turns[S::PAIRS];
      const long long i = work.batch * p.pos_batch + work.n;
      const long long pos = p.pos64 ? static_cast<const long long*>(p.positions)[i] : static_cast<const int*>(p.positions)[i];
      turned = load_turns<S, W, HALF>(p, lane, pos, turns);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if constexpr (kOther) {
          own[c] = make_float2(turns[2 * c].x, turns[2 * c + 1].x);
          cross[c] = make_float2(turns[2 * c].y, turns[2 * c + 1].y);
        } else {
          own[c] = make_float2(turns[c].x, turns[c].x);
          cross[c] = make_float2(-turns[c].y, turns[c].y);
        }
      }
    }
    V xa[2 * NV], ga[2 * NV];
    if constexpr (Feed::kAsync) {
      Feed::wait();
#pragma unroll
      for (int v = 0; v < 2 * NV; ++v) {
        xa[v] = *reinterpret_cast<const V*>(feed.slot(stage, v));
        ga[v] = *reinterpret_cast<const V*>(feed.slot(stage, 2 * NV + v));
      }
      send(stage == 0 ? kNormStages - 1 : stage - 1);   // (the row before this one's slots)
      stage = stage == kNormStages - 1 ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int v = 0; v < 2 * NV; ++v) {
        xa[v] = work.live ? *reinterpret_cast<const V*>(row_of(work) + at[v]) : V{};
        ga[v] = work.live ? *reinterpret_cast<const V*>(grad_of(work) + at[v]) : V{};
      }
    }
    float2 fx[E2], fg[E2];
    widen_pairs<T, W, NV>(xa, fx);
    widen_pairs<T, W, NV>(ga, fg);
    if (turned == all_pairs<S>()) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        if constexpr (kOther) {   // vector pairs i / (W / 2): first vector at a0, second W / 2 behind it
          const int a0 = i / (W / 2) * W + i % (W / 2), a1 = a0 + W / 2;
          const float2 less = make_float2(-cross[i].x, -cross[i].y);
          const float2 u0 = fma2(fg[a1], less, mul2(fg[a0], own[i])), u1 = fma2(fg[a0], cross[i], mul2(fg[a1], own[i]));
          fg[a0] = u0;
          fg[a1] = u1;
        } else {
          fg[i] = fma2(make_float2(fg[i].y, fg[i].x), cross[i], mul2(fg[i], own[i]));
        }
      }
    } else {   // (a column that is not rotated takes nothing from another)
#pragma unroll
      for (int e = 0; e < S::PAIRS; ++e) {
        if (!(turned >> e & 1)) continue;
        if constexpr (kOther) {
          const int i = e / 2, a0 = i / (W / 2) * W + i % (W / 2), a1 = a0 + W / 2;
          float &g0 = e % 2 ? fg[a0].y : fg[a0].x, &g1 = e % 2 ? fg[a1].y : fg[a1].x;
          const float c = e % 2 ? own[i].y : own[i].x, s = e % 2 ? cross[i].y : cross[i].x;
          const float u0 = g0 * c - g1 * s, u1 = g1 * c + g0 * s;
          g0 = u0;
          g1 = u1;
        } else {
          fg[e] = fma2(make_float2(fg[e].y, fg[e].x), cross[e], mul2(fg[e], own[e]));
        }
      }
    }
    float2 square2 = make_float2(0.f, 0.f), dot2 = square2, h[E2];
#pragma unroll
    for (int i = 0; i < E2; ++i) {
      h[i] = mul2(fg[i], w[i]);
      square2 = fma2(fx[i], fx[i], square2);
      dot2 = fma2(fx[i], h[i], dot2);
    }
    float square = square2.x + square2.y, dot = dot2.x + dot2.y;
#pragma unroll
    for (int o = S::kLanes / 2; o > 0; o >>= 1) {
      square += __shfl_xor_sync(0xffffffffu, square, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    const float r = rsqrtf(fmaf(square, 1.f / D, Feed::kAsync ? (work.live ? np.eps : 1.f) : eps));
    const float along = -dot * (1.f / D) * r * r * r;
    const float2 r2 = make_float2(r, r), along2 = make_float2(along, along);
#pragma unroll
    for (int i = 0; i < E2; ++i) {
      dw[i] = fma2(fg[i], mul2(fx[i], r2), dw[i]);   // (a row that is not there adds 0)
      h[i] = fma2(h[i], r2, mul2(fx[i], along2));
    }
    if (work.live) {
      V out[2 * NV];
      narrow_pairs<T, W, NV>(out, h);
      T* y = static_cast<T*>(p.y) + work.batch * p.y_batch + work.n * p.y_token + work.head * p.y_head;
#pragma unroll
      for (int v = 0; v < 2 * NV; ++v) *reinterpret_cast<V*>(y + at[v]) = out[v];
    }
    fresh = work.next(p);
  }
  // the warp's rows, then the block's warps
#pragma unroll
  for (int i = 0; i < E2; ++i)
#pragma unroll
    for (int o = S::kLanes; o < 32; o <<= 1) {
      dw[i].x += __shfl_xor_sync(0xffffffffu, dw[i].x, o);
      dw[i].y += __shfl_xor_sync(0xffffffffu, dw[i].y, o);
    }
  if ((threadIdx.x & 31) < S::kLanes) {
#pragma unroll
    for (int v = 0; v < 2 * NV; ++v)
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float2 d = dw[(v * W + e) / 2];
        sums[threadIdx.x >> 5][at[v] + e] = (v * W + e) % 2 ? d.y : d.x;
      }
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
__global__ void __launch_bounds__(kRopeThreads) fa2_norm_sum_kernel(const float* partial, int blocks, int d,
                                                                    float* out) {   // (not restricted: see fa2_bwd_window.cu)
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

template <typename T, int D, int W, bool HALF>
cudaError_t run_append(NormParams p, int sms, cudaStream_t s) {
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
  return launch_behind(fa2dev::fa2_norm_append_kernel<T, D, W, HALF>,
                       dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(chunks)), fa2dev::kRopeThreads, 0, s, p);
}

// Blocks for the call's places, as many as run at once; at least two places each.
template <typename T, int D, int W, bool HALF>
int norm_blocks(NormParams* p, int sms, int blocks_per_sm) {
  constexpr int tokens = kBlockTokens<T, D, W, HALF>;
  p->places = (p->r.total_tokens + tokens - 1) / tokens * p->r.total_rows;
  p->r.div_n = make_fast_div(static_cast<int>(p->r.N > 0 ? p->r.N : 1));
  const long long most = (p->places + 1) / 2, slots = static_cast<long long>(sms) * blocks_per_sm;
  return static_cast<int>(most < slots ? most : slots);
}

template <typename T, int D, int W, int VECTORS>
constexpr unsigned kFeedBytes = fa2dev::NormFeed<T, W, VECTORS>::kBytes;

template <typename T, int D, int W, bool HALF>
cudaError_t run(NormParams p, int sms, cudaStream_t s) {
  constexpr unsigned smem = kFeedBytes<T, D, W, 2 * fa2dev::NormShape<T, D, W, HALF>::NV>;
  const int grid = norm_blocks<T, D, W, HALF>(&p, sms, fa2dev::kNormBlocksPerSm);
  static_assert(smem <= 49152, "more takes an attribute of the kernel");
  return launch_behind(fa2dev::fa2_norm_rope_kernel<T, D, W, HALF>, dim3(static_cast<unsigned>(grid)),
                       fa2dev::kRopeThreads, smem, s, p);
}

template <typename T, int D, int W, bool HALF>
cudaError_t run_grad(NormParams p, float* dweight, int sms, cudaStream_t s) {
  constexpr unsigned smem = kFeedBytes<T, D, W, 4 * fa2dev::NormShape<T, D, W, HALF>::NV>;
  const int grid = norm_blocks<T, D, W, HALF>(&p, sms, kNormGradBlocksPerSm);
  const cudaError_t e = launch_behind(fa2dev::fa2_norm_rope_grad_kernel<T, D, W, HALF>, dim3(static_cast<unsigned>(grid)),
                                      fa2dev::kRopeThreads, smem, s, p);
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

// The gradient's ring takes more shared memory than a kernel may have unasked.
template <typename T, int D, int W, bool HALF>
cudaError_t prepare_grad() {
  return cudaFuncSetAttribute(fa2dev::fa2_norm_rope_grad_kernel<T, D, W, HALF>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kFeedBytes<T, D, W, 4 * fa2dev::NormShape<T, D, W, HALF>::NV>);
}

}  // namespace

cudaError_t prepare_norm() {
  for (const int dtype : {FA2_DTYPE_BF16, FA2_DTYPE_FP16, FA2_DTYPE_FP32})
    for (const int d : {64, 128, 256})
      for (const bool interleaved : {false, true}) {
        const cudaError_t e = by_shape(dtype, d, true, interleaved, [](auto t, auto dim, auto w, auto half) {
          return prepare_grad<decltype(t), decltype(dim)::value, decltype(w)::value, decltype(half)::value>();
        });
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

cudaError_t launch_norm_rope(NormParams p, bool append, int dtype, bool wide, int sms, cudaStream_t s) {
  return by_shape(dtype, p.r.d, wide, p.r.interleaved != 0, [&](auto t, auto dim, auto w, auto half) {
    using T = decltype(t);
    if constexpr (!std::is_same_v<T, float>) {   // (a cache holds 16-bit elements)
      if (append) return run_append<T, decltype(dim)::value, decltype(w)::value, decltype(half)::value>(p, sms, s);
    }
    return run<T, decltype(dim)::value, decltype(w)::value, decltype(half)::value>(p, sms, s);
  });
}

cudaError_t launch_norm_rope_grad(NormParams p, float* dweight, int dtype, bool wide, int sms, cudaStream_t s) {
  return by_shape(dtype, p.r.d, wide, p.r.interleaved != 0, [&](auto t, auto dim, auto w, auto half) {
    return run_grad<decltype(t), decltype(dim)::value, decltype(w)::value, decltype(half)::value>(p, dweight, sms, s);
  });
}

}  // namespace fa2host
