// Attention over a paged cache whose sequences share prefixes: the kernel that
// joins a row's results.
#include "fa2_launch.h"

namespace fa2dev {

constexpr int kJoinWarps = 4;
constexpr int kJoinRows = 8;   // rows of a block

// The launch over the groups' shared pages (pre) and that over the sequences' own pages
// (own) leave a row's result in parts over disjoint keys: the whole of an item in O
// and LSE, or its pieces in the workspace.  With m = max_s L_s and w_s = exp(L_s - m) over
// all of them: O = sum_s w_s O_s / sum w_s, LSE = m + log sum w_s; parts with L_s =
// -inf have w_s = 0 and their O is not used.
//
// A block has eight rows (token, query head) of one key/value head, a lane one row and
// four of every 16 columns, so that reads are 128 neighbouring bytes at least; its
// four warps take every fourth part each, in the order of the lists, and add up
// through shared memory, always in the same order.  Whose token it is and its group
// are looked up by every lane for its row, while the launch before still runs; then
// the entries of its items.  Bound: the latency of dependent loads, the parts' among them.
template <int D, bool F16>
__global__ void __launch_bounds__(kJoinWarps * 32) fa2_paged_join_kernel(const __grid_constant__ PagedParams pre,
                                                                         const __grid_constant__ PagedParams own,
                                                                         int pre_block, int own_block, void* O,
                                                                         float* LSE, int half_out) {
  __shared__ float4 sums[kJoinWarps - 1][D / 16][32];
  __shared__ float2 weights[kJoinWarps - 1][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane >> 3;
  const int head = blockIdx.y, G = own.G;
  const long long at = static_cast<long long>(blockIdx.x) * kJoinRows + (lane & 7);
  bool live = at < static_cast<long long>(own.T) * G;
  const int t = live ? static_cast<int>(at / G) : 0, h = live ? static_cast<int>(at - static_cast<long long>(t) * G) : 0;
  int b = t, q0 = t;
  if (own.cu_q != nullptr) {   // the last sequence that begins at or before t
    int lo = 0, n = own.B;
    while (n > 1) {
      const int half = n / 2;
      if (own.cu_q[lo + half] <= t) {
        lo += half;
        n -= half;
      } else {
        n = half;
      }
    }
    b = lo;
    q0 = max(0, own.cu_q[b]);
    live = live && q0 <= t && t < own.cu_q[b + 1];   // (else nobody's)
  }
  // the group, as paged_shared finds it
  int group_at = 0, group_begin = 0;
  bool grouped = false;
  if (live) {
    int n = pre.groups;
    while (n > 1) {
      const int half = n / 2;
      if (pre.cu_groups[group_at + half] <= b) {
        group_at += half;
        n -= half;
      } else {
        n = half;
      }
    }
    const PagedGroup g = paged_group(pre, own.B, group_at);
    if (g.prefix > 0 && g.first <= b && b < g.last) {
      group_begin = own.cu_q != nullptr ? max(0, own.cu_q[g.first]) : g.first;
      grouped = group_begin <= t;
    }
  }
  // What was read above neither launch writes, and it was complete when they started; their
  // results are complete from here on.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long row = static_cast<long long>(t) * own.Hq + head * G + h;
  struct List {
    int4 e;
    long long prow;   // the row within a slot
  };
  // A list that does not lie in the workspace (offsets that contradict each other) is reported and left out.
  auto look_up = [&](const PagedParams& p, int first, int block, int seq) {
    List l;
    const int i = (t - first) / block;
    l.e = p.parts[paged_entry(p, first, block, i, seq, head)];
    l.prow = static_cast<long long>(t - first - i * block) * G + h;
    const bool good = l.e.z >= 1 && l.e.z <= p.ctas + 1 && l.e.x >= -1 && l.e.x < p.slots && l.prow < p.part_rows &&
                      (l.e.x >= 0 || l.e.z == 1) && (l.e.z == 1 || (l.e.y >= 0 && l.e.y + (l.e.z - 2) * 2 < p.slots));
    if (!good) {
      atomicOr(p.status, kDevErrPage);
      l.e.z = 0;
    }
    return l;
  };
  List mine = {}, shared = {};
  if (live) {
    mine = look_up(own, q0, own_block, b);
    if (grouped) shared = look_up(pre, group_begin, pre_block, group_at);
  }
  const int parts = mine.e.z + shared.e.z;
  float4 acc[D / 16];
#pragma unroll
  for (int c = 0; c < D / 16; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f, m = -INFINITY;
#pragma unroll 2
  for (int s = warp; s < parts; s += kJoinWarps) {
    const bool first = s < mine.e.z;
    const PagedParams& p = first ? own : pre;
    const List& l = first ? mine : shared;
    const int k = first ? s : s - mine.e.z;
    const long long slot = k == 0 ? l.e.x : l.e.y + (k - 1) * 2;
    const float* x0;
    long long step;
    float ls;
    if (slot < 0) {
      ls = p.LSE[row];
      x0 = static_cast<const float*>(p.O) + row * D + group * 4;
      step = 16;
    } else {
      ls = p.LSE_part[slot * p.part_rows + l.prow];
      x0 = p.O_part + slot * p.part_rows * D + (static_cast<long long>(group) * p.part_rows + l.prow) * 4;
      step = 16ll * p.part_rows;
    }
    float4 x[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c) x[c] = *reinterpret_cast<const float4*>(x0 + c * step);
    const float top = fmaxf(m, ls);
    const float keep = m == -INFINITY ? 0.f : expf(m - top), e = ls == -INFINITY ? 0.f : expf(ls - top);
    m = top;
    sum = fmaf(sum, keep, e);
    const bool has = e != 0.f;   // (the O of a part without keys was not written)
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      acc[c].x = fmaf(acc[c].x, keep, has ? e * x[c].x : 0.f);
      acc[c].y = fmaf(acc[c].y, keep, has ? e * x[c].y : 0.f);
      acc[c].z = fmaf(acc[c].z, keep, has ? e * x[c].z : 0.f);
      acc[c].w = fmaf(acc[c].w, keep, has ? e * x[c].w : 0.f);
    }
  }
  if (warp > 0) {
#pragma unroll
    for (int c = 0; c < D / 16; ++c) sums[warp - 1][c][lane] = acc[c];
    weights[warp - 1][lane] = make_float2(m, sum);
  }
  __syncthreads();
  if (warp > 0 || !live) return;
#pragma unroll
  for (int w = 0; w < kJoinWarps - 1; ++w) {
    const float2 other = weights[w][lane];
    const float top = fmaxf(m, other.x);
    const float keep = m == -INFINITY ? 0.f : expf(m - top), e = other.x == -INFINITY ? 0.f : expf(other.x - top);
    m = top;
    sum = fmaf(sum, keep, e * other.y);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const float4 y = sums[w][c][lane];
      acc[c].x = fmaf(acc[c].x, keep, e * y.x);
      acc[c].y = fmaf(acc[c].y, keep, e * y.y);
      acc[c].z = fmaf(acc[c].z, keep, e * y.z);
      acc[c].w = fmaf(acc[c].w, keep, e * y.w);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    const long long to = row * D + c * 16 + group * 4;
    const float4 x = make_float4(acc[c].x * inv, acc[c].y * inv, acc[c].z * inv, acc[c].w * inv);
    if (half_out)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(O) + to) =
          make_uint2(pack_x2<F16>(x.x, x.y), pack_x2<F16>(x.z, x.w));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(O) + to) = x;
  }
  if (group == 0) LSE[row] = sum == 0.f ? -INFINITY : m + logf(sum);
}

}  // namespace fa2dev

namespace fa2host {

cudaError_t launch_paged_join(int d, bool f16, const fa2dev::PagedParams& p0, int subs0, const fa2dev::PagedParams& p1,
                              int subs1, void* O, float* LSE, bool half_out, cudaStream_t s) {
  const long long rows = static_cast<long long>(p1.T) * p1.G;
  const dim3 grid(static_cast<unsigned>((rows + fa2dev::kJoinRows - 1) / fa2dev::kJoinRows),
                  static_cast<unsigned>(p1.Hkv));
  const auto kernel = d == 64    ? (f16 ? fa2dev::fa2_paged_join_kernel<64, true> : fa2dev::fa2_paged_join_kernel<64, false>)
                      : d == 128 ? (f16 ? fa2dev::fa2_paged_join_kernel<128, true> : fa2dev::fa2_paged_join_kernel<128, false>)
                                 : (f16 ? fa2dev::fa2_paged_join_kernel<256, true> : fa2dev::fa2_paged_join_kernel<256, false>);
  return launch_behind(kernel, grid, fa2dev::kJoinWarps * 32, 0, s, p0, p1, p0.sub_tokens * subs0, p1.sub_tokens * subs1,
                       O, LSE, half_out ? 1 : 0);
}

}  // namespace fa2host
