// Pages of a key/value cache: reserving, forking, freeing, compacting, copying.
//
// State, all on the device: a table int32 [B, width] of page numbers (-1: none),
// lens [B], refs [P] (how many table entries name a page; 0: free).  A page that
// several sequences share is full, because fork copies the last, partly filled
// page; so appending never writes a shared page.  Free pages are taken lowest
// number first, in the order of the sequences (reserve) or pairs (fork): results
// do not depend on timing.  Counts change by integer atomics, whose order does
// not matter.
//
// Each operation is one planning block, which ranks pages by ballots over
// chunks of the reference counts, and where page data moves a copy kernel
// behind it on the same stream (made ready while the block plans), which reads
// the planned list: nothing returns to the host.  Bound: planning by the latency
// of one block's passes over refs, copying by bytes (each page read and written
// once): compacting 4096 pages of 32 KB in 8 planes, 543 MB moved, takes 94.7-94.9
// us, 5.7 TB/s; a beam step of 8 groups of 4 sequences (free, fork, reserve),
// 23.6-28.6 us, is four dependent launches.
#include "fa2_launch.h"
#include "fa2_pages.h"

namespace fa2dev {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanPer = 8;                                  // counts per thread and pass
constexpr int kPlanChunk = kPlanThreads * kPlanPer;

// The next kernel on the stream may be made ready; the one before is complete
// from here on.  All kernels here begin so, whole grids, before any access.
__device__ __forceinline__ void begin_behind() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Exclusive prefix sum of v over the block (thread order) and the total.
__device__ __forceinline__ int block_scan(int v, int* total, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int sum = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += a;
  }
  __syncthreads();   // the last call's sums are read
  if (lane == 31) warp_sums[warp] = sum;
  __syncthreads();
  int w = lane < kPlanWarps ? warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += a;
  }
  *total = __shfl_sync(0xffffffffu, w, kPlanWarps - 1);
  const int before = warp == 0 ? 0 : __shfl_sync(0xffffffffu, w, warp - 1);
  return before + sum - v;
}

// Whole block: calls found(page, rank) for the pages of [first, last) with
// pick(count) in ascending order, until `want` are found; returns how many were
// (at most want).  Warp w of a pass looks at kPlanPer x 32 neighbouring pages.
template <typename Pick, typename Found>
__device__ __forceinline__ int rank_pages(const int* refs, int first, int last, int want, int* warp_sums, Pick pick,
                                          Found found) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int done = 0;
  for (int c0 = first; c0 < last && done < want; c0 += kPlanChunk) {
    const int w0 = c0 + warp * kPlanPer * 32;
    unsigned has[kPlanPer];
    int mine = 0;
    int v[kPlanPer];
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
      const int page = w0 + k * 32 + lane;
      v[k] = page < last ? refs[page] : 0;
    }
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
      has[k] = __ballot_sync(0xffffffffu, w0 + k * 32 + lane < last && pick(v[k]));
      mine += __popc(has[k]);
    }
    int total;
    const int before = block_scan(lane == 31 ? mine : 0, &total, warp_sums);
    // lane 31 holds the warp's count, so its exclusive sum is the warp's start
    int rank = done + __shfl_sync(0xffffffffu, before, 31);
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
      const int r = rank + __popc(has[k] & ((1u << lane) - 1));
      if ((has[k] >> lane & 1) && r < want) found(w0 + k * 32 + lane, r);
      rank += __popc(has[k]);
    }
    done += total;
  }
  return min(done, want);
}

__device__ __forceinline__ int pages_for(long long tokens, int log2) {
  return static_cast<int>((tokens + (1 << log2) - 1) >> log2);
}

// missing: 0, or the pages that lacked, or -1 (a row of the table too short); nothing is changed unless 0.
__global__ void __launch_bounds__(kPlanThreads)
    fa2_pages_reserve_kernel(const PageTables t, const int* add, int* missing, int* fresh) {
  begin_behind();
  __shared__ int warp_sums[kPlanWarps];
  __shared__ int narrow;
  if (threadIdx.x == 0) narrow = 0;
  __syncthreads();
  auto growth = [&](int b, long long& len) {
    const int have = max(t.lens[b], 0);
    len = have + static_cast<long long>(max(add[b], 0));
    return static_cast<int>(((len + (1 << t.page_log2) - 1) >> t.page_log2) - pages_for(have, t.page_log2));
  };
  long long need = 0;
  for (int b0 = 0; b0 < t.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    int grow = 0;
    if (b < t.B) {
      long long len;
      grow = min(growth(b, len), kMaxPoolPages);   // 1024 of them still fit an int
      if (len > (static_cast<long long>(t.width) << t.page_log2)) {
        narrow = 1;
        grow = 0;
      }
    }
    int total;
    block_scan(grow, &total, warp_sums);
    need += total;
  }
  __syncthreads();
  if (narrow) {
    if (threadIdx.x == 0) *missing = -1;
    return;
  }
  const int want = static_cast<int>(min(need, static_cast<long long>(t.num_pages)));   // fresh[] holds num_pages
  const int found = rank_pages(t.refs, 0, t.num_pages, want, warp_sums, [](int v) { return v == 0; },
                               [&](int page, int r) { fresh[r] = page; });
  if (found < need) {
    if (threadIdx.x == 0) *missing = static_cast<int>(min(need - found, 0x7fffffffll));
    return;
  }
  __syncthreads();   // fresh[] is written
  int before = 0;
  for (int b0 = 0; b0 < t.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    long long len = 0;
    const int grow = b < t.B ? growth(b, len) : 0;
    int total;
    const int at = before + block_scan(grow, &total, warp_sums);
    if (b < t.B) {
      int* row = t.table + b * t.table_stride + pages_for(max(t.lens[b], 0), t.page_log2);
      for (int i = 0; i < grow; ++i) {
        const int page = fresh[at + i];
        row[i] = page;
        t.refs[page] = 1;
      }
      t.lens[b] = static_cast<int>(len);
    }
    before += total;
  }
  if (threadIdx.x == 0) *missing = 0;
}

// pairs: [0] their number, then n sources and n destinations (page numbers, -1:
// nothing to copy), then n new lengths.
__global__ void __launch_bounds__(kPlanThreads)
    fa2_pages_fork_kernel(const PageTables t, const int* src, const int* dst, int n, int* missing, int* pairs) {
  begin_behind();
  __shared__ int warp_sums[kPlanWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* from = pairs + 1;
  int* to = from + n;
  int* new_len = to + n;
  // Claims: an empty destination's length becomes -(n - i) for its first pair i
  // (atomicMin), so a destination named twice goes to the first pair.
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int s = src[i], d = dst[i];
    if (s >= 0 && s < t.B && d >= 0 && d < t.B && t.lens[d] <= 0)
      atomicMin(&t.lens[d], -(n - i));
    else
      atomicOr(t.status, kDevErrPage);
  }
  __threadfence_block();
  __syncthreads();
  volatile int* lens = t.lens;
  auto won = [&](int i) {
    const int s = src[i], d = dst[i];
    return s >= 0 && s < t.B && d >= 0 && d < t.B && lens[d] == -(n - i);
  };
  const int in_page = (1 << t.page_log2) - 1;
  const long long cap = static_cast<long long>(t.width) << t.page_log2;
  // length of the source as it was at entry (a claimed source was empty)
  auto source_len = [&](int i) { return static_cast<int>(min(static_cast<long long>(max(lens[src[i]], 0)), cap)); };
  int need = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int part = 0;
    if (i < n) {
      const bool w = won(i);
      if (!w && src[i] >= 0 && src[i] < t.B && dst[i] >= 0 && dst[i] < t.B) atomicOr(t.status, kDevErrPage);
      part = w && (source_len(i) & in_page) != 0;
      from[i] = -1;
      to[i] = -1;
    }
    int total;
    block_scan(part, &total, warp_sums);
    need += total;
  }
  // free pages, kept in to[] by rank until the pairs take theirs
  __syncthreads();
  const int found = rank_pages(t.refs, 0, t.num_pages, need, warp_sums, [](int v) { return v == 0; },
                               [&](int page, int r) { from[r] = page; });
  __syncthreads();
  if (found < need) {
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
      if (won(i)) lens[dst[i]] = 0;
    if (threadIdx.x == 0) {
      *missing = need - found;
      pairs[0] = 0;
    }
    return;
  }
  // ranks of the pairs' fresh pages: to[i] = the page, then from[i] = the page it is copied from
  int before = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const int part = i < n && won(i) && (source_len(i) & in_page) != 0;
    int total;
    const int at = before + block_scan(part, &total, warp_sums);
    if (part) to[i] = from[at];
    before += total;
  }
  __syncthreads();
  for (int i = warp; i < n; i += kPlanWarps) {   // a warp per pair
    int copy_from = -1;
    if (won(i)) {
      const int len = source_len(i);
      const int full = len >> t.page_log2;
      const int* row = t.table + src[i] * t.table_stride;
      int* out = t.table + dst[i] * t.table_stride;
      for (int k = lane; k < t.width; k += 32) {
        int page = -1;
        if (k < full) {
          page = row[k];
          if (page >= 0 && page < t.num_pages)
            atomicAdd(&t.refs[page], 1);
          else
            atomicOr(t.status, kDevErrPage);
        } else if (k == full && (len & in_page) != 0) {
          page = to[i];
          t.refs[page] = 1;
          copy_from = row[k];
          if (copy_from < 0 || copy_from >= t.num_pages) atomicOr(t.status, kDevErrPage);
        }
        out[k] = page;
      }
    }
    copy_from = __reduce_max_sync(0xffffffffu, copy_from);
    __syncwarp();
    if (lane == 0) {
      from[i] = copy_from;
      new_len[i] = won(i) ? source_len(i) : -1;
    }
  }
  __syncthreads();
  // lengths last: the claims and the sources' lengths were read from them
  for (int i = threadIdx.x; i < n; i += kPlanThreads)
    if (new_len[i] >= 0) lens[dst[i]] = new_len[i];
  if (threadIdx.x == 0) {
    *missing = 0;
    pairs[0] = n;
  }
}

// One block per listed sequence.
__global__ void __launch_bounds__(128) fa2_pages_free_kernel(const PageTables t, const int* seqs, int n) {
  begin_behind();
  const int i = blockIdx.x;
  const int b = seqs[i];
  if (b < 0 || b >= t.B) {
    if (threadIdx.x == 0) atomicOr(t.status, kDevErrPage);
    return;
  }
  // listed before: that block frees it
  int again = 0;
  for (int j = threadIdx.x; j < i; j += blockDim.x) again |= seqs[j] == b;
  if (__syncthreads_or(again)) return;
  int* row = t.table + b * t.table_stride;
  for (int k = threadIdx.x; k < t.width; k += blockDim.x) {
    const int page = row[k];
    if (page < 0) continue;
    if (page >= t.num_pages)
      atomicOr(t.status, kDevErrPage);
    else if (atomicSub(&t.refs[page], 1) <= 0) {
      atomicAdd(&t.refs[page], 1);   // it was free already
      atomicOr(t.status, kDevErrPage);
    }
    row[k] = -1;
  }
  if (threadIdx.x == 0) t.lens[b] = 0;
}

// moved[p]: where page p goes (p itself when it stays, -1 when it is free).
// pairs as in fork: pages of number >= used (the count of used pages) go to the
// free numbers below it, in ascending order.
__global__ void __launch_bounds__(kPlanThreads) fa2_pages_compact_kernel(const PageTables t, int* moved, int* pairs) {
  begin_behind();
  __shared__ int warp_sums[kPlanWarps];
  int* from = pairs + 1;
  int* to = from + t.num_pages;
  int used = 0;
  for (int c0 = 0; c0 < t.num_pages; c0 += kPlanChunk) {
    int mine = 0;
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
      const int page = c0 + k * kPlanThreads + threadIdx.x;
      const bool u = page < t.num_pages && t.refs[page] > 0;
      if (page < t.num_pages) moved[page] = u ? page : -1;
      mine += u;
    }
    int total;
    block_scan(mine, &total, warp_sums);
    used += total;
  }
  const int movers = rank_pages(t.refs, used, t.num_pages, t.num_pages, warp_sums, [](int v) { return v > 0; },
                                [&](int page, int r) { from[r] = page; });
  rank_pages(t.refs, 0, used, movers, warp_sums, [](int v) { return v <= 0; }, [&](int page, int r) { to[r] = page; });
  __syncthreads();
  for (int i = threadIdx.x; i < movers; i += kPlanThreads) {
    moved[from[i]] = to[i];
    t.refs[to[i]] = t.refs[from[i]];
    t.refs[from[i]] = 0;
  }
  if (threadIdx.x == 0) pairs[0] = movers;
}

// Pairs of fa2_pages_copy: a warp per pair looks through the list.  A pair is
// dropped when a later one has its destination (the last one counts); a pair
// whose source another pair writes is refused.
__global__ void __launch_bounds__(256)
    fa2_pages_pairs_kernel(const int* src, const int* dst, int n, int num_pages, int* pairs, int* status) {
  begin_behind();
  const int lane = threadIdx.x & 31;
  const int i = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (blockIdx.x == 0 && threadIdx.x == 0) pairs[0] = n;
  if (i >= n) return;
  const int s = src[i], d = dst[i];
  bool later = false, written = false;
  for (int j = lane; j < n; j += 32) {
    if (j == i) continue;
    const int dj = dst[j];
    later |= j > i && dj == d;
    written |= dj == s && src[j] != dj;
  }
  later = __any_sync(0xffffffffu, later);
  written = __any_sync(0xffffffffu, written);
  if (lane == 0) {
    const bool bad = s < 0 || s >= num_pages || d < 0 || d >= num_pages || (written && s != d);
    if (bad) atomicOr(status, kDevErrPage);
    pairs[1 + i] = bad || later || s == d ? -1 : s;
    pairs[1 + n + i] = d;
  }
}

constexpr int kCopyThreads = 256;
constexpr int kCopyPer = 4;   // 16-byte vectors in flight per thread
constexpr int kCopyChunk = kCopyThreads * kCopyPer * 16;

// The listed pairs of every plane, chunk by chunk; and, when `moved` is given,
// the table entries renamed by it.
__global__ void __launch_bounds__(kCopyThreads)
    fa2_pages_copy_kernel(const __grid_constant__ PagePlanes d, const int* pairs, int room, const PageTables t,
                          const int* moved) {
  // launched while the list is planned: it is there from here on
  begin_behind();
  const int n = min(pairs[0], room);
  const int* from = pairs + 1;
  const int* to = from + room;
  const int chunks = static_cast<int>((d.page_bytes + kCopyChunk - 1) / kCopyChunk);
  const long long total = static_cast<long long>(n) * d.planes * chunks;
  for (long long item = blockIdx.x; item < total; item += gridDim.x) {
    const long long pp = item / chunks;
    const long long off = (item - pp * chunks) * kCopyChunk;
    const int pair = static_cast<int>(pp / d.planes);
    const int plane = static_cast<int>(pp - static_cast<long long>(pair) * d.planes);
    const int a = from[pair], b = to[pair];
    if (a < 0 || a >= d.num_pages || b < 0 || b >= d.num_pages) continue;
    const char* x = static_cast<const char*>(d.base[plane]) + a * d.stride + off;
    char* y = static_cast<char*>(d.base[plane]) + b * d.stride + off;
    const long long left = d.page_bytes - off;
    uint4 v[kCopyPer];
#pragma unroll
    for (int k = 0; k < kCopyPer; ++k) {
      const int at = (k * kCopyThreads + threadIdx.x) * 16;
      if (at < left) v[k] = *reinterpret_cast<const uint4*>(x + at);
    }
#pragma unroll
    for (int k = 0; k < kCopyPer; ++k) {
      const int at = (k * kCopyThreads + threadIdx.x) * 16;
      if (at < left) *reinterpret_cast<uint4*>(y + at) = v[k];
    }
  }
  if (moved != nullptr) {
    const long long entries = static_cast<long long>(t.B) * t.width;
    for (long long e = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x; e < entries;
         e += static_cast<long long>(gridDim.x) * kCopyThreads) {
      const long long b = e / t.width;
      int* at = t.table + b * t.table_stride + (e - b * t.width);
      const int page = *at;
      if (page < 0) {
        if (page != -1) *at = -1;
      } else if (page >= t.num_pages) {
        atomicOr(t.status, kDevErrPage);
      } else {
        *at = moved[page];
      }
    }
  }
}

}  // namespace fa2dev

namespace fa2host {
namespace {

using namespace fa2dev;

// Blocks of the copy kernel: as many as there may be chunks, at most eight an SM.
unsigned copy_grid(long long pairs, const PagePlanes& d, int sms) {
  const long long chunks = (d.page_bytes + kCopyChunk - 1) / kCopyChunk * d.planes * pairs;
  const long long most = 8ll * sms;
  return static_cast<unsigned>(chunks < 1 ? 1 : (chunks > most ? most : chunks));
}

}  // namespace

cudaError_t launch_pages_reserve(const PageTables& t, const int* add, int* missing, int* ws, cudaStream_t s) {
  return launch_behind(fa2_pages_reserve_kernel, dim3(1), kPlanThreads, 0, s, t, add, missing, ws);
}

cudaError_t launch_pages_fork(const PageTables& t, const int* src, const int* dst, int n, const PagePlanes& d,
                              int* missing, int* ws, int sms, cudaStream_t s) {
  const cudaError_t e = launch_behind(fa2_pages_fork_kernel, dim3(1), kPlanThreads, 0, s, t, src, dst, n, missing, ws);
  if (e != cudaSuccess) return e;
  return launch_behind(fa2_pages_copy_kernel, dim3(copy_grid(n, d, sms)), kCopyThreads, 0, s, d, ws, n, t,
                       static_cast<const int*>(nullptr));
}

cudaError_t launch_pages_free(const PageTables& t, const int* seqs, int n, cudaStream_t s) {
  return launch_behind(fa2_pages_free_kernel, dim3(static_cast<unsigned>(n)), 128, 0, s, t, seqs, n);
}

cudaError_t launch_pages_compact(const PageTables& t, const PagePlanes& d, int* moved, int* ws, int sms,
                                 cudaStream_t s) {
  const cudaError_t e = launch_behind(fa2_pages_compact_kernel, dim3(1), kPlanThreads, 0, s, t, moved, ws);
  if (e != cudaSuccess) return e;
  return launch_behind(fa2_pages_copy_kernel, dim3(copy_grid(t.num_pages, d, sms)), kCopyThreads, 0, s, d, ws, t.num_pages,
                       t, moved);
}

cudaError_t launch_pages_copy(const PagePlanes& d, const int* src, const int* dst, int n, int* ws, int* status,
                              int sms, cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(n) * 32 + 255) / 256);
  const cudaError_t e = launch_behind(fa2_pages_pairs_kernel, dim3(blocks), 256, 0, s, src, dst, n, d.num_pages, ws, status);
  if (e != cudaSuccess) return e;
  return launch_behind(fa2_pages_copy_kernel, dim3(copy_grid(n, d, sms)), kCopyThreads, 0, s, d, ws, n, PageTables{},
                       static_cast<const int*>(nullptr));
}

}  // namespace fa2host
