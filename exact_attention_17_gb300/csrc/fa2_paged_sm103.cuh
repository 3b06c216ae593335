// Attention of a chunk of new tokens over a paged key/value cache (sm_103a).
//
// Sequence b has n_b keys in the cache (its new tokens' among them) and c_b
// new query tokens, the last of its n_b positions.  Query heads come in groups
// of G that share a key/value head.  For the new token i, query head h:
//   s_j = scale * q_ih . k_j,  j < n_b, and j <= n_b - c_b + i when causal
//   O_ih = sum_j softmax_j(s_j) v_j,   LSE_ih = log sum_j exp(s_j)
// A row that keeps no key (n_b = 0, or n_b - c_b + i < 0) gets O = 0 and
// LSE = -inf.  The online softmax, its lazy offset, the named barriers and the
// two ping-ponged sub-tiles are those of the dense forward kernel
// (fa2_fwd_sm103.cuh); what differs:
//
//  * Rows.  A sub-tile's 128 rows are (token, head of the group) pairs of one
//    key/value head: row = token * G + head.  So one token of 8 heads fills 8
//    rows of the MMA instead of one, and K/V is read once per group.  Rows past
//    the block's tokens compute on whatever the buffer holds (rows do not
//    mix) and are not stored; a warp without a live row skips its softmax.
//  * Few rows.  One warp's softmax of a tile costs the same for one live row as
//    for 32, and as much as the tile's MMAs.  So a block of at most 32 rows
//    (NARROW: single tokens) loads its queries four times, into each warp's 32
//    rows of the tile, and warp w takes the keys 32 w .. 32 w + 31 of every tile:
//    its P is zero elsewhere, so its rows of O hold the share of those keys.
//    The four shares are merged at the end like parts of an item.
//  * Pages.  A 128-key tile is read through a 4-D tensor map (column, slot,
//    head, page), one box per page and 64 columns, page numbers from the table
//    (32 entries at a time in the producer warp's lanes).  Any strides that TMA
//    takes do.  Numbers outside the cache read zeros (TMA bounds) and set the
//    status word.
//  * Stale slots.  Slots behind a sequence's last key may hold anything, NaN
//    too.  Their scores are replaced by -inf before the softmax; their V rows
//    (0 * NaN is NaN in the MMA) are overwritten with zeros in shared memory
//    by the softmax threads before they announce P.
//  * Schedule.  Lengths live on the device and may change between replays of a
//    captured launch, so the kernel finds its work itself.  An item is a
//    (sequence, block of tokens, key/value head), its cost its keys and a fixed
//    part.  With `even` the list of all items is cut into ranges of equal cost,
//    one per CTA of a single wave: a CTA walks its range segment by segment, at
//    most its first and last segment being parts of an item.
//    Without it (many items, the host's choice) the CTAs take whole items one
//    after the other from a counter, in an order that keeps a group of heads in
//    L2, items of more than an even share of the tiles being cut; who computes
//    an item does not change it.  A part's normalised O and LSE go to the workspace,
//    and a second kernel merges them (as fa2_combine.cu, in the order of the
//    keys: results do not depend on timing).
//  * Producers.  The tiled copies that one warp issues run one after the other:
//    20.8 bytes per clock in boxes of 16 KB (a 128-byte row in 6 clocks), 14.0 in
//    boxes of 2 KB, whichever lanes issue them; two warps reach 40.5, four 75 to
//    82.  Two 128-row sub-tiles take a 64 KB key tile in about 3000 clocks at head
//    dimension 128, more than one warp delivers in small pages: two warps share
//    each tile there, by columns (8192 tokens over 16384 keys in pages of 16, 32
//    and 128: 1327, 1180 and 1173 -> 1141, 1116 and 1117 us; a warp each for K and
//    V was slower than one).  At 256 a tile is 64 KB, and with room for one of K
//    and one of V a copy starts only when the MMAs of the tile before are done:
//    three warps share each tile (200 -> 171 us for 2600 tokens over 2000-4096
//    keys when K had two warps and V one).
//  * Segments.  The producer warp runs ahead: it loads the next segment's Q and
//    first tiles while the current one finishes.  One named barrier per segment,
//    which every role passes for every segment, also after an abort, hands over
//    the segment's description (the other producers have one of their own, ahead
//    of it).  A ring of descriptions that each role reads at its own pace was
//    slower: 1115 -> 1158 us for those 8192 tokens.
//
// Bound and measured.  Single tokens: bytes (64 sequences of 1000-8192 keys, 8
// key/value heads of 128: 1.11 GB in 169.5-172 us, 6.48-6.57 TB/s; four of
// 100000-131072 keys, d = 64: 84.3-85.7 us, 5.6-5.7 TB/s).  Chunks: the tensor pipe,
// fed by one issuing thread per SM, and the K/V tiles that the SMs read from L2
// (8192 tokens over 16384 keys, 32 heads of 128, causal: 1115-1150 us on different
// GPUs, 1435-1480 TFLOP/s; d = 256: 159-160 us for 146 GFLOP, each SM reading 128 KB
// a tile).  Small calls: latency, 4 us from the launch to the first S, 2 us a tile,
// and the merge (two tokens over 1000 keys: 13.8-14.1 us, the merge's launch
// included).
#pragma once

#include <type_traits>

#include "fa2_fwd_sm103.cuh"

namespace fa2dev {

// A page number, length or offset read on the device lies outside the cache.
constexpr int kDevErrPage = 2;

struct PagedParams {
  const int* page_table;   // [B, table_stride]
  const int* kv_lens;      // [B]
  const int* cu_q;         // [B + 1], or null: one token per sequence
  void* O;                 // [T, Hq, D] fp32, or the input type (o_half)
  float* LSE;              // [T, Hq]
  float* O_part;           // [slots][D / 4][part_rows][4]: a warp's rows write 512 neighbouring bytes
  float* LSE_part;         // [slots][part_rows]
  int slots;
  int part_rows;
  int B, T, Hq, Hkv, G;
  int sub_tokens;          // tokens per sub-tile (sub_tokens * G <= 128 rows)
  int box_tokens;          // tokens per Q box (divides sub_tokens)
  int page_log2;           // log2 of the slots per page
  int num_pages;
  long long table_stride;
  int max_len;             // table_width << page_log2, at most 2^30
  int even;                // equal ranges of the work, one per CTA (else whole items)
  int ctas;                // CTAs of the grid; an item of more than one CTA's share is cut
  int* counter;            // whole items: how many CTAs have taken besides their first (starts at 0)
  double inv_ctas;
  int min_tiles;           // least key tiles per range
  int item_keys;           // what an item costs besides its keys, in keys
  int causal;
  int o_half;
  int narrow;              // blocks of at most 32 rows
  float scale_log2;
  int* status;
  unsigned long long timeout_ns;
};

// Key tiles [t_begin, t_end) of an item.
struct PagedUnit {
  int valid;
  int head;
  int row0;       // first token of the block in the packed queries
  int tok0;       // the same within its sequence
  int ntok;       // tokens of the block
  int q_len, kv_len;
  int t_begin, t_end;
  int slot;       // workspace slot of this part, -1: the whole item
  long long table;   // offset of the sequence's row in the page table
};

// Keys that the token `tok` of a sequence keeps: [0, kept).
__device__ __forceinline__ int paged_kept(int causal, int kv_len, int q_len, int tok) {
  return causal ? max(0, min(kv_len, kv_len - q_len + tok + 1)) : kv_len;
}

__device__ __forceinline__ int key_tiles_of(int keys) { return (keys + kKeysPerTile - 1) / kKeysPerTile; }

// Sequence b's new tokens and keys.
struct PagedSeq {
  int q0, q_len, kv_len, blocks;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b, int block) {
  int begin = 0, end = 0, kv = 0;   // nothing for b >= B
  if (b < p.B) {
    begin = p.cu_q ? p.cu_q[b] : b;
    end = p.cu_q ? p.cu_q[b + 1] : b + 1;
    kv = p.kv_lens[b];
  }
  PagedSeq s;
  s.q0 = min(max(begin, 0), p.T);
  s.q_len = max(0, min(end, p.T) - s.q0);
  s.kv_len = min(max(kv, 0), p.max_len);
  if (blockIdx.x == 0 && (begin < 0 || end < begin || end > p.T || kv < 0 || kv > p.max_len))
    atomicOr(p.status, kDevErrPage);
  s.blocks = (s.q_len + block - 1) / block;
  return s;
}

// Cost of an item: item_keys for its start and end, then its keys, at least one (a
// lone sub-tile takes about as long as two, whose MMAs and softmax overlap).
// Sums of costs over a sequence's blocks are closed forms in keys, which tiles
// would not be; a position x inside an item stands for tile ceil((x - item_keys) /
// 128), cut to the item's tiles.
__device__ __forceinline__ int block_keys(const PagedParams& p, const PagedSeq& s, int block, int i) {
  return max(1, paged_kept(p.causal, s.kv_len, s.q_len, min((i + 1) * block, s.q_len) - 1));
}

// Cost of the blocks 0 .. i-1 of a sequence (0 <= i <= blocks).
template <int SUBS>
__device__ __forceinline__ long long cost_before(const PagedParams& p, const PagedSeq& s, int i) {
  if (i == 0) return 0;
  const int block = p.sub_tokens * SUBS;
  // all but the last block are full: block k keeps kv_len - q_len + (k + 1) block keys when causal
  const int full = i == s.blocks ? i - 1 : i;
  long long keys;
  if (p.causal) {
    const long long lead = static_cast<long long>(s.kv_len) - s.q_len;
    const int none = lead >= 0 ? 0 : min(full, static_cast<int>(-lead) / block);   // blocks without a key count one
    const long long n = full - none;
    keys = none + n * (lead + none * static_cast<long long>(block)) + block * (n * (n + 1) / 2);
  } else {
    keys = static_cast<long long>(full) * max(1, s.kv_len);
  }
  keys += static_cast<long long>(i) * p.item_keys;
  if (i == s.blocks) keys += max(1, s.kv_len);
  return keys;
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ long long warp_scan(long long v) {   // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += a;
  }
  return v;
}

__device__ __forceinline__ PagedSeq seq_from(const PagedSeq& s, int src) {
  PagedSeq r;
  r.q0 = __shfl_sync(0xffffffffu, s.q0, src);
  r.q_len = __shfl_sync(0xffffffffu, s.q_len, src);
  r.kv_len = __shfl_sync(0xffffffffu, s.kv_len, src);
  r.blocks = __shfl_sync(0xffffffffu, s.blocks, src);
  return r;
}

// An item in the list of all items (sequences, their heads, their blocks) and
// the cost of all items before it.
struct PagedPlace {
  int b, head, i;
  int tiles;
  long long start, cost;
  PagedSeq s;

  // the item's tile at position `pos` of the list
  __device__ __forceinline__ int tile(const PagedParams& p, long long pos) const {
    const long long x = pos - start - p.item_keys;
    if (x <= 0) return 0;
    if (pos >= start + cost) return tiles;
    return min(tiles, key_tiles_of(static_cast<int>(x)));
  }
  template <int SUBS>
  __device__ __forceinline__ void measure(const PagedParams& p) {
    const int keys = block_keys(p, s, p.sub_tokens * SUBS, i);
    tiles = key_tiles_of(keys);
    cost = p.item_keys + keys;
  }
};

// Lane x: the cost of the blocks of its strip of the sequences, x strip .. (x +
// 1) strip - 1, and the sequence where a strip is one (32 sequences or fewer).
// After a strip's first lines its loads hit the first-level cache.  (Four
// sequences a step made the code longer and every small call slower, by up to
// 3 of 84 us; strips against steps of 32 sequences, read twice: 4096 sequences of
// at most 512 keys 964 -> 842 us.)
struct PagedStrips {
  int strip;
  PagedSeq s;
  long long cost;
};

template <int SUBS>
__device__ __forceinline__ PagedStrips paged_strips(const PagedParams& p) {
  const int lane = threadIdx.x & 31, block = p.sub_tokens * SUBS;
  PagedStrips f;
  f.strip = (p.B + 31) / 32;
  if (f.strip == 1) {
    f.s = paged_seq(p, lane, block);
    f.cost = cost_before<SUBS>(p, f.s, f.s.blocks);
    return f;
  }
  const int end = min(p.B, (lane + 1) * f.strip);
  f.s = {};
  f.cost = 0;
#pragma unroll 1
  for (int b = lane * f.strip; b < end; ++b) {
    const PagedSeq s = paged_seq(p, b, block);
    f.cost += cost_before<SUBS>(p, s, s.blocks);
  }
  return f;
}

// Whole warp: the length of one of p.ctas equal ranges of the list, at least an
// item's fixed cost and one tile, so that an item's inner ranges all have tiles;
// and the length of the list.
template <int SUBS>
__device__ __forceinline__ long long paged_share(const PagedParams& p, const PagedStrips& f, long long* total) {
  const long long sum = warp_sum(f.cost) * p.Hkv;
  *total = sum;
  // total / ctas rounded up (the 64-bit product is off by less than one), so that the ranges cover the list
  const long long share = static_cast<long long>(static_cast<double>(sum) * p.inv_ctas) + 2;
  return max(share, static_cast<long long>(p.min_tiles) * kKeysPerTile + p.item_keys);
}

// Whole warp: the item that position `pos` (below the list's length) lies in.
template <int SUBS>
__device__ __forceinline__ PagedPlace paged_find(const PagedParams& p, const PagedStrips& f, long long pos) {
  const int lane = threadIdx.x & 31;
  PagedPlace w = {};
  long long before = 0;
  int begin = 0, end = p.B;
  if (f.strip > 1) {   // the strip
    const long long mine = f.cost * p.Hkv, sum = warp_scan(mine);
    const unsigned here = __ballot_sync(0xffffffffu, pos >= sum - mine && pos < sum);
    if (here == 0) return w;
    const int src = __ffs(here) - 1;
    before = __shfl_sync(0xffffffffu, sum - mine, src);
    begin = src * f.strip;
    end = min(p.B, begin + f.strip);
  }
  for (int b0 = begin; b0 < end; b0 += 32) {
    const PagedSeq s = f.strip == 1 ? f.s : paged_seq(p, b0 + lane < end ? b0 + lane : p.B, p.sub_tokens * SUBS);
    const long long per_head = f.strip == 1 ? f.cost : cost_before<SUBS>(p, s, s.blocks);
    const long long mine = per_head * p.Hkv, sum = warp_scan(mine) + before;
    const unsigned here = __ballot_sync(0xffffffffu, pos >= sum - mine && pos < sum);
    if (here == 0) {
      before = __shfl_sync(0xffffffffu, sum, 31);
      continue;
    }
    const int src = __ffs(here) - 1;
    w.start = __shfl_sync(0xffffffffu, sum - mine, src);
    const long long each = __shfl_sync(0xffffffffu, per_head, src);
    w.b = b0 + src;
    w.s = seq_from(s, src);
    // heads and blocks that start at or before pos, 32 candidates at a time
    for (int h0 = 0; h0 < p.Hkv; h0 += 32) {
      const unsigned some =
          __ballot_sync(0xffffffffu, h0 + lane < p.Hkv && w.start + (h0 + lane) * each <= pos);
      if (some == 0) break;
      w.head = h0 + 31 - __clz(some);
    }
    w.start += w.head * each;
    int lo = 0, n = w.s.blocks;
    while (n > 1) {
      const int step = (n + 31) / 32;
      const bool below =
          lane * step < n && w.start + cost_before<SUBS>(p, w.s, lo + min(lane * step, n)) <= pos;
      const int last = 31 - __clz(__ballot_sync(0xffffffffu, below));
      n = min(step, n - last * step);
      lo += last * step;
    }
    w.i = lo;
    w.start += cost_before<SUBS>(p, w.s, lo);
    w.measure<SUBS>(p);
    return w;
  }
  return w;
}

__device__ __forceinline__ PagedUnit paged_unit(const PagedParams& p, const PagedSeq& s, int b, int head, int block,
                                                int i) {
  PagedUnit u;
  u.valid = 1;
  u.head = head;
  u.q_len = s.q_len;
  u.kv_len = s.kv_len;
  u.tok0 = i * block;
  u.ntok = min(block, s.q_len - u.tok0);
  u.row0 = s.q0 + u.tok0;
  u.table = b * p.table_stride;
  u.t_begin = u.t_end = 0;
  u.slot = -1;
  return u;
}

// Whole warp: walks the segments of range `cta` (even).  A part that begins inside an
// item goes to slot 2 cta, one that begins it and does not end it to slot 2 cta
// + 1: a range has at most one of each.
struct PagedWalk {
  PagedPlace at;
  long long lo, hi;   // the range
  int cta;

  template <int SUBS>
  __device__ __forceinline__ PagedUnit next(const PagedParams& p) {
    const int lane = threadIdx.x & 31;
    PagedUnit u;
    u.valid = 0;
    while (lo < hi && !u.valid) {
      const int from = at.tile(p, lo), to = at.tile(p, hi);
      if (from < to) {
        u = paged_unit(p, at.s, at.b, at.head, p.sub_tokens * SUBS, at.i);
        u.t_begin = from;
        u.t_end = to;
        if (from > 0)
          u.slot = 2 * cta;
        else if (to < at.tiles)
          u.slot = 2 * cta + 1;
      }
      at.start += at.cost;
      lo = max(lo, at.start);
      if (lo >= hi) break;
      // the next block, head or sequence with new tokens
      if (++at.i == at.s.blocks) {
        at.i = 0;
        if (++at.head == p.Hkv) {
          at.head = 0;
          int b0 = at.b + 1;
          for (; b0 < p.B; b0 += 32) {
            const PagedSeq s = paged_seq(p, b0 + lane, p.sub_tokens * SUBS);
            const unsigned some = __ballot_sync(0xffffffffu, s.blocks > 0);
            if (some != 0) {
              const int src = __ffs(some) - 1;
              at.s = seq_from(s, src);
              at.b = b0 + src;
              break;
            }
          }
          if (b0 >= p.B) {
            lo = hi;
            break;
          }
        }
      }
      at.measure<SUBS>(p);
    }
    return u;
  }
};

template <int SUBS>
__device__ __forceinline__ PagedWalk paged_walk(const PagedParams& p, int cta) {
  PagedWalk w;
  long long total;
  const PagedStrips f = paged_strips<SUBS>(p);
  const long long share = paged_share<SUBS>(p, f, &total);
  w.cta = cta;
  w.lo = cta * share;
  w.hi = cta < p.ctas ? min(w.lo + share, total) : w.lo;
  if (w.lo < w.hi) w.at = paged_find<SUBS>(p, f, w.lo);
  return w;
}

// Parts of an item that the merge reads: the first in slot `first`, the others
// in `rest`, `rest` + step, ...
struct PagedParts {
  PagedUnit u;
  int parts, first, rest, step;
};

// Whole warp: the item that the boundary between the ranges `index` and `index`
// + 1 cuts, when it is the first boundary to do so; otherwise u.valid = 0.
template <int SUBS>
__device__ __forceinline__ PagedParts paged_parts_even(const PagedParams& p, int index) {
  PagedParts r;
  r.u.valid = 0;
  long long total;
  const PagedStrips f = paged_strips<SUBS>(p);
  const long long share = paged_share<SUBS>(p, f, &total);
  const long long pos = (index + 1ll) * share;
  if (index + 1 >= p.ctas || pos >= total) return r;
  const PagedPlace w = paged_find<SUBS>(p, f, pos);
  const int t = w.tile(p, pos);
  if (t == 0 || t == w.tiles || w.tile(p, pos - share) > 0) return r;
  r.u = paged_unit(p, w.s, w.b, w.head, p.sub_tokens * SUBS, w.i);
  r.first = 2 * index + 1;
  r.rest = 2 * (index + 1);
  r.step = 2;
  r.parts = 2;
  for (long long next = pos + share; next < total && w.tile(p, next) < w.tiles; next += share) ++r.parts;
  return r;
}

// Whole warp: the page numbers of a sequence's tiles, in ascending order of the
// tiles, 32 table entries at a time (one per lane) and the next 32 on their way.
struct PageCursor {
  const int* table;
  int live;        // table entries that hold keys
  int chunk0;      // first entry in `pages`
  int pages, pages_next;

  __device__ __forceinline__ PageCursor(const PagedParams& p, const PagedUnit& w, int tiles) {
    table = p.page_table + (tiles > 0 ? w.table : 0);
    live = tiles > 0 ? (w.kv_len + (1 << p.page_log2) - 1) >> p.page_log2 : 0;
    chunk0 = tiles > 0 ? (w.t_begin << 7) >> p.page_log2 : 0;
    pages = fetch(p, chunk0);
    pages_next = fetch(p, chunk0 + 32);
  }
  __device__ __forceinline__ int fetch(const PagedParams& p, int first) const {
    const int i = first + (threadIdx.x & 31);
    int id = 0;
    if (i < live) {
      id = table[i];
      if (id < 0 || id >= p.num_pages) atomicOr(p.status, kDevErrPage);
    }
    return id;
  }
  // lane x: the tile's x-th page; *count: how many there are
  __device__ __forceinline__ int tile(const PagedParams& p, int t, int* count) {
    const int first = (t << 7) >> p.page_log2;
    if (first >= chunk0 + 32) {
      chunk0 += 32;
      pages = pages_next;
      pages_next = fetch(p, chunk0 + 32);
    }
    *count = min(kKeysPerTile >> min(p.page_log2, 7), live - first);
    return __shfl_sync(0xffffffffu, pages, (first - chunk0 + (threadIdx.x & 31)) & 31);
  }
};

// Bytes of one head's K and V that a group of heads may hold in L2 together.
constexpr long long kPagedL2Bytes = 64ll << 20;

// Whole warp, items from a counter: unit `index` (items = false), or the item of
// rank `index` among those cut into several units (items = true; its parts are
// in slots first, first + 1, ...).
template <int SUBS>
__device__ __forceinline__ PagedParts paged_item(const PagedParams& p, int index, bool items, int D) {
  const int lane = threadIdx.x & 31;
  const int block = p.sub_tokens * SUBS;
  long long total = 0;
  for (int b = lane; b < p.B; b += 32) {
    const PagedSeq s = paged_seq(p, b, block);
    total += static_cast<long long>(s.blocks) * key_tiles_of(s.kv_len);
  }
  total = warp_sum(total) * p.Hkv;
  const int per_unit = static_cast<int>(
      min(max((total + p.ctas - 1) / p.ctas, static_cast<long long>(p.min_tiles)), 1ll << 24));   // more than any length

  PagedParts r;
  r.u.valid = 0;
  r.step = 1;
  int before = 0, slots_before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const PagedSeq q = paged_seq(p, b0 + lane, block);
    const int tiles = key_tiles_of(q.kv_len);
    const int s = max(1, (tiles + per_unit - 1) / per_unit);
    const int blocks = q.blocks * p.Hkv;
    const int slots = s > 1 ? blocks * s : 0;
    const int count = items ? (s > 1 ? blocks : 0) : blocks * s;
    const int sum = static_cast<int>(warp_scan(count)), slot_sum = static_cast<int>(warp_scan(slots));
    const int at = index - before;
    const unsigned here = __ballot_sync(0xffffffffu, at >= sum - count && at < sum);
    if (here != 0) {
      const int src = __ffs(here) - 1;
      auto get = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
      const int splits = get(s), all_tiles = get(tiles);
      const PagedSeq seq = seq_from(q, src);
      int in = at - get(sum - count);
      if (items) in *= splits;
      const int slot = slots_before + get(slot_sum - slots) + in;
      // Units of a sequence: groups of heads whose K and V fit in L2 together;
      // within a group the last query blocks (the longest under the causal
      // mask) first, all heads of the group for one block, then the next.
      const long long kv_bytes = static_cast<long long>(max(seq.kv_len, 1)) * D * 4;
      const int hg = static_cast<int>(min(max(kPagedL2Bytes / kv_bytes, 1ll), static_cast<long long>(p.Hkv)));
      const int per_group = hg * seq.blocks * splits;
      const int group = in / per_group;
      in -= group * per_group;
      const int per_block = min(hg, p.Hkv - group * hg) * splits;
      const int rank = in / per_block;
      in -= rank * per_block;
      const int h = in / splits, split = in - h * splits;
      r.u = paged_unit(p, seq, b0 + src, group * hg + h, block, seq.blocks - 1 - rank);
      r.u.t_begin = split * per_unit;
      r.u.t_end = min(all_tiles, r.u.t_begin + per_unit);
      if (splits > 1) r.u.slot = slot;
      r.parts = splits;
      r.first = slot;
      r.rest = slot + 1;
      return r;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
    slots_before += __shfl_sync(0xffffffffu, slot_sum, 31);
  }
  return r;
}

template <int N>
using Int = std::integral_constant<int, N>;

// Named barrier of the segments (kBarP0 and kBarP1 are the dense kernel's).
constexpr int kBarSegment = 3;
constexpr int kBarShares = 4;      // the softmax warps, while they merge their shares
constexpr int kBarProducers = 5;   // the producers, at a segment's description

template <int D, int SUBS>
struct PagedConfig : FwdConfig<D, SUBS> {
  using Base = FwdConfig<D, SUBS>;
  // Epilogue staging: 64 bytes of each of a warp's 32 rows (Q's buffer already
  // takes the next segment's queries by then).
  static constexpr uint32_t kStageBytes = 32 * 64;
  static constexpr uint32_t kSmemStage = Base::kSmemData;
  static constexpr uint32_t kSmemBars = Base::kSmemData + 4 * SUBS * kStageBytes;
  static constexpr uint32_t kSmemBytes = kSmemBars + 1024 /*align*/ + 2048 /*barriers, shares*/;
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static_assert(SUBS == 2 || D == 256 || 2 * (kSmemBytes + 1024) <= 233472, "two CTAs per SM");
  // Registers per thread after the start: the producer warp walks the schedule
  // in 64 bits and needs more than the dense kernel's.
  static constexpr int kSoftmax = SUBS == 2 ? 216 : 184;
  static constexpr int kProducer = 72;
  static_assert(SUBS * 128 * kSoftmax + 128 * kProducer <= FwdShape<SUBS>::kLaunch * FwdShape<SUBS>::kThreads,
                "register rebalancing exceeds the launch allocation");
  // Producer warps, each with its 64-column chunks of every K and V tile.
  static constexpr bool kThree = D == 256, kTwo = D == 128 && SUBS == 2;
  static constexpr int kProducers = kThree ? 3 : kTwo ? 2 : 1;
  // softmax, first producer and MMA warps, and the watcher where there is one
  static constexpr int kSegmentThreads = SUBS * 128 + 64 + (Base::kNamedP ? 32 : 0);
};

template <int STAGES>
struct alignas(8) PagedShared {
  FwdBarriers<STAGES> bars;
  uint64_t q_empty;
  PagedUnit unit[2];   // segment k in unit[k % 2]
  float2 shares[4][32];   // NARROW: (m, l) of the warps' rows
};

// F16: Q, K, V (and P) are fp16 instead of bf16.  SUBS: sub-tiles per CTA, as
// in the dense kernel (2: one CTA per SM, for blocks of more than 128 rows).
//
// Counters that run on over a CTA's segments: `base` K/V copies (two per key
// tile, in order K, V), `done[sub]` tiles of a sub-tile, `loads` segments that
// loaded Q.  A barrier's phase is taken from them.
template <int D, bool F16, int SUBS, bool NARROW>
__global__ void __launch_bounds__(FwdShape<SUBS>::kThreads, FwdShape<SUBS>::kCtasPerSm)
    fa2_paged_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedParams p) {
  using Cfg = PagedConfig<D, SUBS>;
  constexpr int kWarpProducer = 4 * SUBS;      // schedule and copies
  constexpr int kWarpMma = 4 * SUBS + 1;       // MMA warp, owns the TMEM allocation
  constexpr int kWarpWatch = 4 * SUBS + 2;     // K/V watcher (named-barrier variants)
  constexpr int STAGES = Cfg::kStages;
  constexpr uint32_t TILE = Cfg::kTileBytes;
  constexpr int NCH = Cfg::kChunks;
  constexpr uint32_t kChunkBytes = kRowsPerSub * 128;  // one 64-column chunk of a 128-row tile
  static_assert(sizeof(PagedShared<STAGES>) <= 2048, "barrier page");
  static_assert(!NARROW || SUBS == 1, "narrow blocks have one sub-tile");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;                  // SUBS sub-tiles
  uint8_t* sKV = smem + SUBS * TILE;   // STAGES tiles
  auto* shared = reinterpret_cast<PagedShared<STAGES>*>(smem + Cfg::kSmemBars);
  auto* bars = &shared->bars;
  volatile int* abort = &bars->abort;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // key tiles that sub-tile `sub` of unit w visits
  auto tiles_for = [&](const PagedUnit& w, int sub) {
    const int first = sub * p.sub_tokens;
    if (first >= w.ntok) return 0;
    const int last = min(first + p.sub_tokens, w.ntok) - 1;
    const int kept = paged_kept(p.causal, w.kv_len, w.q_len, w.tok0 + last);
    return max(0, min(w.t_end, key_tiles_of(kept)) - w.t_begin);
  };

  // ---- the producers' copies; whole warps, `ok` is cleared after an abort
  auto warp_wait = [&](uint64_t* bar, int phase, bool& ok) {
    if (!ok) return;
    ok = __all_sync(0xffffffffu, wait_bar(bar, phase, abort, p.timeout_ns));
    if (!ok && lane == 0) raise_abort(abort, p.status);
  };
  // Chunks C0 .. C1 - 1 of copy `index` into the ring: K (even) or V (odd) of the
  // key tile `tile`, which lies at or behind the cursor.  Everything is ready
  // before the wait for the slot: instructions after it delay every tile.
  int last[2] = {-1, -1};   // this warp's last copies of K and of V
  auto copy = [&](auto C0, auto C1, const PagedUnit& w, PageCursor& pages, int tile, int index, bool& ok) {
    constexpr int kFirst = decltype(C0)::value, kEnd = decltype(C1)::value;
    const int slot = index % STAGES, lap = index / STAGES;
    const int slots_log2 = min(p.page_log2, 7);   // slots of a page that the tile reads
    int count;
    const int id = pages.tile(p, tile, &count);
    const CUtensorMap* map = (index & 1) == 0 ? &tm_k : &tm_v;
    const int row = (tile << 7) & ((1 << p.page_log2) - 1);
    uint8_t* dst = sKV + slot * TILE + (static_cast<uint32_t>(lane) << slots_log2) * 128;
    const uint32_t bytes = static_cast<uint32_t>(count * (kEnd - kFirst)) * (128u << slots_log2);
    if (lap > 0) warp_wait(&bars->kv_empty[slot], (lap - 1) & 1, ok);
    if (!ok) return;
    if (lane == 0) bar_arrive_expect_tx(&bars->kv_full[slot], bytes);
    __syncwarp();
    if (lane < count) {
#pragma unroll
      for (int c = kFirst; c < kEnd; ++c)
        tma_load_4d(dst + c * kChunkBytes, map, &bars->kv_full[slot], c * 64, row, w.head, id);
    }
    __syncwarp();
    last[index & 1] = index;
  };
  // Three producers: their chunks of K and of V.  In the order of the MMAs: K(j+1),
  // whose slot S(j) frees, then V(j), whose slot P(j-1) V frees.
  auto copy_three = [&](auto K0, auto K1, auto V0, auto V1, const PagedUnit& w, int n, int tiles, PageCursor& k_pages,
                        PageCursor& v_pages, int first, bool& ok) {
    for (int j = first; j <= n && ok; ++j) {
      if (j < n) copy(K0, K1, w, k_pages, w.t_begin + j, 2 * (tiles + j), ok);
      if (j > 0 && ok) copy(V0, V1, w, v_pages, w.t_begin + j - 1, 2 * (tiles + j) - 1, ok);
    }
  };
  // Before the CTA may exit, the copies of a producer must have landed: the last
  // STAGES, where it made them all, else the last of K and of V (a two-slot ring).
  auto drain = [&]() {
    if (lane != 0) return;
    volatile int never = 0;
    const int end = max(last[0], last[1]);
    for (int i = max(0, end - STAGES + 1); i <= end; ++i)
      if (!Cfg::kThree || i == last[i & 1])
        wait_bar(&bars->kv_full[i % STAGES], (i / STAGES) & 1, &never, p.timeout_ns);
  };
  static_assert(!Cfg::kThree || STAGES == 2, "a slot each for K and V");

  if (warp == kWarpProducer && lane == 0) {
    bar_init(&bars->q_full, 1);
    bar_init(&shared->q_empty, 1);
    for (int s = 0; s < STAGES; ++s) {
      bar_init(&bars->kv_full[s], Cfg::kProducers);
      bar_init(&bars->kv_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&bars->s_full[i], 1);
      bar_init(&bars->p_ready[i], kRowsPerSub);
      bar_init(&bars->o_done[i], 1);
    }
    bar_init(&bars->mma_drain, 1);
    bars->abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == kWarpMma) {
    tmem_alloc(&bars->tmem_base, Cfg::kTmemCols);
    tmem_relinquish();
    tc_fence_before_sync();
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;

  // The grid before this one is complete from here on; behind that, the merge may
  // start (it finds its items and then waits for this grid to end).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp >= kWarpProducer) {
    regs_decrease<Cfg::kProducer>();
    if (warp == kWarpProducer) {
      // ------------------------------------------------------------ schedule and copies
      constexpr int kMine = Cfg::kThree ? 2 : Cfg::kTwo ? 1 : NCH;   // chunks of K that this warp copies
      PagedWalk walk;
      bool begun = false;
      auto next_unit = [&]() {
        if (NARROW || p.even) return walk.next<SUBS>(p);   // (narrow blocks always have equal ranges)
        int index = blockIdx.x;   // the first unit by number, the others as CTAs become free
        if (begun) {
          if (lane == 0) index = gridDim.x + atomicAdd(p.counter, 1);
          index = __shfl_sync(0xffffffffu, index, 0);
        }
        begun = true;
        return paged_item<SUBS>(p, index, false, D).u;
      };
      if (NARROW || p.even) walk = paged_walk<SUBS>(p, static_cast<int>(blockIdx.x));
      PagedUnit w = next_unit();
      int tiles = 0, loads = 0;   // tiles of the segments before; Q loads
      bool ok = true;
      for (int k = 0;; ++k) {
        if (lane == 0) shared->unit[k & 1] = w;
        __syncwarp();
        if (Cfg::kProducers > 1) named_sync(kBarProducers, Cfg::kProducers * 32);
        int n = 0;
        if (w.valid) {
          n = tiles_for(w, 0);
          if (SUBS == 2) n = max(n, tiles_for(w, 1));
        }
        PageCursor pages(p, w, n);
        // Ahead of the hand-over: the first copies, which do not wait for the
        // last V of the segment before (its slot comes STAGES - 1 copies
        // later), and Q, once the last S of the segment before is complete.
        // (The first segment is handed over at once.)
        const int early = k == 0 ? min(1, n) : min(STAGES - 1, 2 * n);
        for (int i = 0; i < early; ++i) {
          copy(Int<0>{}, Int<kMine>{}, w, pages, w.t_begin + (i >> 1), 2 * tiles + i, ok);
          if (i == 0) {
            if (loads > 0) warp_wait(&shared->q_empty, (loads - 1) & 1, ok);
            if (ok) {
              // Q boxes of the live tokens, a box per lane
              const uint32_t box_bytes = static_cast<uint32_t>(p.box_tokens) * p.G * 128;
              const int per_sub = p.sub_tokens / p.box_tokens;
              const int boxes = (w.ntok + p.box_tokens - 1) / p.box_tokens;
              constexpr int kCopies = NARROW ? 4 : 1;   // one in each warp's rows
              if (lane == 0)
                bar_arrive_expect_tx(&bars->q_full, static_cast<uint32_t>(boxes) * kCopies * NCH * box_bytes);
              __syncwarp();
              for (int y = lane; y < boxes * kCopies; y += 32) {
                const int x = y / kCopies, part = y % kCopies;
                const int sub = x / per_sub;
                uint8_t* dst = sQ + sub * TILE + (x - sub * per_sub) * box_bytes + part * (32 * 128);
                for (int c = 0; c < NCH; ++c)
                  tma_load_3d(dst + c * kChunkBytes, &tm_q, &bars->q_full, c * 64, w.head * p.G,
                              w.row0 + x * p.box_tokens);
              }
              __syncwarp();
              ++loads;
            }
          }
        }
        named_sync(kBarSegment, Cfg::kSegmentThreads);
        if (!w.valid) break;
        if constexpr (Cfg::kThree) {
          PageCursor v_pages(p, w, n);
          copy_three(Int<0>{}, Int<2>{}, Int<0>{}, Int<1>{}, w, n, tiles, pages, v_pages, 1, ok);
        } else {
          for (int i = early; i < 2 * n && ok; ++i)
            copy(Int<0>{}, Int<kMine>{}, w, pages, w.t_begin + (i >> 1), 2 * tiles + i, ok);
        }
        tiles += n;
        w = next_unit();
      }
      if (lane == 0 && loads > 0) {
        volatile int never = 0;
        wait_bar(&bars->q_full, (loads - 1) & 1, &never, p.timeout_ns);
      }
      drain();
      __syncwarp();
    } else if (Cfg::kThree ? warp != kWarpMma : Cfg::kTwo && warp == kWarpWatch + 1) {
      // ------------------------------------------------------------ the other producers
      int tiles = 0;
      bool ok = true;
      for (int k = 0;; ++k) {
        named_sync(kBarProducers, Cfg::kProducers * 32);
        const PagedUnit w = shared->unit[k & 1];
        if (!w.valid) break;
        int n = tiles_for(w, 0);
        if (SUBS == 2) n = max(n, tiles_for(w, 1));
        PageCursor pages(p, w, n);
        if constexpr (Cfg::kThree) {
          PageCursor v_pages(p, w, n);
          if (warp == kWarpMma + 1)
            copy_three(Int<2>{}, Int<3>{}, Int<1>{}, Int<3>{}, w, n, tiles, pages, v_pages, 0, ok);
          else
            copy_three(Int<3>{}, Int<4>{}, Int<3>{}, Int<4>{}, w, n, tiles, pages, v_pages, 0, ok);
        } else {
          for (int i = 0; i < 2 * n && ok; ++i)
            copy(Int<1>{}, Int<NCH>{}, w, pages, w.t_begin + (i >> 1), 2 * tiles + i, ok);
        }
        tiles += n;
      }
      drain();
      __syncwarp();
    } else if (warp == kWarpWatch && Cfg::kNamedP) {
      // ------------------------------------------------------------ K/V watcher
      // After an abort the waits are skipped, not the phases.
      bool ok = true;
      int base = 0;
      for (int k = 0;; ++k) {
        named_sync(kBarSegment, Cfg::kSegmentThreads);
        const PagedUnit& w = shared->unit[k & 1];
        if (!w.valid) break;
        const int n0 = tiles_for(w, 0), nmax = SUBS == 2 ? max(n0, tiles_for(w, 1)) : n0;
        for (int j = 0; j < nmax; ++j) {
          if (lane == 0 && ok) {
            const int iv = base + 2 * j + 1, ik = iv + 1;
            ok = wait_bar(&bars->kv_full[iv % STAGES], (iv / STAGES) & 1, abort, p.timeout_ns);
            if (ok && j + 1 < nmax)
              ok = wait_bar(&bars->kv_full[ik % STAGES], (ik / STAGES) & 1, abort, p.timeout_ns);
            if (!ok) raise_abort(abort, p.status);
          }
          __syncwarp();
          named_sync(kBarP0, j < n0 ? kBarP0Count : kBarP0Idle);
        }
        base += 2 * nmax;
      }
    } else if (warp == kWarpMma) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t kIdescS = idesc_f32acc(kRowsPerSub, kKeysPerTile, false, false, F16);
      constexpr uint32_t kIdescO = idesc_f32acc(kRowsPerSub, D, false, true, F16);
      const uint32_t sQaddr = smem_addr(sQ);
      const uint32_t sKVaddr = smem_addr(sKV);
      // S = Q_sub K^T into S buffer `buf`
      auto issue_s = [&](int sub, int slot, int buf) {
        const uint64_t da = sdesc_sw128(sQaddr + sub * TILE, 16, 1024);
        const uint64_t db = sdesc_sw128(sKVaddr + slot * TILE, 16, 1024);
        uint32_t a_lo = static_cast<uint32_t>(da), b_lo = static_cast<uint32_t>(db);
        const uint32_t a_hi = static_cast<uint32_t>(da >> 32), b_hi = static_cast<uint32_t>(db >> 32);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          mma_ss_halves(tmem + buf * 128, a_lo, a_hi, b_lo, b_hi, kIdescS, kk > 0 ? 1u : 0u);
          const uint32_t step = ((kk & 3) == 3 ? kChunkBytes - 3 * 32 : 32) >> 4;
          a_lo += step;
          b_lo += step;
          asm volatile("" : "+r"(a_lo), "+r"(b_lo));
        }
      };
      // O_sub (+)= P V, P in S buffer `buf`
      auto issue_pv = [&](int sub, int slot, bool acc, int buf) {
        const uint64_t dv = sdesc_sw128(sKVaddr + slot * TILE, kChunkBytes, 1024);
        uint32_t v_lo = static_cast<uint32_t>(dv);
        const uint32_t v_hi = static_cast<uint32_t>(dv >> 32);
        const uint32_t o = tmem + (sub == 0 ? Cfg::kColsO0 : Cfg::kColsO1);
        const uint32_t a = tmem + buf * 128;
#pragma unroll
        for (int kk = 0; kk < kKeysPerTile / 16; ++kk) {
          mma_ts_halves(o, a + kk * 8, v_lo, v_hi, kIdescO, (acc || kk > 0) ? 1u : 0u);
          v_lo += (16 * 128) >> 4;
          asm volatile("" : "+r"(v_lo));
        }
      };
      bool ok = true;
      int base = 0, done0 = 0, loads = 0;
      for (int k = 0;; ++k) {
        named_sync(kBarSegment, Cfg::kSegmentThreads);
        const PagedUnit& w = shared->unit[k & 1];
        if (!w.valid) break;
        const int n0 = tiles_for(w, 0), n1 = SUBS == 2 ? tiles_for(w, 1) : 0, nmax = max(n0, n1);
        if (nmax == 0) continue;
        if (lane == 0 && ok) {
          ok = wait_bar(&bars->q_full, loads & 1, abort, p.timeout_ns) &&
               wait_bar(&bars->kv_full[base % STAGES], (base / STAGES) & 1, abort, p.timeout_ns);
          if (!ok) raise_abort(abort, p.status);
        }
        ++loads;
        if (lane == 0 && (ok || Cfg::kNamedP)) {
          tc_fence_after_sync();
          if (n0 > 0) {
            const int buf = Cfg::kDoubleS ? done0 & 1 : 0;
            issue_s(0, base % STAGES, buf);
            mma_commit(&bars->s_full[buf]);
          }
          if (n1 > 0) { issue_s(1, base % STAGES, 1); mma_commit(&bars->s_full[1]); }
          if (!Cfg::kSoftmaxRelease) mma_commit(&bars->kv_empty[base % STAGES]);
          if (nmax == 1) mma_commit(&shared->q_empty);
        }
        __syncwarp();
        if constexpr (Cfg::kNamedP) {
          // Named barriers: every phase is passed, also after an abort (the
          // MMAs then still go out, on whatever the buffers hold).
          for (int j = 0; j < nmax; ++j) {
            const int slot_v = (base + 2 * j + 1) % STAGES, slot_k = (base + 2 * j + 2) % STAGES;
            named_sync(kBarP0, j < n0 ? kBarP0Count : kBarP0Idle);   // P_0(j); V_j, K_(j+1) landed
            if (lane == 0) {
              tc_fence_after_sync();
              if (j < n0) {
                issue_pv(0, slot_v, j > 0, 0);
                if (j + 1 == n0) mma_commit(&bars->o_done[0]);
              }
              if (j + 1 < n0) { issue_s(0, slot_k, 0); mma_commit(&bars->s_full[0]); }
            }
            __syncwarp();
            if (j < n1) {
              named_sync(kBarP1, kBarP1Count);                      // P_1(j)
              if (lane == 0) {
                tc_fence_after_sync();
                issue_pv(1, slot_v, j > 0, 1);
                if (j + 1 == n1) mma_commit(&bars->o_done[1]);
                if (j + 1 < n1) { issue_s(1, slot_k, 1); mma_commit(&bars->s_full[1]); }
              }
            }
            if (lane == 0 && j + 2 == nmax) mma_commit(&shared->q_empty);   // after the last S
            __syncwarp();
          }
        } else if (lane == 0 && ok) {
          static_assert(Cfg::kNamedP || SUBS == 1, "polled order: one sub-tile");
          for (int j = 0; j < n0; ++j) {
            const int g = done0 + j;   // tile count over all segments
            const int iv = base + 2 * j + 1, ik = iv + 1;
            const int slot_v = iv % STAGES, slot_k = ik % STAGES;
            uint64_t* bv = &bars->kv_full[slot_v];
            const uint32_t pv = (iv / STAGES) & 1;
            auto next_s = [&](int buf) {   // S(j+1)
              ok = wait_bar(&bars->kv_full[slot_k], (ik / STAGES) & 1, abort, p.timeout_ns);
              if (!ok) return;
              tc_fence_after_sync();
              issue_s(0, slot_k, buf);
              mma_commit(&bars->s_full[buf]);
              mma_commit(&bars->kv_empty[slot_k]);
              if (j + 2 == n0) mma_commit(&shared->q_empty);
            };
            // double-buffered: S(j+1) into the other buffer ahead of P(j) V
            const int buf = Cfg::kDoubleS ? g & 1 : 0;
            if (Cfg::kDoubleS && j + 1 < n0) next_s(buf ^ 1);
            ok = ok && wait_bar3(bv, pv, &bars->p_ready[buf], Cfg::kDoubleS ? (g >> 1) & 1 : g & 1, bv, pv, abort,
                                 p.timeout_ns);
            if (!ok) break;
            tc_fence_after_sync();
            issue_pv(0, slot_v, j > 0, buf);
            if (!Cfg::kOutDoneLast || j + 1 == n0) mma_commit(&bars->o_done[0]);
            mma_commit(&bars->kv_empty[slot_v]);
            if (!Cfg::kDoubleS && j + 1 < n0) next_s(0);
            if (!ok) break;
          }
          if (!ok) raise_abort(abort, p.status);
        }
        __syncwarp();
        base += 2 * nmax;
        done0 += n0;
      }
      if (lane == 0) {
        // Every MMA must be complete before TMEM is released.
        mma_commit(&bars->mma_drain);
        volatile int never = 0;
        wait_bar(&bars->mma_drain, 0, &never, p.timeout_ns);
      }
      __syncwarp();
    }
  } else {
    regs_increase<Cfg::kSoftmax>();
    // ------------------------------------------------------------ softmax
    const int sub = warp >> 2;
    const int wq = warp & 3;
    // TMEM lane wq * 32 + lane is row `row` of the sub-tile
    const int row = NARROW ? lane : wq * 32 + lane;
    const int sub_tok0 = sub * p.sub_tokens;
    const int tok = row / p.G;                            // token of the sub-tile
    const uint32_t lane_bits = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS0 = tmem + lane_bits + sub * 128;
    const uint32_t tO = tmem + lane_bits + (sub == 0 ? Cfg::kColsO0 : Cfg::kColsO1);
    const float sl2 = p.scale_log2;
    bool ok = true;
    int base = 0, done = 0, outs = 0;   // outs: segments in which this sub-tile had tiles
    for (int k = 0;; ++k) {
      named_sync(kBarSegment, Cfg::kSegmentThreads);
      const PagedUnit& w = shared->unit[k & 1];
      if (!w.valid) break;
      const int n0 = tiles_for(w, 0), n1 = SUBS == 2 ? tiles_for(w, 1) : 0, nmax = max(n0, n1);
      const int n_tiles = sub == 0 ? n0 : n1;
      const int rows = max(0, min(p.sub_tokens, w.ntok - sub_tok0)) * p.G;   // live rows
      const bool live = row < rows;
      const bool warp_live = NARROW || wq * 32 < rows;
      const int kv_len = w.kv_len, t_begin = w.t_begin;
      const int lim = live ? paged_kept(p.causal, kv_len, w.q_len, w.tok0 + sub_tok0 + tok) : 0;
      // every live row keeps at least the first token's keys
      const int lim_min = paged_kept(p.causal, kv_len, w.q_len, w.tok0 + sub_tok0);

      // One thread of the sub-tile that visits every key tile releases the ring slots.
      const bool releaser = (threadIdx.x & (kRowsPerSub - 1)) == 0 && n_tiles == nmax && n_tiles > 0 &&
                            (sub == SUBS - 1 || n1 == 0);
      float m = -INFINITY;
      float l = 0.f;
      int announced = 0;
      for (int j = 0; j < n_tiles && ok; ++j) {
        const int g = done + j;
        uint64_t* sbar = &bars->s_full[Cfg::kDoubleS ? (g & 1) : sub];
        const uint32_t s_phase = Cfg::kDoubleS ? (g >> 1) & 1 : g & 1;
        const uint32_t tS = Cfg::kDoubleS ? tS0 + (g & 1) * 128 : tS0;
        if (!__all_sync(0xffffffffu, wait_bar(sbar, s_phase, abort, p.timeout_ns))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        if (Cfg::kSoftmaxRelease && releaser) {
          if (j > 0) bar_arrive(&bars->kv_empty[(base + 2 * j - 1) % STAGES]);
          bar_arrive(&bars->kv_empty[(base + 2 * j) % STAGES]);
        }
        const int key0 = (t_begin + j) * kKeysPerTile;
        // V rows behind the last key: zeros, written by the first sub-tile that reads them
        if (key0 + kKeysPerTile > kv_len && (sub == 0 || j >= n0)) {
          const int tid = wq * 32 + lane;
          // In the double-buffered order S(j) may complete before V(j-1) has
          // landed, and a wait for V(j) could not tell it from V(j-2) then (the
          // parity is the same): P(j-1) V first.
          const int iv = base + 2 * j + 1;
          bool landed = true;
          if (Cfg::kDoubleS && j > 0) landed = wait_bar(&bars->o_done[sub], (g - 1) & 1, abort, p.timeout_ns);
          landed = landed && wait_bar(&bars->kv_full[iv % STAGES], (iv / STAGES) & 1, abort, p.timeout_ns);
          landed = __all_sync(0xffffffffu, landed);
          if (landed) {
            const uint32_t v_addr = smem_addr(sKV + (iv % STAGES) * TILE);
            const uint32_t keep_bytes = static_cast<uint32_t>(kv_len - key0) * 128;
#pragma unroll
            for (int c = 0; c < NCH; ++c)
              for (uint32_t at = keep_bytes + tid * 16; at < kChunkBytes; at += kRowsPerSub * 16)
                st_shared_v4(v_addr + c * kChunkBytes + at, 0u, 0u, 0u, 0u);
          }
          if (!landed) {
            ok = false;
            break;
          }
          fence_proxy_async_shared();
        }
        if (warp_live) {
          constexpr int kChunks = NARROW ? 1 : 4;   // of 32 keys of the tile that this warp takes
          const int first = key0 + (NARROW ? wq * 32 : 0);
          const uint32_t tMine = tS + (NARROW ? wq * 32 : 0);
          uint32_t s[kChunks][32];
          const bool masked = key0 + kKeysPerTile > lim_min;
          auto load_s = [&]() {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) tmem_ld32(tMine + c * 32, s[c]);
            tmem_ld_wait(s[0]);
#pragma unroll
            for (int c = 1; c < kChunks; ++c) regs_after_wait(s[c]);
            if (masked) {
#pragma unroll
              for (int c = 0; c < kChunks; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (first + c * 32 + e >= lim) s[c][e] = __float_as_uint(-INFINITY);
            }
          };
          // the row max, and the offset moved to it when it exceeds it by more than kRescaleLog2
          float m_new = m;
          float alpha = 1.f;
          auto decide = [&]() {
#define FA2_S(f) __uint_as_float(s[(f) >> 5][(f) & 31])
            float mx8[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) mx8[k] = FA2_S(k);
#pragma unroll
            for (int f = 8; f < kChunks * 32 - 8; f += 16)
#pragma unroll
              for (int k = 0; k < 8; ++k) mx8[k] = fmax3(mx8[k], FA2_S(f + k), FA2_S(f + 8 + k));
#pragma unroll
            for (int k = 0; k < 8; ++k) mx8[k] = fmaxf(mx8[k], FA2_S(kChunks * 32 - 8 + k));
#undef FA2_S
            const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                                   fmaxf(mx8[6], mx8[7]));
            const float m_cand = fmaxf(m, mx * sl2);
            const bool move = m == -INFINITY || m_cand > m + kRescaleLog2;
            m_new = move ? m_cand : m;
            alpha = !move ? 1.f : (m == -INFINITY ? 0.f : ex2_approx(m - m_new));
          };
          uint32_t pk[kChunks][16];
          float rs;
          auto exps = [&]() {
            const float off = m_new == -INFINITY ? 0.f : m_new;
            const float2 c2 = make_float2(sl2, sl2);
            const float2 o2 = make_float2(-off, -off);
            float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                             make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float2 t = __ffma2_rn(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), c2, o2);
                const float2 pe = make_float2(ex2_approx(t.x), ex2_approx(t.y));
                acc[(e >> 1) & 3] = __fadd2_rn(acc[(e >> 1) & 3], pe);
                pk[c][e >> 1] = pack_x2<F16>(pe.x, pe.y);
              }
            }
            const float2 a01 = __fadd2_rn(acc[0], acc[1]);
            const float2 a23 = __fadd2_rn(acc[2], acc[3]);
            const float2 a = __fadd2_rn(a01, a23);
            rs = a.x + a.y;
          };
          // Once the offset is finite the exponentials come first, with the
          // offset as it stands (see the dense kernel); one loop, so that the
          // code, which every cold launch has to fetch, is there once.
          bool decided = __any_sync(0xffffffffu, live && m == -INFINITY);   // take the row max first
          for (;;) {
            load_s();
            if (decided) decide();
            exps();
            if (decided || !__any_sync(0xffffffffu, live && rs > kRescaleBound)) break;
            decided = true;
          }
          if constexpr (NARROW) {
            // P: my keys, zeros for the other warps' (S covers all of P's columns);
            // all loads of S by this warp are complete, the others read other rows
            const uint32_t none[16] = {};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (c == wq)
                tmem_st16(tS + c * 16, pk[0]);
              else
                tmem_st16(tS + c * 16, none);
            }
          } else {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) tmem_st16(tS + c * 16, pk[c]);
          }
          l = l * alpha + rs;
          m = m_new;
          const bool rescale = decided && j > 0 && __any_sync(0xffffffffu, live && alpha != 1.f);
          if (!Cfg::kOutDoneLast && j > 0 && (rescale || j == n_tiles - 1) &&
              !__all_sync(0xffffffffu, wait_bar(&bars->o_done[sub], (g - 1) & 1, abort, p.timeout_ns))) {
            ok = false;
          }
          if (rescale && ok) {
            tc_fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tO + c * 32, o);
            }
          }
          tmem_st_wait();
        }
        tc_fence_before_sync();
        if constexpr (Cfg::kNamedP) {
          __syncwarp();
          named_sync(sub == 0 ? kBarP0 : kBarP1, sub == 0 ? kBarP0Count : kBarP1Count);
        } else {
          bar_arrive(&bars->p_ready[Cfg::kDoubleS ? (g & 1) : sub]);
        }
        announced = j + 1;
      }
      if constexpr (Cfg::kNamedP) {
        // after an abort: the remaining phases, in step with the issuing warp
        __syncwarp();
        for (int j = announced; j < n_tiles; ++j)
          named_sync(sub == 0 ? kBarP0 : kBarP1, sub == 0 ? kBarP0Count : kBarP1Count);
      }

      // Outputs: the item's rows, or this part's rows in its workspace slot.
      const bool part = w.slot >= 0;
      const bool fits = w.slot < p.slots;   // always, but for offsets that contradict each other
      const bool store = live && fits;
      const int in_token = row - tok * p.G;
      const long long prow =
          part ? static_cast<long long>(w.slot) * p.part_rows + sub_tok0 * p.G + row
               : static_cast<long long>(w.row0 + sub_tok0 + tok) * p.Hq + w.head * p.G + in_token;
      float* lse_out = (part ? p.LSE_part : p.LSE) + prow;
      const bool half_out = p.o_half != 0 && !part;
      if (!fits && threadIdx.x == 0) atomicOr(p.status, kDevErrPage);
      if (n_tiles == 0 && store && ok && (!NARROW || wq == 0)) {
        // no kept key: O = 0 and LSE = -inf (a part: LSE alone, the merge skips its O)
        *lse_out = -INFINITY;
        if (!part) {
          uint8_t* o = static_cast<uint8_t*>(p.O) + prow * (half_out ? D * 2 : D * 4);
          for (int c = 0; c < (half_out ? D * 2 : D * 4); c += 16)
            *reinterpret_cast<uint4*>(o + c) = make_uint4(0, 0, 0, 0);
        }
      }
      const uint32_t o_phase = Cfg::kOutDoneLast ? outs & 1 : (done + n_tiles - 1) & 1;
      if constexpr (NARROW) {
        // The four warps' shares of the rows: O = sum_w e_w O_w / sum_w e_w l_w, e_w =
        // 2^(m_w - max m).  512 values of each warp at a time through the staging
        // rows.  Every warp passes every barrier, also after an abort.
        if (n_tiles > 0) {
          if (ok) ok = __all_sync(0xffffffffu, wait_bar(&bars->o_done[0], o_phase, abort, p.timeout_ns));
          tc_fence_after_sync();
          if (ok && Cfg::kSoftmaxRelease && releaser) bar_arrive(&bars->kv_empty[(base + 2 * nmax - 1) % STAGES]);
          shared->shares[wq][lane] = make_float2(m, l);
          named_sync(kBarShares, kRowsPerSub);
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int x = 0; x < 4; ++x) top = fmaxf(top, shared->shares[x][lane].x);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 ml = shared->shares[x][lane];
            sum += ml.y == 0.f ? 0.f : ex2_approx(ml.x - top) * ml.y;   // (a warp without keys has m = -inf, l = 0)
          }
          const float mine = l == 0.f ? 0.f : ex2_approx(m - top) / sum;
          if (store && ok && wq == 0) *lse_out = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
          // per warp 2 KB: 16 rows of 32 columns, or 8 of 64 or 4 of 128
          const uint32_t stage = smem_addr(smem + Cfg::kSmemStage);
          const int wide = D == 64 ? 0 : rows <= 4 ? 2 : rows <= 8 ? 1 : 0;   // log2 of the column blocks of 32 in a pass
          const int out_row = threadIdx.x >> (3 + wide), unit = threadIdx.x & ((8 << wide) - 1);   // what I add up and store
#pragma unroll 1
          for (int c = 0; c < D / 32; c += 1 << wide) {
#pragma unroll 1
            for (int r0 = 0; r0 < rows; r0 += 16) {
              const int slot = lane - r0;
#pragma unroll 1
              for (int x = 0; x < 1 << wide; ++x) {
                uint32_t o[32];
                tmem_ld32(tO + (c + x) * 32, o);
                tmem_ld_wait(o);
                if (slot >= 0 && slot < 16 >> wide) {
#pragma unroll
                  for (int u = 0; u < 8; ++u)
                    st_shared_v4(stage + wq * 2048 + (slot << (7 + wide)) + x * 128 + ((u ^ (slot & 7)) << 4),
                                 __float_as_uint(__uint_as_float(o[4 * u]) * mine),
                                 __float_as_uint(__uint_as_float(o[4 * u + 1]) * mine),
                                 __float_as_uint(__uint_as_float(o[4 * u + 2]) * mine),
                                 __float_as_uint(__uint_as_float(o[4 * u + 3]) * mine));
                }
              }
              named_sync(kBarShares, kRowsPerSub);
              const int r = r0 + out_row;
              if (r < rows && fits && ok) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                const uint32_t from = stage + (out_row << (7 + wide)) + ((unit ^ (out_row & 7)) << 4);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  float4 y;
                  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                               : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w)
                               : "r"(from + x * 2048)
                               : "memory");
                  v.x += y.x;
                  v.y += y.y;
                  v.z += y.z;
                  v.w += y.w;
                }
                const int column = c * 32 + unit * 4, t = r / p.G;
                const long long o_row = static_cast<long long>(w.row0 + t) * p.Hq + w.head * p.G + (r - t * p.G);
                if (part)
                  *reinterpret_cast<float4*>(p.O_part + static_cast<long long>(w.slot) * p.part_rows * D +
                                             (static_cast<long long>(column / 4) * p.part_rows + r) * 4) = v;
                else if (half_out)
                  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.O) + o_row * D + column) =
                      make_uint2(pack_x2<F16>(v.x, v.y), pack_x2<F16>(v.z, v.w));
                else
                  *reinterpret_cast<float4*>(static_cast<float*>(p.O) + o_row * D + column) = v;
              }
              named_sync(kBarShares, kRowsPerSub);
            }
          }
          tc_fence_before_sync();
        }
      } else if (n_tiles > 0 && ok) {
        if (store) *lse_out = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
        if (!__all_sync(0xffffffffu, wait_bar(&bars->o_done[sub], o_phase, abort, p.timeout_ns))) {
          ok = false;
        } else {
          tc_fence_after_sync();
          // the last V of the segment: every MMA that reads it is complete
          if (Cfg::kSoftmaxRelease && releaser) bar_arrive(&bars->kv_empty[(base + 2 * nmax - 1) % STAGES]);
          const float inv_l = l == 0.f ? 0.f : 1.f / l;
          if (part && warp_live) {
            float* dst = p.O_part + static_cast<long long>(w.slot) * p.part_rows * D + (sub_tok0 * p.G + row) * 4;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_ld_wait(o);
              if (store) {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                  *reinterpret_cast<float4*>(dst + static_cast<long long>(c * 8 + e / 4) * p.part_rows * 4) =
                      make_float4(__uint_as_float(o[e]) * inv_l, __uint_as_float(o[e + 1]) * inv_l,
                                  __uint_as_float(o[e + 2]) * inv_l, __uint_as_float(o[e + 3]) * inv_l);
              }
            }
          } else if (warp_live) {
            // O / l, 64 bytes of each row at a time through this warp's staging
            // rows (16-byte units exchanged so that writes touch every bank),
            // so that four lanes store 64 neighbouring bytes of a row.
            const uint32_t stage = smem_addr(smem + Cfg::kSmemStage) + warp * Cfg::kStageBytes;
            const uint32_t mine = stage + lane * 64;
            const int turn = (lane >> 1) & 3;
            uint8_t* out = static_cast<uint8_t*>(p.O);
            const long long my_off = store ? prow * (half_out ? D * 2 : D * 4) : -1;
            const int warp_rows = min(32, rows - wq * 32);
            auto put = [&](int column_bytes, const uint32_t (&v)[16]) {   // 64 bytes of my row
              __syncwarp();
#pragma unroll
              for (int u = 0; u < 4; ++u)
                st_shared_v4(mine + ((u ^ turn) << 4), v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                if (i >= warp_rows) break;
                const int rr = i + (lane >> 2), unit = lane & 3;
                const long long off = __shfl_sync(0xffffffffu, my_off, rr);
                uint32_t x[4];
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                             : "r"(stage + rr * 64 + ((unit ^ ((rr >> 1) & 3)) << 4))
                             : "memory");
                if (off >= 0)
                  *reinterpret_cast<uint4*>(out + off + column_bytes + unit * 16) = make_uint4(x[0], x[1], x[2], x[3]);
              }
            };
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_ld_wait(o);
              uint32_t v[16];
              if (half_out) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  v[e] = pack_x2<F16>(__uint_as_float(o[2 * e]) * inv_l, __uint_as_float(o[2 * e + 1]) * inv_l);
                put(c * 64, v);
              } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                  for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(o[16 * h + e]) * inv_l);
                  put(c * 128 + h * 64, v);
                }
              }
            }
          }
          tc_fence_before_sync();
        }
      }
      if (n_tiles > 0) ++outs;
      done += n_tiles;
      base += 2 * nmax;
      if (!ok) raise_abort(abort, p.status);
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

constexpr int kPagedMergeWarps = 4;
constexpr int kPagedMergeRows = 8;    // rows of a warp
constexpr int kPagedMergeMany = 6;    // parts from which the warps of a block share one row group's parts

// Merge of the parts of cut items: blockIdx.x names an item, the blocks of a
// column share its rows, eight rows a warp: lane = (row, 4 of 16 columns), so
// that reads are 128 and writes 32 neighbouring bytes at least.  With m = max_s
// L_s and w_s = exp(L_s - m): O = sum_s w_s O_s / sum w_s, LSE = m + log sum w_s;
// parts with L_s = -inf have w_s = 0 and their O is not used.  An item of many
// parts has few rows (it was cut because there were few items): its block's
// warps take every fourth part each and add up through shared memory.
template <int D, bool F16, int SUBS>
__global__ void __launch_bounds__(kPagedMergeWarps * 32) fa2_paged_merge_kernel(const __grid_constant__ PagedParams p) {
  __shared__ float4 sums[kPagedMergeWarps - 1][D / 16][32];
  __shared__ float2 weights[kPagedMergeWarps - 1][32];
  const int index = static_cast<int>(blockIdx.x);
  const PagedParts w = p.even ? paged_parts_even<SUBS>(p, index) : paged_item<SUBS>(p, index, true, D);
  // launched while the partial results are computed: they are complete from here on
  // (what was read above the kernel before this one does not write, and that one lets
  // this one start behind its own wait for what came before it)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!w.u.valid || w.first < 0 || w.first >= p.slots || w.rest + (w.parts - 2) * w.step >= p.slots) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = w.u.ntok * p.G;
  const bool share = w.parts >= kPagedMergeMany;
  const int first = share ? warp : 0, step = share ? kPagedMergeWarps : 1;
  const int groups = share ? 1 : kPagedMergeWarps;   // row groups of the block
  for (int g0 = blockIdx.y * groups; g0 * kPagedMergeRows < rows; g0 += groups * gridDim.y) {
    const int row = (g0 + (share ? 0 : warp)) * kPagedMergeRows + (lane & 7), group = lane >> 3;
    const bool live = row < rows;
    auto slot = [&](int s) { return static_cast<long long>(s == 0 ? w.first : w.rest + (s - 1) * w.step); };
    // One pass, the parts' loads independent of each other: m is the running
    // maximum, sums are scaled when it moves.
    const float* L = p.LSE_part + (live ? row : 0);
    const float* O = p.O_part + static_cast<long long>(group) * p.part_rows * 4 + (live ? row : 0) * 4;
    float4 acc[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f, m = -INFINITY;
#pragma unroll 2
    for (int s = first; s < w.parts; s += step) {
      const long long at = slot(s) * p.part_rows;
      const float ls = L[at];
      float4 x[D / 16];
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        x[c] = *reinterpret_cast<const float4*>(O + at * D + static_cast<long long>(c) * 16 * p.part_rows);
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
    if (share) {
      __syncthreads();   // the last row group's sums are read
      if (warp > 0) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) sums[warp - 1][c][lane] = acc[c];
        weights[warp - 1][lane] = make_float2(m, sum);
      }
      __syncthreads();
      if (warp > 0) continue;
#pragma unroll
      for (int x = 0; x < kPagedMergeWarps - 1; ++x) {
        const float2 other = weights[x][lane];
        const float top = fmaxf(m, other.x);
        const float keep = m == -INFINITY ? 0.f : expf(m - top), e = other.x == -INFINITY ? 0.f : expf(other.x - top);
        m = top;
        sum = fmaf(sum, keep, e * other.y);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const float4 y = sums[x][c][lane];
          acc[c].x = fmaf(acc[c].x, keep, e * y.x);
          acc[c].y = fmaf(acc[c].y, keep, e * y.y);
          acc[c].z = fmaf(acc[c].z, keep, e * y.z);
          acc[c].w = fmaf(acc[c].w, keep, e * y.w);
        }
      }
    }
    if (!live) continue;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int tok = row / p.G;
    const long long out = static_cast<long long>(w.u.row0 + tok) * p.Hq + w.u.head * p.G + (row - tok * p.G);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const long long at = out * D + c * 16 + group * 4;
      const float4 x = make_float4(acc[c].x * inv, acc[c].y * inv, acc[c].z * inv, acc[c].w * inv);
      if (p.o_half)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.O) + at) =
            make_uint2(pack_x2<F16>(x.x, x.y), pack_x2<F16>(x.z, x.w));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(p.O) + at) = x;
    }
    if (group == 0) p.LSE[out] = sum == 0.f ? -INFINITY : m + logf(sum);
  }
}

}  // namespace fa2dev
