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
//    captured launch, so each CTA finds its work unit itself: the tiles of all
//    (sequence, query block, head) items are counted, L = ceil(tiles / target)
//    key tiles make one unit, and a warp scan over the sequences finds unit
//    blockIdx.x.  An item of more than L tiles is cut into several units, whose
//    normalised O and LSE go to the workspace and are merged by a second kernel
//    (the merge of fa2_combine.cu, in range order, so results do not vary).
#pragma once

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
  float* O_part;           // [slots][part_rows][D]
  float* LSE_part;         // [slots][part_rows]
  int slots;
  int part_rows;
  int B, T, Hq, Hkv, G;
  int sub_tokens;          // tokens per sub-tile (sub_tokens * G <= 128 rows)
  int box_tokens;          // tokens per Q box (divides sub_tokens)
  int page_log2;           // log2 of the slots per page
  int num_pages;
  int table_width;
  long long table_stride;
  int max_len;             // table_width << page_log2, at most 2^30
  int target_units;
  int min_tiles;           // least key tiles per unit
  int causal;
  int o_half;
  float scale_log2;
  int* status;
  unsigned long long timeout_ns;
};

// One work unit: key tiles [t_begin, t_end) of a block of tokens and a head.
struct PagedUnit {
  int valid;
  int b, head;
  int row0;       // first token of the block in the packed queries
  int tok0;       // the same within its sequence
  int ntok;       // tokens of the block
  int q_len, kv_len;
  int t_begin, t_end;
  int splits, split;
  int slot;       // workspace slot of split 0 is slot - split (splits > 1)
};

// Keys that the token `tok` of a sequence keeps: [0, kept).
__device__ __forceinline__ int paged_kept(int causal, int kv_len, int q_len, int tok) {
  return causal ? max(0, min(kv_len, kv_len - q_len + tok + 1)) : kv_len;
}

// Bytes of one head's K and V that a group of heads may hold in L2 together.
constexpr long long kPagedL2Bytes = 64ll << 20;

// Whole warp: unit `index` (items = false), or the item of rank `index` among
// those cut into several units (items = true; split 0 of it is returned).
template <int SUBS>
__device__ __forceinline__ PagedUnit paged_locate(const PagedParams& p, int index, bool items, int D) {
  const int lane = threadIdx.x & 31;
  const int block = p.sub_tokens * SUBS;
  auto lengths = [&](int b, int& q0, int& nq, int& tiles, int& q_len, int& kv_len) {
    q0 = 0;
    q_len = kv_len = 0;
    if (b < p.B) {
      const int begin = p.cu_q ? p.cu_q[b] : b;
      const int end = p.cu_q ? p.cu_q[b + 1] : b + 1;
      const int kv = p.kv_lens[b];
      q0 = min(max(begin, 0), p.T);
      q_len = max(0, min(end, p.T) - q0);
      kv_len = min(max(kv, 0), p.max_len);
      if (blockIdx.x == 0 && (begin < 0 || end < begin || end > p.T || kv < 0 || kv > p.max_len))
        atomicOr(p.status, kDevErrPage);
    }
    nq = (q_len + block - 1) / block;
    tiles = (kv_len + kKeysPerTile - 1) / kKeysPerTile;
  };
  int q0, nq, tiles, q_len, kv_len;
  long long total = 0;
  for (int b = lane; b < p.B; b += 32) {
    lengths(b, q0, nq, tiles, q_len, kv_len);
    total += static_cast<long long>(nq) * tiles;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  total *= p.Hkv;
  const long long want = (total + p.target_units - 1) / p.target_units;
  const int per_unit = static_cast<int>(max(want, static_cast<long long>(p.min_tiles)));

  PagedUnit u;
  u.valid = 0;
  int before = 0, slots_before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    lengths(b0 + lane, q0, nq, tiles, q_len, kv_len);
    const int s = max(1, (tiles + per_unit - 1) / per_unit);
    const int blocks = nq * p.Hkv;
    const int slots = s > 1 ? blocks * s : 0;
    const int count = items ? (s > 1 ? blocks : 0) : blocks * s;
    int sum = count, slot_sum = slots;   // inclusive scans
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, sum, o);
      const int c = __shfl_up_sync(0xffffffffu, slot_sum, o);
      if (lane >= o) {
        sum += a;
        slot_sum += c;
      }
    }
    const int at = index - before;
    const unsigned here = __ballot_sync(0xffffffffu, at >= sum - count && at < sum);
    if (here != 0) {
      const int src = __ffs(here) - 1;
      auto get = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
      const int splits = get(s), n_blocks = get(nq), all_tiles = get(tiles);
      int in = at - get(sum - count);
      if (items) in *= splits;
      const int slot0 = slots_before + get(slot_sum - slots);
      u.valid = 1;
      u.b = b0 + src;
      u.q_len = get(q_len);
      u.kv_len = get(kv_len);
      u.splits = splits;
      u.slot = slot0 + in;
      // Units of a sequence: groups of heads whose K and V fit in L2 together;
      // within a group the last query blocks (the longest under the causal
      // mask) first, all heads of the group for one block, then the next.
      const long long kv_bytes = static_cast<long long>(max(u.kv_len, 1)) * D * 4;
      const int hg = static_cast<int>(min(max(kPagedL2Bytes / kv_bytes, 1ll), static_cast<long long>(p.Hkv)));
      const int per_group = hg * n_blocks * splits;
      const int group = in / per_group;
      in -= group * per_group;
      const int per_block = min(hg, p.Hkv - group * hg) * splits;
      const int rank = in / per_block;
      in -= rank * per_block;
      const int h = in / splits;
      u.split = in - h * splits;
      u.head = group * hg + h;
      u.tok0 = (n_blocks - 1 - rank) * block;
      u.ntok = min(block, u.q_len - u.tok0);
      u.row0 = get(q0) + u.tok0;
      u.t_begin = u.split * per_unit;
      u.t_end = min(all_tiles, u.t_begin + per_unit);
      return u;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
    slots_before += __shfl_sync(0xffffffffu, slot_sum, 31);
  }
  return u;
}

template <int STAGES>
struct alignas(8) PagedShared {
  FwdBarriers<STAGES> bars;
  PagedUnit unit;
};

// F16: Q, K, V (and P) are fp16 instead of bf16.  SUBS: sub-tiles per CTA, as
// in the dense kernel (2: one CTA per SM, for blocks of more than 128 rows).
template <int D, bool F16, int SUBS>
__global__ void __launch_bounds__(FwdShape<SUBS>::kThreads, FwdShape<SUBS>::kCtasPerSm)
    fa2_paged_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
  using Cfg = FwdConfig<D, SUBS>;
  using Shape = FwdShape<SUBS>;
  constexpr int kWarpProducer = 4 * SUBS;      // schedule and TMA warp
  constexpr int kWarpMma = 4 * SUBS + 1;       // MMA warp, owns the TMEM allocation
  constexpr int STAGES = Cfg::kStages;
  constexpr uint32_t TILE = Cfg::kTileBytes;
  constexpr int NCH = Cfg::kChunks;
  constexpr uint32_t kChunkBytes = kRowsPerSub * 128;  // one 64-column chunk of a 128-row tile
  static_assert(sizeof(PagedShared<STAGES>) <= 1024, "barrier page");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;                  // SUBS sub-tiles
  uint8_t* sKV = smem + SUBS * TILE;   // STAGES tiles
  auto* shared = reinterpret_cast<PagedShared<STAGES>*>(smem + Cfg::kSmemData);
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
    return max(0, min(w.t_end, (kept + kKeysPerTile - 1) / kKeysPerTile) - w.t_begin);
  };

  // State of the producer warp: table entries [chunk0, chunk0 + 32) of the
  // sequence in `pages`, the next 32 in `pages_next`, one per lane.
  const int slots_log2 = min(p.page_log2, 7);           // slots of a page that one tile reads
  const int tile_pages = kKeysPerTile >> slots_log2;    // pages (boxes per 64 columns) of a tile
  int pages = 0, pages_next = 0, chunk0 = 0;
  const int* table = nullptr;
  int live_pages = 0;                                   // table entries that hold keys
  auto fetch = [&](int first) {
    const int i = first + lane;
    int id = 0;
    if (i < live_pages) {
      id = table[i];
      if (id < 0 || id >= p.num_pages) atomicOr(p.status, kDevErrPage);
    }
    return id;
  };
  // whole warp: K (kind 0) or V (kind 1) tile `tile` into ring slot `slot`
  auto load_tile = [&](const PagedUnit& w, int tile, int kind, int slot) {
    const int first = (tile << 7) >> p.page_log2;       // table entry of the tile's first page
    if (first >= chunk0 + 32) {
      chunk0 += 32;
      pages = pages_next;
      pages_next = fetch(chunk0 + 32);
    }
    const int n = min(tile_pages, live_pages - first);
    const int id = __shfl_sync(0xffffffffu, pages, (first - chunk0 + lane) & 31);
    if (lane == 0) bar_arrive_expect_tx(&bars->kv_full[slot], static_cast<uint32_t>(n) * NCH * (128u << slots_log2));
    __syncwarp();
    if (lane < n) {
      const CUtensorMap* map = kind == 0 ? &tm_k : &tm_v;
      const int row = p.page_log2 > 7 ? (tile << 7) & ((1 << p.page_log2) - 1) : 0;
      uint8_t* dst = sKV + slot * TILE + (static_cast<uint32_t>(lane) << slots_log2) * 128;
#pragma unroll
      for (int c = 0; c < NCH; ++c)
        tma_load_4d(dst + c * kChunkBytes, map, &bars->kv_full[slot], c * 64, row, w.head, id);
    }
    __syncwarp();
  };

  if (warp == kWarpProducer) {
    if (lane == 0) {
      bar_init(&bars->q_full, 1);
      for (int s = 0; s < STAGES; ++s) {
        bar_init(&bars->kv_full[s], 1);
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
    const PagedUnit w = paged_locate<SUBS>(p, static_cast<int>(blockIdx.x), false, D);
    if (lane == 0) shared->unit = w;
    __syncwarp();
    if (w.valid) {
      const int n0 = tiles_for(w, 0), n1 = SUBS == 2 ? tiles_for(w, 1) : 0;
      const int nmax = max(n0, n1);
      if (nmax > 0) {
        table = p.page_table + static_cast<long long>(w.b) * p.table_stride;
        live_pages = (w.kv_len + (1 << p.page_log2) - 1) >> p.page_log2;
        chunk0 = (w.t_begin << 7) >> p.page_log2;
        pages = fetch(chunk0);
        pages_next = fetch(chunk0 + 32);
        // Q boxes of the live tokens: lane i loads box i of each sub-tile
        const uint32_t box_bytes = static_cast<uint32_t>(p.box_tokens) * p.G * 128;
        const int per_sub = p.sub_tokens / p.box_tokens;
        const int boxes = (w.ntok + p.box_tokens - 1) / p.box_tokens;
        if (lane == 0) bar_arrive_expect_tx(&bars->q_full, static_cast<uint32_t>(boxes) * NCH * box_bytes);
        __syncwarp();
        for (int i = lane; i < boxes; i += 32) {
          const int sub = i / per_sub;
          uint8_t* dst = sQ + sub * TILE + (i - sub * per_sub) * box_bytes;
          for (int c = 0; c < NCH; ++c)
            tma_load_3d(dst + c * kChunkBytes, &tm_q, &bars->q_full, c * 64, w.head * p.G,
                        w.row0 + i * p.box_tokens);
        }
        __syncwarp();
        const int primed = min(STAGES, 2 * nmax);
        for (int g = 0; g < primed; ++g) load_tile(w, w.t_begin + g / 2, g & 1, g);
      }
    }
  }
  if (warp == kWarpMma) {
    tmem_alloc(&bars->tmem_base, Cfg::kTmemCols);
    tmem_relinquish();
    tc_fence_before_sync();
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  const PagedUnit w = shared->unit;
  const int n0 = w.valid ? tiles_for(w, 0) : 0;
  const int n1 = w.valid && SUBS == 2 ? tiles_for(w, 1) : 0;
  const int nmax = max(n0, n1);

  if (warp >= kWarpProducer) {
    regs_decrease<Shape::kProducer>();
    if (warp == kWarpProducer) {
      // ------------------------------------------------------------ TMA producer
      int issued = min(STAGES, 2 * nmax);
      bool ok = true;
      for (; issued < 2 * nmax && ok; ++issued) {
        const int slot = issued % STAGES;
        const int lap = issued / STAGES;
        if (lane == 0) ok = wait_bar(&bars->kv_empty[slot], (lap - 1) & 1, abort, p.timeout_ns);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          if (lane == 0) raise_abort(abort, p.status);
          break;
        }
        load_tile(w, w.t_begin + issued / 2, issued & 1, slot);
      }
      // Before the CTA may exit, every copy it started must have landed.
      if (lane == 0 && nmax > 0) {
        volatile int never = 0;
        wait_bar(&bars->q_full, 0, &never, p.timeout_ns);
        for (int k = max(0, issued - STAGES); k < issued; ++k)
          wait_bar(&bars->kv_full[k % STAGES], (k / STAGES) & 1, &never, p.timeout_ns);
      }
      __syncwarp();
    } else if (warp == kWarpMma + 1 && Cfg::kNamedP) {
      // ------------------------------------------------------------ K/V watcher
      bool ok = true;
      for (int j = 0; j < nmax; ++j) {
        if (lane == 0 && ok) {
          const int iv = 2 * j + 1, ik = 2 * j + 2;
          ok = wait_bar(&bars->kv_full[iv % STAGES], (iv / STAGES) & 1, abort, p.timeout_ns);
          if (ok && j + 1 < nmax)
            ok = wait_bar(&bars->kv_full[ik % STAGES], (ik / STAGES) & 1, abort, p.timeout_ns);
          if (!ok) raise_abort(abort, p.status);
        }
        __syncwarp();
        named_sync(kBarP0, j < n0 ? kBarP0Count : kBarP0Idle);
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
      if (lane == 0 && nmax > 0) {
        ok = wait_bar(&bars->q_full, 0, abort, p.timeout_ns) &&
             wait_bar(&bars->kv_full[0], 0, abort, p.timeout_ns);
        if (!ok) raise_abort(abort, p.status);
        tc_fence_after_sync();
        if (ok || Cfg::kNamedP) {
          if (n0 > 0) { issue_s(0, 0, 0); mma_commit(&bars->s_full[0]); }
          if (n1 > 0) { issue_s(1, 0, 1); mma_commit(&bars->s_full[1]); }
          if (!Cfg::kSoftmaxRelease) mma_commit(&bars->kv_empty[0]);
        }
      }
      __syncwarp();
      if constexpr (Cfg::kNamedP) {
        // named barriers: every phase is passed, also after an abort
        for (int j = 0; j < nmax; ++j) {
          const int slot_v = (2 * j + 1) % STAGES, slot_k = (2 * j + 2) % STAGES;
          named_sync(kBarP0, j < n0 ? kBarP0Count : kBarP0Idle);
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
            named_sync(kBarP1, kBarP1Count);
            if (lane == 0) {
              tc_fence_after_sync();
              issue_pv(1, slot_v, j > 0, 1);
              if (j + 1 == n1) mma_commit(&bars->o_done[1]);
              if (j + 1 < n1) { issue_s(1, slot_k, 1); mma_commit(&bars->s_full[1]); }
            }
            __syncwarp();
          }
        }
      } else if (lane == 0 && nmax > 0) {
        if constexpr (Cfg::kDoubleS) {
          for (int j = 0; j < n0 && ok; ++j) {
            const int iv = 2 * j + 1, ik = 2 * j + 2;
            const int slot_v = iv % STAGES, slot_k = ik % STAGES;
            if (j + 1 < n0) {
              if (!wait_bar(&bars->kv_full[slot_k], (ik / STAGES) & 1, abort, p.timeout_ns)) { ok = false; break; }
              tc_fence_after_sync();
              issue_s(0, slot_k, (j + 1) & 1);
              mma_commit(&bars->s_full[(j + 1) & 1]);
              mma_commit(&bars->kv_empty[slot_k]);
            }
            uint64_t* bv = &bars->kv_full[slot_v];
            const uint32_t pv = (iv / STAGES) & 1;
            if (!wait_bar3(bv, pv, &bars->p_ready[j & 1], (j >> 1) & 1, bv, pv, abort, p.timeout_ns)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            issue_pv(0, slot_v, j > 0, j & 1);
            mma_commit(&bars->o_done[0]);
            mma_commit(&bars->kv_empty[slot_v]);
          }
        } else {
          static_assert(Cfg::kNamedP || Cfg::kDoubleS || SUBS == 1, "polled order: one sub-tile");
          for (int j = 0; j < n0 && ok; ++j) {
            const int iv = 2 * j + 1, ik = 2 * j + 2;
            const int slot_v = iv % STAGES, slot_k = ik % STAGES;
            uint64_t* bv = &bars->kv_full[slot_v];
            const uint32_t pv = (iv / STAGES) & 1;
            if (!wait_bar3(bv, pv, &bars->p_ready[0], j & 1, bv, pv, abort, p.timeout_ns)) { ok = false; break; }
            tc_fence_after_sync();
            issue_pv(0, slot_v, j > 0, 0);
            if (j + 1 == n0) mma_commit(&bars->o_done[0]);
            mma_commit(&bars->kv_empty[slot_v]);
            if (j + 1 < n0) {
              if (!wait_bar(&bars->kv_full[slot_k], (ik / STAGES) & 1, abort, p.timeout_ns)) { ok = false; break; }
              tc_fence_after_sync();
              issue_s(0, slot_k, 0);
              mma_commit(&bars->s_full[0]);
              mma_commit(&bars->kv_empty[slot_k]);
            }
          }
        }
        if (!ok) raise_abort(abort, p.status);
      }
      if (lane == 0 && nmax > 0) {
        // Every MMA must be complete before TMEM is released.
        mma_commit(&bars->mma_drain);
        volatile int never = 0;
        wait_bar(&bars->mma_drain, 0, &never, p.timeout_ns);
      }
      __syncwarp();
    }
  } else {
    regs_increase<Shape::kSoftmax>();
    // ------------------------------------------------------------ softmax
    const int sub = warp >> 2;
    const int n_tiles = sub == 0 ? n0 : n1;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;                       // TMEM lane = row of the sub-tile
    const int sub_tok0 = w.valid ? sub * p.sub_tokens : 0;
    const int rows = w.valid ? max(0, min(p.sub_tokens, w.ntok - sub_tok0)) * p.G : 0;   // live rows
    const bool live = row < rows;
    const bool warp_live = wq * 32 < rows;
    const int tok = row / p.G;                            // token of the sub-tile
    const int lim = live ? paged_kept(p.causal, w.kv_len, w.q_len, w.tok0 + sub_tok0 + tok) : 0;
    // every live row keeps at least the first token's keys
    const int lim_min = w.valid ? paged_kept(p.causal, w.kv_len, w.q_len, w.tok0 + sub_tok0) : 0;
    const uint32_t lane_bits = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS0 = tmem + lane_bits + sub * 128;
    const uint32_t tO = tmem + lane_bits + (sub == 0 ? Cfg::kColsO0 : Cfg::kColsO1);
    const float sl2 = p.scale_log2;

    // One thread of the sub-tile that visits every key tile releases the ring slots.
    const bool releaser = (threadIdx.x & (kRowsPerSub - 1)) == 0 && n_tiles == nmax &&
                          (sub == SUBS - 1 || n1 == 0);
    float m = -INFINITY;
    float l = 0.f;
    bool ok = true;
    int announced = 0;
    for (int j = 0; j < n_tiles; ++j) {
      uint64_t* sbar = &bars->s_full[Cfg::kDoubleS ? (j & 1) : sub];
      const uint32_t s_phase = Cfg::kDoubleS ? (j >> 1) & 1 : j & 1;
      const uint32_t tS = Cfg::kDoubleS ? tS0 + (j & 1) * 128 : tS0;
      if (!__all_sync(0xffffffffu, wait_bar(sbar, s_phase, abort, p.timeout_ns))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      if (Cfg::kSoftmaxRelease && releaser) {
        if (j > 0) bar_arrive(&bars->kv_empty[(2 * j - 1) % STAGES]);
        bar_arrive(&bars->kv_empty[(2 * j) % STAGES]);
      }
      const int key0 = (w.t_begin + j) * kKeysPerTile;
      // V rows behind the last key: zeros, written by the first sub-tile that reads them
      if (key0 + kKeysPerTile > w.kv_len && (sub == 0 || j >= n0)) {
        const int iv = 2 * j + 1;
        if (!__all_sync(0xffffffffu, wait_bar(&bars->kv_full[iv % STAGES], (iv / STAGES) & 1, abort, p.timeout_ns))) {
          ok = false;
          break;
        }
        const uint32_t v_addr = smem_addr(sKV + (iv % STAGES) * TILE);
        const uint32_t keep_bytes = static_cast<uint32_t>(w.kv_len - key0) * 128;
#pragma unroll
        for (int c = 0; c < NCH; ++c)
          for (uint32_t at = keep_bytes + row * 16; at < kChunkBytes; at += kRowsPerSub * 16)
            st_shared_v4(v_addr + c * kChunkBytes + at, 0u, 0u, 0u, 0u);
        fence_proxy_async_shared();
      }
      if (warp_live) {
        uint32_t s[4][32];
        const bool masked = key0 + kKeysPerTile > lim_min;
        auto load_s = [&]() {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, s[c]);
          tmem_ld_wait(s[0]);
#pragma unroll
          for (int c = 1; c < 4; ++c) regs_after_wait(s[c]);
          if (masked) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (key0 + c * 32 + e >= lim) s[c][e] = __float_as_uint(-INFINITY);
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
          for (int f = 8; f < 120; f += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k) mx8[k] = fmax3(mx8[k], FA2_S(f + k), FA2_S(f + 8 + k));
#pragma unroll
          for (int k = 0; k < 8; ++k) mx8[k] = fmaxf(mx8[k], FA2_S(120 + k));
#undef FA2_S
          const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                                 fmaxf(mx8[6], mx8[7]));
          const float m_cand = fmaxf(m, mx * sl2);
          const bool move = m == -INFINITY || m_cand > m + kRescaleLog2;
          m_new = move ? m_cand : m;
          alpha = !move ? 1.f : (m == -INFINITY ? 0.f : ex2_approx(m - m_new));
        };
        uint32_t pk[2][32];
        float rs;
        auto exps = [&]() {
          const float off = m_new == -INFINITY ? 0.f : m_new;
          const float2 c2 = make_float2(sl2, sl2);
          const float2 o2 = make_float2(-off, -off);
          float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                           make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 t = __ffma2_rn(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), c2, o2);
              const float2 pe = make_float2(ex2_approx(t.x), ex2_approx(t.y));
              acc[(e >> 1) & 3] = __fadd2_rn(acc[(e >> 1) & 3], pe);
              pk[c >> 1][(c & 1) * 16 + (e >> 1)] = pack_x2<F16>(pe.x, pe.y);
            }
          }
          const float2 a01 = __fadd2_rn(acc[0], acc[1]);
          const float2 a23 = __fadd2_rn(acc[2], acc[3]);
          const float2 a = __fadd2_rn(a01, a23);
          rs = a.x + a.y;
        };
        load_s();
        const bool max_first = __any_sync(0xffffffffu, live && m == -INFINITY);
        bool decided = max_first;
        if (max_first) decide();
        exps();
        if (!max_first && __any_sync(0xffffffffu, live && rs > kRescaleBound)) {
          load_s();
          decide();
          exps();
          decided = true;
        }
        tmem_st32(tS, pk[0]);
        tmem_st32(tS + 32, pk[1]);
        l = l * alpha + rs;
        m = m_new;
        const bool rescale = decided && j > 0 && __any_sync(0xffffffffu, live && alpha != 1.f);
        if (!Cfg::kOutDoneLast && j > 0 && (rescale || j == n_tiles - 1) &&
            !__all_sync(0xffffffffu, wait_bar(&bars->o_done[sub], (j - 1) & 1, abort, p.timeout_ns))) {
          ok = false;
        }
        if (rescale && ok) {
          tc_fence_after_sync();
#pragma unroll
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
        bar_arrive(&bars->p_ready[Cfg::kDoubleS ? (j & 1) : sub]);
      }
      announced = j + 1;
      if (!ok) break;
    }
    if constexpr (Cfg::kNamedP) {
      // after an abort: the remaining phases, in step with the issuing warp
      __syncwarp();
      for (int j = announced; j < n_tiles; ++j)
        named_sync(sub == 0 ? kBarP0 : kBarP1, sub == 0 ? kBarP0Count : kBarP1Count);
    }

    // Outputs: the final rows, or this key range's rows in its workspace slot.
    const bool part = w.valid && w.splits > 1;
    const bool fits = !part || (w.slot >= 0 && w.slot < p.slots);   // always, for lengths within the launch's bounds
    const bool store = live && fits;
    const long long prow = part ? static_cast<long long>(w.slot) * p.part_rows + sub_tok0 * p.G + row
                                : static_cast<long long>(w.row0 + sub_tok0 + tok) * p.Hq + w.head * p.G + (row - tok * p.G);
    float* lse_out = (part ? p.LSE_part : p.LSE) + prow;
    const bool half_out = p.o_half != 0 && !part;
    if (w.valid && !fits && threadIdx.x == 0) atomicOr(p.status, kDevErrPage);
    if (n_tiles == 0 && store) {
      // no kept key: O = 0 and LSE = -inf (a key range: LSE alone, the merge skips its O)
      *lse_out = -INFINITY;
      if (!part) {
        uint8_t* o = static_cast<uint8_t*>(p.O) + prow * (half_out ? D * 2 : D * 4);
        for (int c = 0; c < (half_out ? D * 2 : D * 4); c += 16) *reinterpret_cast<uint4*>(o + c) = make_uint4(0, 0, 0, 0);
      }
    }
    if (n_tiles > 0 && ok) {
      if (store) *lse_out = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
      if (!__all_sync(0xffffffffu,
                      wait_bar(&bars->o_done[sub], Cfg::kOutDoneLast ? 0u : (n_tiles - 1) & 1, abort, p.timeout_ns))) {
        ok = false;
      } else if (warp_live) {
        tc_fence_after_sync();
        // O / l goes through this warp's quarter of its sub-tile's Q buffer
        // (every S MMA that read it has completed) so that the global stores
        // are whole rows: D * 2 bytes a row and round (fp32 O: two rounds).
        const float inv_l = l == 0.f ? 0.f : 1.f / l;
        constexpr int kUnits = D / 8;               // 16-byte units of a staged row
        const uint32_t stage = smem_addr(sQ + sub * TILE) + wq * (TILE / 4);
        const uint32_t mine = stage + lane * (D * 2);
        const long long row_bytes = half_out ? D * 2 : D * 4;
        uint8_t* base = static_cast<uint8_t*>(part ? static_cast<void*>(p.O_part) : p.O);
        const long long my_off = store ? prow * row_bytes : -1;
        const int parts = half_out ? 1 : 2;
        for (int r = 0; r < parts; ++r) {
          if (r > 0) __syncwarp();
#pragma unroll
          for (int b = 0; b < D / 64; ++b) {
            if (!half_out) {
              uint32_t o[32];
              tmem_ld32(tO + r * (D / 2) + 32 * b, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int u = 0; u < 8; ++u)
                st_shared_v4(mine + (((b * 8 + u) ^ (lane & 7)) << 4), __float_as_uint(__uint_as_float(o[4 * u]) * inv_l),
                             __float_as_uint(__uint_as_float(o[4 * u + 1]) * inv_l),
                             __float_as_uint(__uint_as_float(o[4 * u + 2]) * inv_l),
                             __float_as_uint(__uint_as_float(o[4 * u + 3]) * inv_l));
            } else {
              uint32_t o[2][32];
              tmem_ld32(tO + 64 * b, o[0]);
              tmem_ld32(tO + 64 * b + 32, o[1]);
              tmem_ld_wait(o[0]);
              tmem_ld_wait(o[1]);
              uint32_t h[32];
#pragma unroll
              for (int e = 0; e < 32; ++e)
                h[e] = pack_x2<F16>(__uint_as_float(o[e >> 4][(2 * e) & 31]) * inv_l,
                                    __uint_as_float(o[e >> 4][(2 * e + 1) & 31]) * inv_l);
#pragma unroll
              for (int u = 0; u < 8; ++u)
                st_shared_v4(mine + (((b * 8 + u) ^ (lane & 7)) << 4), h[4 * u], h[4 * u + 1], h[4 * u + 2], h[4 * u + 3]);
            }
          }
          __syncwarp();
          constexpr int kRowsPer = 32 / kUnits > 0 ? 32 / kUnits : 1;   // rows written by one warp store
#pragma unroll 4
          for (int i = 0; i < 32; i += kRowsPer) {
            const int rr = i + lane / kUnits, unit = lane % kUnits;
            const long long off = __shfl_sync(0xffffffffu, my_off, rr);
            uint32_t v[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(stage + rr * (D * 2) + ((unit ^ (rr & 7)) << 4)));
            if (off >= 0)
              *reinterpret_cast<uint4*>(base + off + r * (D * 2) + unit * 16) = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
      }
    }
    if (!ok) raise_abort(abort, p.status);
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

constexpr int kPagedMergeWarps = 8;

// Merge of the key ranges of one item: one CTA per item that was cut, a warp
// per row.  With m = max_s L_s and w_s = exp(L_s - m): O = sum_s w_s O_s / sum
// w_s, LSE = m + log sum w_s; ranges with L_s = -inf are skipped unread.
template <int D, bool F16, int SUBS>
__global__ void __launch_bounds__(kPagedMergeWarps * 32) fa2_paged_merge_kernel(const PagedParams p) {
  constexpr int V = D / 32;
  const PagedUnit w = paged_locate<SUBS>(p, static_cast<int>(blockIdx.x), true, D);
  if (!w.valid || w.slot < 0 || w.slot + w.splits > p.slots) return;
  const int lane = threadIdx.x & 31;
  for (int row = threadIdx.x >> 5; row < w.ntok * p.G; row += kPagedMergeWarps) {
    const float* L = p.LSE_part + static_cast<long long>(w.slot) * p.part_rows + row;
    float mx = -INFINITY;
    for (int s = lane; s < w.splits; s += 32) mx = fmaxf(mx, L[static_cast<long long>(s) * p.part_rows]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    float sum = 0.f;
    for (int s = 0; s < w.splits; ++s) {
      const float ls = L[static_cast<long long>(s) * p.part_rows];
      if (ls == -INFINITY) continue;
      const float e = expf(ls - mx);
      sum += e;
      const float* src = p.O_part + ((static_cast<long long>(w.slot) + s) * p.part_rows + row) * D + lane * V;
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] = fmaf(e, src[c], acc[c]);
    }
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    const int tok = row / p.G;
    const long long out = static_cast<long long>(w.row0 + tok) * p.Hq + w.head * p.G + (row - tok * p.G);
    if (p.o_half) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.O) + out * D + lane * V);
#pragma unroll
      for (int c = 0; c < V; c += 2) dst[c / 2] = pack_x2<F16>(acc[c] * inv, acc[c + 1] * inv);
    } else {
      float* dst = static_cast<float*>(p.O) + out * D + lane * V;
#pragma unroll
      for (int c = 0; c < V; ++c) dst[c] = acc[c] * inv;
    }
    if (lane == 0) p.LSE[out] = sum == 0.f ? -INFINITY : mx + logf(sum);
  }
}

}  // namespace fa2dev
