// Host side of the paged-cache entry points (include/fa2.h): argument
// validation, tensor maps, launch plans.
#include <cmath>
#include <cstdint>

#include "fa2.h"
#include "fa2_host.h"
#include "fa2_launch.h"
#include "fa2_pages.h"
#include "fa2_rope.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr long long kMaxStride = 1ll << 38;   // elements; TMA strides stay below 2^40 bytes

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

bool misaligned(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

int log2_exact(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return (1 << l) == x ? l : -1;
}

int page_log2(int page_size) {
  return page_size >= 16 && page_size <= 1024 ? log2_exact(page_size) : -1;
}

// Elements that a strided array reaches, or -1: sizes and strides of its outer
// dimensions, the last dimension of `inner` neighbouring elements.
template <int N>
long long extent(const long long (&sizes)[N], const long long (&strides)[N], long long inner) {
  long long e = inner;
  for (int i = 0; i < N; ++i) {
    if (strides[i] < 0 || strides[i] > kMaxStride || sizes[i] < 0 || sizes[i] > 0x7fffffffll) return -1;
    if (sizes[i] > 1) {
      if (strides[i] > (1ll << 60) / sizes[i]) return -1;
      e += (sizes[i] - 1) * strides[i];
    }
  }
  return e;
}

// The rows of an array that is written lie apart: with its outer dimensions (those
// of more than one step) in the order of their strides, each steps past all that
// the smaller ones reach.  Strides that interleave dimensions without a common
// element are refused too; no view of a dense array has such.
template <int N>
bool rows_apart(const long long (&sizes)[N], const long long (&strides)[N], long long inner) {
  bool taken[N] = {};
  long long reach = inner;
  for (int n = 0; n < N; ++n) {
    int least = -1;
    for (int i = 0; i < N; ++i)
      if (!taken[i] && sizes[i] > 1 && (least < 0 || strides[i] < strides[least])) least = i;
    if (least < 0) return true;
    if (strides[least] < reach) return false;
    if (strides[least] > (1ll << 60) / sizes[least]) return false;
    reach += (sizes[least] - 1) * strides[least];
    taken[least] = true;
  }
  return true;
}

bool range_ok(const void* p, long long elems, int size) {
  return elems >= 0 && fa2host::device_memory_ok(p, static_cast<size_t>(elems) * size);
}

// Everything about a cache that can be checked on the host without a device.
int check_cache(const fa2_paged_cache* c) {
  if (!c) return FA2_ERR_NULL;
  if (c->dtype != FA2_DTYPE_BF16 && c->dtype != FA2_DTYPE_FP16) return FA2_ERR_DTYPE;
  if (c->num_pages < 1 || c->kv_heads < 1 || c->B < 0 || c->table_width < 1 || page_log2(c->page_size) < 0)
    return FA2_ERR_SHAPE;
  if (c->d != 64 && c->d != 128 && c->d != 256) return FA2_ERR_HEADDIM;
  if (static_cast<long long>(c->table_width) * c->page_size > (1ll << 30)) return FA2_ERR_SHAPE;
  // a slot, a head and a page may not overlap the next
  if (c->slot_stride < c->d || c->slot_stride > kMaxStride) return FA2_ERR_SHAPE;
  if (c->kv_heads > 1 && (c->head_stride < c->d || c->head_stride > kMaxStride)) return FA2_ERR_SHAPE;
  if (c->num_pages > 1 && (c->page_stride < c->d || c->page_stride > kMaxStride)) return FA2_ERR_SHAPE;
  if (c->B > 1 && (c->table_stride < c->table_width || c->table_stride > kMaxStride)) return FA2_ERR_SHAPE;
  if (!c->k_pages || !c->v_pages || !c->page_table || !c->kv_lens) return FA2_ERR_NULL;
  if (misaligned(c->k_pages, 15) || misaligned(c->v_pages, 15) || c->slot_stride % 8 != 0 ||
      (c->kv_heads > 1 && c->head_stride % 8 != 0) || (c->num_pages > 1 && c->page_stride % 8 != 0) ||
      misaligned(c->page_table, 3) || misaligned(c->kv_lens, 3))
    return FA2_ERR_ALIGN;
  return FA2_OK;
}

int check_cache_memory(const fa2_paged_cache* c) {
  const long long sizes[3] = {c->num_pages, c->kv_heads, c->page_size};
  const long long strides[3] = {c->num_pages > 1 ? c->page_stride : 0, c->kv_heads > 1 ? c->head_stride : 0,
                                c->slot_stride};
  const long long e = extent(sizes, strides, c->d);
  const long long ts[1] = {c->B}, tr[1] = {c->B > 1 ? c->table_stride : 0};
  if (!range_ok(c->k_pages, e, 2) || !range_ok(c->v_pages, e, 2) ||
      !range_ok(c->page_table, extent(ts, tr, c->table_width), 4) || !range_ok(c->kv_lens, c->B, 4))
    return FA2_ERR_MEMORY;
  return FA2_OK;
}

// Packed rows [T, H, d]: token and head strides in elements.
int check_rows(const void* p, long long token, long long head, long long T, int H, int d) {
  if ((T > 1 && (token < d || token > kMaxStride)) || (H > 1 && (head < d || head > kMaxStride))) return FA2_ERR_SHAPE;
  if (!p) return FA2_ERR_NULL;
  if (misaligned(p, 15) || (T > 1 && token % 8 != 0) || (H > 1 && head % 8 != 0)) return FA2_ERR_ALIGN;
  return FA2_OK;
}

bool rows_in_memory(const void* p, long long token, long long head, long long T, int H, int d) {
  const long long sizes[2] = {T, H};
  const long long strides[2] = {T > 1 ? token : 0, H > 1 ? head : 0};
  return range_ok(p, extent(sizes, strides, d), 2);
}

// How a call of fa2_forward_paged is laid out; depends on sizes alone.
struct PagedPlan {
  int G, subs, sub_tokens, box_tokens, part_rows;
  bool narrow;            // blocks of at most 32 rows (single tokens)
  bool even;              // equal ranges of key tiles, one per CTA of a single wave
  int ctas, slots;
  long long items;        // most (sequence, block, head) items there can be
  size_t lse_at, counter_at, bytes;   // workspace: partial O, partial LSE, the counter
};

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

// Blocks of queries that fill this many waves of CTAs are taken whole: many at a
// time then share keys in L2, where equal ranges spread over all heads at once,
// but the last wave ends unevenly.  Over 90 ragged batches (time whole / equal
// ranges): d <= 128, below 3 waves 0.83 to 1.60, mean 1.2; 3.5 to 7 waves 0.88 to
// 1.18, mean 1.0, and 0.90 for 32 long heads at 6.7.  d = 256, whose blocks have
// half the rows and whose tiles are twice as large: below 2 waves 0.80 to 1.45,
// mean 1.1; above 0.77 to 1.07, mean 0.9.
constexpr int kItemWaves = 4;
constexpr int kItemWaves256 = 2;
// The three below from 40 random batches each (1 to 300 sequences of 20 to 60000
// keys, every head size, groups of 1 to 8; geometric mean of the times against the
// value taken, worst and best batch).
// Least key tiles of a range: two 1.03 (0.94 to 1.20), four 1.07 (0.85 to 1.40).
constexpr int kMinTiles = 1;
// What an item costs besides its keys (pipeline fill, epilogue), in keys; a range
// is at least that and a tile.  Chunks: 128 1.05 (0.86 to 1.27), 256 1.01 (0.91 to
// 1.13), 384 1.00 (0.93 to 1.08), 768 1.02 (0.94 to 1.09), 1024 1.04 (0.94 to 1.16).
// Single tokens: none 1.16 (1.00 to 1.87), 128 1.02 (0.91 to 1.11), 384 1.01 (0.91 to
// 1.21), 512 1.02 (0.88 to 1.21).
constexpr int kItemKeys = 512;
constexpr int kItemKeysNarrow = 256;

// Sub-tiles per CTA: two (256 rows on one K/V stream) where the sequences'
// average chunk fills more than one sub-tile, else one with two CTAs per SM, of
// at most 32 rows where the average chunk has no more.  The host knows the sizes
// alone, so one form serves the whole batch: 64 single tokens and a chunk of 512
// take 149 us together, 109 and 58 apart, but a chunk that is long for the average
// is cut into blocks of 32 rows (1024 single tokens over 100-500 keys and a chunk of
// 7000: 1497 us, 252 and 319 apart).
PagedPlan plan_paged(int B, int T, int Hq, int Hkv, int d, bool has_cu, int sms) {
  PagedPlan q;
  q.G = Hq / Hkv;
  q.subs = has_cu && d != 256 && static_cast<long long>(T) * q.G > 128ll * B ? 2 : 1;
  // Q boxes start on whole 1024-byte swizzle atoms (8 rows): the tokens per
  // box are the fewest that fill whole atoms, where 128 rows hold that many.
  q.narrow = q.G <= 32 && (!has_cu || static_cast<long long>(T) * q.G <= 32ll * B);
  const int most = (q.narrow ? 32 : 128) / q.G, unit = 8 / gcd(q.G, 8);
  q.box_tokens = most >= unit ? unit : most;
  q.sub_tokens = most / q.box_tokens * q.box_tokens;
  const int block = q.sub_tokens * q.subs;
  q.items = (has_cu ? T / block + static_cast<long long>(B < T ? B : T) : B) * Hkv;
  q.ctas = sms * (q.subs == 2 || d == 256 ? 1 : 2);
  const long long waves = d == 256 ? kItemWaves256 : kItemWaves;
  q.even = q.narrow || !has_cu || T / block * static_cast<long long>(Hkv) < waves * q.ctas;
  q.slots = 2 * q.ctas;
  const long long rows = static_cast<long long>(has_cu ? (T < block ? T : block) : 1) * q.G;
  q.part_rows = static_cast<int>(rows);
  q.lse_at = align256(static_cast<size_t>(q.slots) * rows * d * 4);
  q.counter_at = q.lse_at + align256(static_cast<size_t>(q.slots) * rows * 4);
  q.bytes = q.counter_at + 256;
  return q;
}

}  // namespace

extern "C" size_t fa2_forward_paged_workspace_bytes(int B, int T, int Hq, int kv_heads, int d, int has_cu_q) {
  if (B < 1 || T < 1 || Hq < 1 || kv_heads < 1 || Hq % kv_heads != 0 || Hq / kv_heads > 128) return 0;
  if (d != 64 && d != 128 && d != 256) return 0;
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return plan_paged(B, T, Hq, kv_heads, d, has_cu_q != 0, sms).bytes;
}

extern "C" int fa2_forward_paged(const fa2_paged_cache* cache, const void* Q, long long q_token_stride,
                                 long long q_head_stride, void* O, float* LSE, const int* cu_q, int T, int Hq,
                                 int causal, float scale, int o_dtype, void* workspace, size_t workspace_size,
                                 fa2_stream_t stream) {
  if (!cache) return FA2_ERR_NULL;
  if (T < 0 || Hq < 0) return FA2_ERR_SHAPE;
  if (T == 0 || Hq == 0 || cache->B == 0) return FA2_OK;
  int rc = check_cache(cache);
  if (rc != FA2_OK) return rc;
  const fa2_paged_cache& c = *cache;
  if (o_dtype != FA2_DTYPE_FP32 && o_dtype != c.dtype) return FA2_ERR_DTYPE;
  if (Hq % c.kv_heads != 0 || Hq / c.kv_heads > 128 || (!cu_q && T != c.B)) return FA2_ERR_SHAPE;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA2_ERR_SCALE;
  if ((rc = check_rows(Q, q_token_stride, q_head_stride, T, Hq, c.d)) != FA2_OK) return rc;
  if (!O || !LSE || !workspace) return FA2_ERR_NULL;
  if (misaligned(O, 15) || misaligned(LSE, 3) || misaligned(cu_q, 3) || misaligned(workspace, 255)) return FA2_ERR_ALIGN;
  if ((rc = fa2host::require_device()) != FA2_OK) return rc;
  const bool half_out = o_dtype != FA2_DTYPE_FP32, f16 = c.dtype == FA2_DTYPE_FP16;
  const long long rows = static_cast<long long>(T) * Hq;
  const PagedPlan plan = plan_paged(c.B, T, Hq, c.kv_heads, c.d, cu_q != nullptr, fa2host::device_sms());
  if ((rc = check_cache_memory(cache)) != FA2_OK) return rc;
  if (!rows_in_memory(Q, q_token_stride, q_head_stride, T, Hq, c.d) || !range_ok(O, rows * c.d, half_out ? 2 : 4) ||
      !range_ok(LSE, rows, 4) || (cu_q && !range_ok(cu_q, c.B + 1ll, 4)) || workspace_size < plan.bytes ||
      !fa2host::device_memory_ok(workspace, plan.bytes))
    return FA2_ERR_MEMORY;
  if (plan.items + 2ll * plan.ctas > 0x7fffffffll) return FA2_ERR_SHAPE;

  using ull = unsigned long long;
  CUtensorMap mq, mk, mv;
  const ull qd[3] = {static_cast<ull>(c.d), static_cast<ull>(Hq), static_cast<ull>(T)};
  const ull row_bytes = static_cast<ull>(c.d) * 2;
  const ull qs[2] = {Hq > 1 ? static_cast<ull>(q_head_stride) * 2 : row_bytes,
                     T > 1 ? static_cast<ull>(q_token_stride) * 2 : row_bytes};
  const unsigned qb[3] = {64, static_cast<unsigned>(plan.G), static_cast<unsigned>(plan.box_tokens)};
  const ull kd[4] = {static_cast<ull>(c.d), static_cast<ull>(c.page_size), static_cast<ull>(c.kv_heads),
                     static_cast<ull>(c.num_pages)};
  const ull ks[3] = {static_cast<ull>(c.slot_stride) * 2,
                     c.kv_heads > 1 ? static_cast<ull>(c.head_stride) * 2 : row_bytes,
                     c.num_pages > 1 ? static_cast<ull>(c.page_stride) * 2 : row_bytes};
  const unsigned kb[4] = {64, static_cast<unsigned>(c.page_size < 128 ? c.page_size : 128), 1, 1};
  if (!fa2host::encode_tiled(&mq, f16, 3, Q, qd, qs, qb) || !fa2host::encode_tiled(&mk, f16, 4, c.k_pages, kd, ks, kb) ||
      !fa2host::encode_tiled(&mv, f16, 4, c.v_pages, kd, ks, kb))
    return FA2_ERR_SHAPE;

  fa2dev::PagedParams p;
  p.page_table = c.page_table;
  p.kv_lens = c.kv_lens;
  p.cu_q = cu_q;
  p.O = O;
  p.LSE = LSE;
  p.O_part = static_cast<float*>(workspace);
  p.LSE_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.lse_at);
  p.counter = reinterpret_cast<int*>(static_cast<char*>(workspace) + plan.counter_at);
  p.slots = plan.slots;
  p.part_rows = plan.part_rows;
  p.B = c.B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = c.kv_heads;
  p.G = plan.G;
  p.sub_tokens = plan.sub_tokens;
  p.box_tokens = plan.box_tokens;
  p.page_log2 = page_log2(c.page_size);
  p.num_pages = c.num_pages;
  p.table_stride = c.table_stride;
  p.max_len = c.table_width << p.page_log2;
  p.even = plan.even ? 1 : 0;
  p.ctas = plan.ctas;
  p.inv_ctas = 1.0 / plan.ctas;
  p.min_tiles = kMinTiles;
  p.item_keys = plan.narrow ? kItemKeysNarrow : kItemKeys;
  p.causal = causal != 0;
  p.o_half = half_out ? 1 : 0;
  p.narrow = plan.narrow ? 1 : 0;
  p.scale_log2 = scale * kLog2e;
  p.status = fa2host::device_status_word();
  p.timeout_ns = fa2host::wait_timeout_ns();
  if (p.status == nullptr) return FA2_ERR_LAUNCH;
  // columns: items that may be cut; rows: warps for their rows
  constexpr int kMergeRows = fa2dev::kPagedMergeWarps * fa2dev::kPagedMergeRows;
  dim3 merge(static_cast<unsigned>(plan.even ? plan.ctas - 1 : plan.ctas),
             static_cast<unsigned>((plan.part_rows + kMergeRows - 1) / kMergeRows));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!plan.even && cudaMemsetAsync(p.counter, 0, sizeof(int), s) != cudaSuccess) return FA2_ERR_LAUNCH;
  const auto launch = f16 ? fa2host::launch_paged_f16 : fa2host::launch_paged_bf16;
  return launch(c.d, plan.subs, mq, mk, mv, p, static_cast<unsigned>(plan.ctas), merge, s) ==
                 cudaSuccess
             ? FA2_OK
             : FA2_ERR_LAUNCH;
}

namespace {

int check_rotary(const double* inv_freq, int rotary_dim, int d, float mscale) {
  if (rotary_dim < 0 || rotary_dim > d || rotary_dim % 2 != 0) return FA2_ERR_SHAPE;
  if (!std::isfinite(mscale)) return FA2_ERR_SCALE;
  if (rotary_dim > 0 && !inv_freq) return FA2_ERR_NULL;
  if (misaligned(inv_freq, 7)) return FA2_ERR_ALIGN;
  return FA2_OK;
}

// Whole vectors fill the rotated columns (their halves, unless interleaved) and the rest.
bool wide_rotary(int d, int r, bool interleaved, int elem) {
  const int w = fa2host::rope_width(elem, interleaved);
  return d % w == 0 && (interleaved ? r % w == 0 : r % (2 * w) == 0);
}

}  // namespace

extern "C" int fa2_rope(const void* X, const long long* x_strides, void* Y, const long long* y_strides, int B, int H,
                        int N, int d, const void* positions, int positions_int64, long long positions_batch_stride,
                        const double* inv_freq, int rotary_dim, int interleaved, float mscale, int transposed,
                        int dtype, fa2_stream_t stream) {
  if (dtype != FA2_DTYPE_BF16 && dtype != FA2_DTYPE_FP16 && dtype != FA2_DTYPE_FP32) return FA2_ERR_DTYPE;
  if (B < 0 || H < 0 || N < 0 || d < 1) return FA2_ERR_SHAPE;
  if (d > 1024 || d % 2 != 0) return FA2_ERR_HEADDIM;
  if (B == 0 || H == 0 || N == 0) return FA2_OK;
  int rc = check_rotary(inv_freq, rotary_dim, d, mscale);
  if (rc != FA2_OK) return rc;
  if (!X || !Y || !positions || !x_strides || !y_strides) return FA2_ERR_NULL;
  const int elem = dtype == FA2_DTYPE_FP32 ? 4 : 2;
  const long long sizes[3] = {B, H, N};
  long long xs[3], ys[3];
  const int vec = fa2host::rope_width(elem, interleaved != 0) * elem;   // bytes
  bool wide = wide_rotary(d, rotary_dim, interleaved != 0, elem) && !misaligned(X, vec - 1) && !misaligned(Y, vec - 1);
  bool pairs = !misaligned(X, 2 * elem - 1) && !misaligned(Y, 2 * elem - 1);
  for (int i = 0; i < 3; ++i) {
    xs[i] = sizes[i] > 1 ? x_strides[i] : 0;
    ys[i] = sizes[i] > 1 ? y_strides[i] : 0;
    // reading the same row twice is fine, writing it twice is not
    if (xs[i] < 0 || xs[i] > kMaxStride || (sizes[i] > 1 && (ys[i] < d || ys[i] > kMaxStride))) return FA2_ERR_SHAPE;
    wide = wide && xs[i] * elem % vec == 0 && ys[i] * elem % vec == 0;
    pairs = pairs && xs[i] % 2 == 0 && ys[i] % 2 == 0;
  }
  if (misaligned(X, elem - 1) || misaligned(Y, elem - 1) || misaligned(positions, positions_int64 ? 7 : 3) ||
      (interleaved && !wide && !pairs))
    return FA2_ERR_ALIGN;
  if (!rows_apart(sizes, ys, d)) return FA2_ERR_SHAPE;
  const long long ps = B > 1 ? positions_batch_stride : 0;
  if (ps < 0 || ps > kMaxStride) return FA2_ERR_SHAPE;
  if ((rc = fa2host::require_device()) != FA2_OK) return rc;
  const long long pos_sizes[1] = {B}, pos_strides[1] = {ps};
  const long long xe = extent(sizes, xs, d), ye = extent(sizes, ys, d);
  if (!range_ok(X, xe, elem) || !range_ok(Y, ye, elem) ||
      !range_ok(positions, extent(pos_sizes, pos_strides, N), positions_int64 ? 8 : 4) ||
      (rotary_dim > 0 && !range_ok(inv_freq, rotary_dim / 2, 8)))
    return FA2_ERR_MEMORY;
  // in place, or apart: never shifted against each other
  const bool in_place = X == Y && xs[0] == ys[0] && xs[1] == ys[1] && xs[2] == ys[2];
  const char *x0 = static_cast<const char*>(X), *y0 = static_cast<const char*>(Y);
  if (!in_place && x0 < y0 + ye * elem && y0 < x0 + xe * elem) return FA2_ERR_MEMORY;

  fa2dev::RopeParams p = {};
  p.x = X;
  p.y = Y;
  p.positions = positions;
  p.pos64 = positions_int64 != 0;
  p.pos_batch = ps;
  p.N = N;
  p.x_batch = xs[0]; p.x_head = xs[1]; p.x_token = xs[2];
  p.y_batch = ys[0]; p.y_head = ys[1]; p.y_token = ys[2];
  p.inv_freq = inv_freq;
  p.d = d;
  p.r = rotary_dim;
  p.interleaved = interleaved != 0;
  p.transposed = transposed != 0;
  p.mscale = mscale;
  p.total_tokens = static_cast<long long>(B) * N;
  p.total_rows = H;
  return fa2host::launch_rope(p, false, dtype, wide, fa2host::device_sms(), reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? FA2_OK
             : FA2_ERR_LAUNCH;
}

extern "C" int fa2_append_paged(const fa2_paged_cache* cache, const void* K, const long long* k_strides, const void* V,
                                const long long* v_strides, const void* Q, const long long* q_strides, void* Q_out,
                                const long long* q_out_strides, int Hq, const int* cu_q, int T,
                                const double* inv_freq, int rotary_dim, int interleaved, float mscale,
                                fa2_stream_t stream) {
  if (!cache) return FA2_ERR_NULL;
  if (T < 0 || Hq < 0) return FA2_ERR_SHAPE;
  if (T == 0 || cache->B == 0) return FA2_OK;
  int rc = check_cache(cache);
  if (rc != FA2_OK) return rc;
  const fa2_paged_cache& c = *cache;
  if (!cu_q && T != c.B) return FA2_ERR_SHAPE;
  if (Hq > (1 << 20) || c.kv_heads > (1 << 20)) return FA2_ERR_SHAPE;
  if ((rc = check_rotary(inv_freq, rotary_dim, c.d, mscale)) != FA2_OK) return rc;
  if (!k_strides || !v_strides) return FA2_ERR_NULL;
  if ((rc = check_rows(K, k_strides[0], k_strides[1], T, c.kv_heads, c.d)) != FA2_OK) return rc;
  if ((rc = check_rows(V, v_strides[0], v_strides[1], T, c.kv_heads, c.d)) != FA2_OK) return rc;
  if (Hq > 0) {
    if (!q_strides || !q_out_strides) return FA2_ERR_NULL;
    if ((rc = check_rows(Q, q_strides[0], q_strides[1], T, Hq, c.d)) != FA2_OK) return rc;
    if ((rc = check_rows(Q_out, q_out_strides[0], q_out_strides[1], T, Hq, c.d)) != FA2_OK) return rc;
  }
  if (misaligned(cu_q, 3)) return FA2_ERR_ALIGN;
  const long long page_sizes[3] = {c.num_pages, c.kv_heads, c.page_size};
  const long long page_strides[3] = {c.page_stride, c.head_stride, c.slot_stride};
  if (!rows_apart(page_sizes, page_strides, c.d)) return FA2_ERR_SHAPE;
  if (Hq > 0) {
    const long long out_sizes[2] = {T, Hq}, out_strides[2] = {q_out_strides[0], q_out_strides[1]};
    if (!rows_apart(out_sizes, out_strides, c.d)) return FA2_ERR_SHAPE;
  }
  if ((rc = fa2host::require_device()) != FA2_OK) return rc;
  if ((rc = check_cache_memory(cache)) != FA2_OK) return rc;
  if (!rows_in_memory(K, k_strides[0], k_strides[1], T, c.kv_heads, c.d) ||
      !rows_in_memory(V, v_strides[0], v_strides[1], T, c.kv_heads, c.d) ||
      (Hq > 0 && (!rows_in_memory(Q, q_strides[0], q_strides[1], T, Hq, c.d) ||
                  !rows_in_memory(Q_out, q_out_strides[0], q_out_strides[1], T, Hq, c.d))) ||
      (cu_q && !range_ok(cu_q, c.B + 1ll, 4)) || (rotary_dim > 0 && !range_ok(inv_freq, rotary_dim / 2, 8)))
    return FA2_ERR_MEMORY;
  fa2dev::RopeParams p = {};
  p.q = Q;
  p.k = K;
  p.v = V;
  p.q_out = Q_out;
  p.k_pages = c.k_pages;
  p.v_pages = c.v_pages;
  p.k_token = k_strides[0]; p.k_head = k_strides[1];
  p.v_token = v_strides[0]; p.v_head = v_strides[1];
  if (Hq > 0) {
    p.q_token = q_strides[0]; p.q_head = q_strides[1];
    p.qo_token = q_out_strides[0]; p.qo_head = q_out_strides[1];
    const long long sizes[2] = {T, Hq};
    const long long qs[2] = {T > 1 ? p.q_token : 0, Hq > 1 ? p.q_head : 0};
    const long long os[2] = {T > 1 ? p.qo_token : 0, Hq > 1 ? p.qo_head : 0};
    const bool in_place = Q == Q_out && qs[0] == os[0] && qs[1] == os[1];
    const char *x0 = static_cast<const char*>(Q), *y0 = static_cast<const char*>(Q_out);
    if (!in_place && x0 < y0 + extent(sizes, os, c.d) * 2 && y0 < x0 + extent(sizes, qs, c.d) * 2)
      return FA2_ERR_MEMORY;
  }
  p.page_stride = c.page_stride;
  p.page_head = c.head_stride;
  p.slot_stride = c.slot_stride;
  p.page_table = c.page_table;
  p.kv_lens = c.kv_lens;
  p.cu_q = cu_q;
  p.table_stride = c.table_stride;
  p.B = c.B;
  p.Hq = Hq;
  p.Hkv = c.kv_heads;
  p.page_log2 = page_log2(c.page_size);
  p.num_pages = c.num_pages;
  p.max_len = c.table_width << p.page_log2;
  p.status = fa2host::device_status_word();
  if (p.status == nullptr) return FA2_ERR_LAUNCH;
  p.inv_freq = inv_freq;
  p.d = c.d;
  p.r = rotary_dim;
  p.interleaved = interleaved != 0;
  p.mscale = mscale;
  p.total_tokens = T;
  p.total_rows = Hq + 2 * c.kv_heads;
  const bool wide = wide_rotary(c.d, rotary_dim, interleaved != 0, 2);
  return fa2host::launch_rope(p, true, c.dtype, wide, fa2host::device_sms(),
                              reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA2_OK
             : FA2_ERR_LAUNCH;
}

namespace {

int check_tables(const fa2_page_tables* t) {
  if (!t) return FA2_ERR_NULL;
  if (t->B < 0 || t->table_width < 1 || t->num_pages < 1 || t->num_pages > fa2dev::kMaxPoolPages ||
      page_log2(t->page_size) < 0 || static_cast<long long>(t->table_width) * t->page_size > (1ll << 30) ||
      (t->B > 1 && (t->table_stride < t->table_width || t->table_stride > kMaxStride)))
    return FA2_ERR_SHAPE;
  if (t->B > 0 && (!t->page_table || !t->lens || !t->refs)) return FA2_ERR_NULL;
  if (misaligned(t->page_table, 3) || misaligned(t->lens, 3) || misaligned(t->refs, 3)) return FA2_ERR_ALIGN;
  return FA2_OK;
}

int check_tables_memory(const fa2_page_tables* t) {
  const long long sizes[1] = {t->B}, strides[1] = {t->B > 1 ? t->table_stride : 0};
  return range_ok(t->page_table, extent(sizes, strides, t->table_width), 4) && range_ok(t->lens, t->B, 4) &&
                 range_ok(t->refs, t->num_pages, 4)
             ? FA2_OK
             : FA2_ERR_MEMORY;
}

int check_pools(const fa2_page_pools* d) {
  if (!d) return FA2_ERR_NULL;
  if (d->num_planes < 0 || d->num_planes > fa2dev::kMaxPlanes || d->num_pages < 1 || d->page_bytes < 16 ||
      d->page_bytes > kMaxStride || (d->num_pages > 1 && (d->page_stride < d->page_bytes || d->page_stride > kMaxStride)))
    return FA2_ERR_SHAPE;
  if (d->num_planes > 0 && !d->planes) return FA2_ERR_NULL;
  if (d->page_bytes % 16 != 0 || (d->num_pages > 1 && d->page_stride % 16 != 0)) return FA2_ERR_ALIGN;
  for (int i = 0; i < d->num_planes; ++i) {
    if (!d->planes[i]) return FA2_ERR_NULL;
    if (misaligned(d->planes[i], 15)) return FA2_ERR_ALIGN;
  }
  return FA2_OK;
}

int check_pools_memory(const fa2_page_pools* d) {
  const long long sizes[1] = {d->num_pages}, strides[1] = {d->num_pages > 1 ? d->page_stride : 0};
  const long long e = extent(sizes, strides, d->page_bytes);
  // planes in ascending order within one allocation (a pool of all layers): one look
  bool ascending = d->num_planes > 1;
  for (int i = 1; i < d->num_planes; ++i) ascending = ascending && d->planes[i] > d->planes[i - 1];
  if (ascending && e >= 0) {
    const char *first = static_cast<const char*>(d->planes[0]), *last = static_cast<const char*>(d->planes[d->num_planes - 1]);
    if (range_ok(first, last - first + e, 1)) return FA2_OK;
  }
  for (int i = 0; i < d->num_planes; ++i)
    if (!range_ok(d->planes[i], e, 1)) return FA2_ERR_MEMORY;
  return FA2_OK;
}

fa2dev::PageTables device_tables(const fa2_page_tables* t) {
  fa2dev::PageTables o;
  o.table = t->page_table;
  o.table_stride = t->table_stride;
  o.width = t->table_width;
  o.B = t->B;
  o.lens = t->lens;
  o.refs = t->refs;
  o.num_pages = t->num_pages;
  o.page_log2 = page_log2(t->page_size);
  o.status = fa2host::device_status_word();
  return o;
}

fa2dev::PagePlanes device_planes(const fa2_page_pools* d) {
  fa2dev::PagePlanes o;
  for (int i = 0; i < fa2dev::kMaxPlanes; ++i) o.base[i] = i < d->num_planes ? d->planes[i] : nullptr;
  o.stride = d->page_stride;
  o.page_bytes = d->page_bytes;
  o.planes = d->num_planes;
  o.num_pages = d->num_pages;
  return o;
}

int check_workspace(const void* ws, size_t size, size_t ints) {
  if (!ws) return FA2_ERR_NULL;
  if (misaligned(ws, 15)) return FA2_ERR_ALIGN;
  return size >= ints * 4 && fa2host::device_memory_ok(ws, ints * 4) ? FA2_OK : FA2_ERR_MEMORY;
}

// a list of n ints on the device
int check_list(const int* p, int n) {
  if (!p) return FA2_ERR_NULL;
  if (misaligned(p, 3)) return FA2_ERR_ALIGN;
  return range_ok(p, n, 4) ? FA2_OK : FA2_ERR_MEMORY;
}

size_t reserve_ints(int num_pages) { return static_cast<size_t>(num_pages); }
size_t fork_ints(int n) { return 1 + 3 * static_cast<size_t>(n); }
size_t compact_ints(int num_pages) { return 1 + 2 * static_cast<size_t>(num_pages); }
size_t copy_ints(int n) { return 1 + 2 * static_cast<size_t>(n); }

int launched(cudaError_t e) { return e == cudaSuccess ? FA2_OK : FA2_ERR_LAUNCH; }

// The lists are searched for indices named twice, each entry against all: copies of
// 1 KB take 22 us for 1024 pairs, 52 for 4096, 294 for 16384 and 3.6 ms for 65536;
// freeing as many sequences 10 us, 14, 55 and 0.76 ms.
constexpr int kMaxPairs = 1 << 16;

}  // namespace

extern "C" size_t fa2_pages_workspace_bytes(int num_pages, int n) {
  if (num_pages < 0 || n < 0 || num_pages > fa2dev::kMaxPoolPages || n > kMaxPairs) return 0;
  const size_t a = compact_ints(num_pages), b = fork_ints(n);
  return align256((a > b ? a : b) * 4);
}

extern "C" int fa2_pages_reserve(const fa2_page_tables* tables, const int* add, int* missing, void* workspace,
                                 size_t workspace_size, fa2_stream_t stream) {
  int rc = check_tables(tables);
  if (rc != FA2_OK) return rc;
  if (!missing) return FA2_ERR_NULL;
  if (tables->B > 0 && !add) return FA2_ERR_NULL;
  if ((rc = fa2host::require_device()) != FA2_OK) return rc;
  if (tables->B > 0 && ((rc = check_tables_memory(tables)) != FA2_OK || (rc = check_list(add, tables->B)) != FA2_OK))
    return rc;
  if ((rc = check_list(missing, 1)) != FA2_OK) return rc;
  if ((rc = check_workspace(workspace, workspace_size, reserve_ints(tables->num_pages))) != FA2_OK) return rc;
  const fa2dev::PageTables t = device_tables(tables);
  if (t.status == nullptr) return FA2_ERR_LAUNCH;
  return launched(fa2host::launch_pages_reserve(t, add, missing, static_cast<int*>(workspace),
                                                reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" int fa2_pages_fork(const fa2_page_tables* tables, const fa2_page_pools* pools, const int* src,
                              const int* dst, int n, int* missing, void* workspace, size_t workspace_size,
                              fa2_stream_t stream) {
  int rc = check_tables(tables);
  if (rc != FA2_OK) return rc;
  if ((rc = check_pools(pools)) != FA2_OK) return rc;
  if (n < 0 || n > kMaxPairs || pools->num_pages != tables->num_pages) return FA2_ERR_SHAPE;
  if (!missing || (n > 0 && (!src || !dst))) return FA2_ERR_NULL;
  if ((rc = fa2host::require_device()) != FA2_OK) return rc;
  if (tables->B > 0 && (rc = check_tables_memory(tables)) != FA2_OK) return rc;
  if ((rc = check_pools_memory(pools)) != FA2_OK) return rc;
  if (n > 0 && ((rc = check_list(src, n)) != FA2_OK || (rc = check_list(dst, n)) != FA2_OK)) return rc;
  if ((rc = check_list(missing, 1)) != FA2_OK) return rc;
  if ((rc = check_workspace(workspace, workspace_size, fork_ints(n))) != FA2_OK) return rc;
  const fa2dev::PageTables t = device_tables(tables);
  if (t.status == nullptr) return FA2_ERR_LAUNCH;
  return launched(fa2host::launch_pages_fork(t, src, dst, n, device_planes(pools), missing, static_cast<int*>(workspace),
                                             fa2host::device_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" int fa2_pages_free(const fa2_page_tables* tables, const int* seqs, int n, fa2_stream_t stream) {
  int rc = check_tables(tables);
  if (rc != FA2_OK) return rc;
  if (n < 0 || n > kMaxPairs) return FA2_ERR_SHAPE;
  if (n == 0) return FA2_OK;
  if (!seqs) return FA2_ERR_NULL;
  if ((rc = fa2host::require_device()) != FA2_OK) return rc;
  if ((tables->B > 0 && (rc = check_tables_memory(tables)) != FA2_OK) || (rc = check_list(seqs, n)) != FA2_OK) return rc;
  const fa2dev::PageTables t = device_tables(tables);
  if (t.status == nullptr) return FA2_ERR_LAUNCH;
  return launched(fa2host::launch_pages_free(t, seqs, n, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" int fa2_pages_compact(const fa2_page_tables* tables, const fa2_page_pools* pools, int* moved,
                                 void* workspace, size_t workspace_size, fa2_stream_t stream) {
  int rc = check_tables(tables);
  if (rc != FA2_OK) return rc;
  if ((rc = check_pools(pools)) != FA2_OK) return rc;
  if (pools->num_pages != tables->num_pages) return FA2_ERR_SHAPE;
  if (!moved) return FA2_ERR_NULL;
  if (!tables->refs) return FA2_ERR_NULL;
  if ((rc = fa2host::require_device()) != FA2_OK) return rc;
  if (tables->B > 0 && (rc = check_tables_memory(tables)) != FA2_OK) return rc;
  if ((rc = check_list(tables->refs, tables->num_pages)) != FA2_OK) return rc;
  if ((rc = check_pools_memory(pools)) != FA2_OK) return rc;
  if ((rc = check_list(moved, tables->num_pages)) != FA2_OK) return rc;
  if ((rc = check_workspace(workspace, workspace_size, compact_ints(tables->num_pages))) != FA2_OK) return rc;
  const fa2dev::PageTables t = device_tables(tables);
  if (t.status == nullptr) return FA2_ERR_LAUNCH;
  return launched(fa2host::launch_pages_compact(t, device_planes(pools), moved, static_cast<int*>(workspace),
                                                fa2host::device_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" int fa2_pages_copy(const fa2_page_pools* pools, const int* src, const int* dst, int n, void* workspace,
                              size_t workspace_size, fa2_stream_t stream) {
  int rc = check_pools(pools);
  if (rc != FA2_OK) return rc;
  if (n < 0 || n > kMaxPairs) return FA2_ERR_SHAPE;
  if (n == 0) return FA2_OK;
  if (!src || !dst) return FA2_ERR_NULL;
  if ((rc = fa2host::require_device()) != FA2_OK) return rc;
  if ((rc = check_pools_memory(pools)) != FA2_OK || (rc = check_list(src, n)) != FA2_OK ||
      (rc = check_list(dst, n)) != FA2_OK)
    return rc;
  if ((rc = check_workspace(workspace, workspace_size, copy_ints(n))) != FA2_OK) return rc;
  int* status = fa2host::device_status_word();
  if (status == nullptr) return FA2_ERR_LAUNCH;
  return launched(fa2host::launch_pages_copy(device_planes(pools), src, dst, n, static_cast<int*>(workspace), status,
                                             fa2host::device_sms(), reinterpret_cast<cudaStream_t>(stream)));
}
