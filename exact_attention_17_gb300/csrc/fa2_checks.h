// Internal: argument checks that the entry points of the paged cache and its
// neighbours share.  Each unit has its own copy (unnamed namespace).
#pragma once

#include <cmath>
#include <cstdint>

#include "fa2.h"
#include "fa2_host.h"
#include "fa2_rope.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr long long kMaxStride = 1ll << 38;   // elements; TMA strides stay below 2^40 bytes

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline bool misaligned(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

inline int log2_exact(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return (1 << l) == x ? l : -1;
}

inline int page_log2(int page_size) {
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
inline bool rows_apart(const long long (&sizes)[N], const long long (&strides)[N], long long inner) {
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

inline bool range_ok(const void* p, long long elems, int size) {
  return elems >= 0 && fa2host::device_memory_ok(p, static_cast<size_t>(elems) * size);
}

// Everything about a cache that can be checked on the host without a device.
inline int check_cache(const fa2_paged_cache* c) {
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

inline int check_cache_memory(const fa2_paged_cache* c) {
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
inline int check_rows(const void* p, long long token, long long head, long long T, int H, int d) {
  if ((T > 1 && (token < d || token > kMaxStride)) || (H > 1 && (head < d || head > kMaxStride))) return FA2_ERR_SHAPE;
  if (!p) return FA2_ERR_NULL;
  if (misaligned(p, 15) || (T > 1 && token % 8 != 0) || (H > 1 && head % 8 != 0)) return FA2_ERR_ALIGN;
  return FA2_OK;
}

inline bool rows_in_memory(const void* p, long long token, long long head, long long T, int H, int d) {
  const long long sizes[2] = {T, H};
  const long long strides[2] = {T > 1 ? token : 0, H > 1 ? head : 0};
  return range_ok(p, extent(sizes, strides, d), 2);
}

inline int check_rotary(const double* inv_freq, int rotary_dim, int d, float mscale) {
  if (rotary_dim < 0 || rotary_dim > d || rotary_dim % 2 != 0) return FA2_ERR_SHAPE;
  if (!std::isfinite(mscale)) return FA2_ERR_SCALE;
  if (rotary_dim > 0 && !inv_freq) return FA2_ERR_NULL;
  if (misaligned(inv_freq, 7)) return FA2_ERR_ALIGN;
  return FA2_OK;
}

// Whole vectors fill the rotated columns (their halves, unless interleaved) and the rest.
inline bool wide_rotary(int d, int r, bool interleaved, int elem) {
  const int w = fa2host::rope_width(elem, interleaved);
  return d % w == 0 && (interleaved ? r % w == 0 : r % (2 * w) == 0);
}

// Weights of the rows' type or fp32, a finite eps that is not negative.
inline int check_norm(int weight_dtype, int dtype, float eps) {
  if (weight_dtype != FA2_DTYPE_FP32 && weight_dtype != dtype) return FA2_ERR_DTYPE;
  return eps >= 0.f && std::isfinite(eps) ? FA2_OK : FA2_ERR_SCALE;
}

// Whole 16-byte vectors hold the rotated columns (their halves, unless interleaved).
inline bool wide_norm(int r, bool interleaved, int elem) {
  const int w = 16 / elem;
  return interleaved ? r % w == 0 : r % (2 * w) == 0;
}

}  // namespace
