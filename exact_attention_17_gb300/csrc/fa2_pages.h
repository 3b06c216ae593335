// Internal: the page-management kernels' launches (fa2_pages.cu).
#pragma once

#include <cuda_runtime.h>

#include "fa2.h"
#include "fa2_paged_sm103.cuh"

namespace fa2dev {

constexpr int kMaxPlanes = 256;
constexpr int kMaxPoolPages = (1 << 21) - 1;   // pages that the planning block ranks

// Where the page data is: `planes` arrays of pages of `page_bytes` bytes.
struct PagePlanes {
  void* base[kMaxPlanes];
  long long stride;      // bytes from one page to the next
  long long page_bytes;  // a multiple of 16
  int planes;
  int num_pages;
};

// The tables: int32 [B, width] (row stride table_stride), lens [B], refs [num_pages].
struct PageTables {
  int* table;
  long long table_stride;
  int width;
  int B;
  int* lens;
  int* refs;
  int num_pages;
  int page_log2;
  int* status;
};

}  // namespace fa2dev

namespace fa2host {

// ws (ints): reserve num_pages; fork 1 + 3 n; compact 1 + 2 num_pages; copy 1 + 2 n.
cudaError_t launch_pages_reserve(const fa2dev::PageTables& t, const int* add, int* missing, int* ws, cudaStream_t s);
cudaError_t launch_pages_fork(const fa2dev::PageTables& t, const int* src, const int* dst, int n,
                              const fa2dev::PagePlanes& d, int* missing, int* ws, int sms, cudaStream_t s);
cudaError_t launch_pages_free(const fa2dev::PageTables& t, const int* seqs, int n, cudaStream_t s);
cudaError_t launch_pages_compact(const fa2dev::PageTables& t, const fa2dev::PagePlanes& d, int* moved, int* ws,
                                 int sms, cudaStream_t s);
cudaError_t launch_pages_copy(const fa2dev::PagePlanes& d, const int* src, const int* dst, int n, int* ws,
                              int* status, int sms, cudaStream_t s);

}  // namespace fa2host
