// Attention over a paged cache: f16 inputs (head dimensions 64, 128, 256; one
// or two query sub-tiles per CTA, or one of at most 32 rows).
#include "fa2_launch.h"

namespace fa2host {

namespace {
constexpr bool kF16 = true;

template <int D, int SUBS, bool NARROW>
cudaError_t set_limits() {
  return cudaFuncSetAttribute(fa2dev::fa2_paged_tc_kernel<D, kF16, SUBS, NARROW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              fa2dev::PagedConfig<D, SUBS>::kSmemBytes);
}

template <int D, int SUBS, bool NARROW>
cudaError_t run(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const fa2dev::PagedParams& p,
                unsigned grid, dim3 merge_grid, cudaStream_t s) {
  const auto kernel = fa2dev::fa2_paged_tc_kernel<D, kF16, SUBS, NARROW>;
  constexpr int kThreads = fa2dev::FwdShape<SUBS>::kThreads;
  constexpr unsigned kSmem = fa2dev::PagedConfig<D, SUBS>::kSmemBytes;
  cudaError_t e;
  if (p.even) {
    e = launch_behind(kernel, dim3(grid), kThreads, kSmem, s, mq, mk, mv, p);
  } else {   // (behind the counter's memset)
    kernel<<<grid, kThreads, kSmem, s>>>(mq, mk, mv, p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || merge_grid.x == 0) return e;
  return launch_behind(fa2dev::fa2_paged_merge_kernel<D, kF16, SUBS>, merge_grid, fa2dev::kPagedMergeWarps * 32, 0, s, p);
}
}  // namespace

cudaError_t prepare_paged_f16() {
  cudaError_t e;
  if ((e = set_limits<64, 1, false>()) != cudaSuccess || (e = set_limits<64, 2, false>()) != cudaSuccess ||
      (e = set_limits<128, 1, false>()) != cudaSuccess || (e = set_limits<128, 2, false>()) != cudaSuccess ||
      (e = set_limits<256, 1, false>()) != cudaSuccess || (e = set_limits<64, 1, true>()) != cudaSuccess ||
      (e = set_limits<128, 1, true>()) != cudaSuccess)
    return e;
  return set_limits<256, 1, true>();
}

cudaError_t launch_paged_f16(int d, int subs, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                              const fa2dev::PagedParams& p, unsigned grid, dim3 merge_grid, cudaStream_t s) {
  const auto f = p.narrow ? (d == 64 ? run<64, 1, true> : d == 128 ? run<128, 1, true> : run<256, 1, true>)
                 : d == 64 ? (subs == 1 ? run<64, 1, false> : run<64, 2, false>)
                 : d == 128 ? (subs == 1 ? run<128, 1, false> : run<128, 2, false>)
                            : run<256, 1, false>;
  return f(mq, mk, mv, p, grid, merge_grid, s);
}

}  // namespace fa2host
