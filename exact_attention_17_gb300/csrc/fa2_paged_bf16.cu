// Attention over a paged cache: bf16 inputs (head dimensions 64, 128, 256; one
// or two query sub-tiles per CTA).
#include "fa2_launch.h"

namespace fa2host {

namespace {
constexpr bool kF16 = false;

template <int D, int SUBS>
cudaError_t set_limits() {
  return cudaFuncSetAttribute(fa2dev::fa2_paged_tc_kernel<D, kF16, SUBS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              fa2dev::FwdConfig<D, SUBS>::kSmemBytes);
}

template <int D, int SUBS>
cudaError_t run(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const fa2dev::PagedParams& p,
                unsigned grid, unsigned merge_grid, cudaStream_t s) {
  fa2dev::fa2_paged_tc_kernel<D, kF16, SUBS>
      <<<grid, fa2dev::FwdShape<SUBS>::kThreads, fa2dev::FwdConfig<D, SUBS>::kSmemBytes, s>>>(mq, mk, mv, p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || merge_grid == 0) return e;
  fa2dev::fa2_paged_merge_kernel<D, kF16, SUBS><<<merge_grid, fa2dev::kPagedMergeWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}
}  // namespace

cudaError_t prepare_paged_bf16() {
  cudaError_t e;
  if ((e = set_limits<64, 1>()) != cudaSuccess || (e = set_limits<64, 2>()) != cudaSuccess ||
      (e = set_limits<128, 1>()) != cudaSuccess || (e = set_limits<128, 2>()) != cudaSuccess)
    return e;
  return set_limits<256, 1>();
}

cudaError_t launch_paged_bf16(int d, int subs, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                              const fa2dev::PagedParams& p, unsigned grid, unsigned merge_grid, cudaStream_t s) {
  if (d == 64)
    return subs == 1 ? run<64, 1>(mq, mk, mv, p, grid, merge_grid, s) : run<64, 2>(mq, mk, mv, p, grid, merge_grid, s);
  if (d == 128)
    return subs == 1 ? run<128, 1>(mq, mk, mv, p, grid, merge_grid, s) : run<128, 2>(mq, mk, mv, p, grid, merge_grid, s);
  return run<256, 1>(mq, mk, mv, p, grid, merge_grid, s);
}

}  // namespace fa2host
