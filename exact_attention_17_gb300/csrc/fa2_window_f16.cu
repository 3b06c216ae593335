// Forward kernels of windows: fp16 inputs (head dimensions 64, 128, 256; one or
// two query sub-tiles per CTA).
#include "fa2_launch.h"

namespace fa2host {

namespace {
constexpr bool kF16 = true;

template <int D, int SUBS>
cudaError_t set_limits() {
  return cudaFuncSetAttribute(fa2dev::fa2_fwd_tc_kernel<D, true, kF16, SUBS, true>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, fa2dev::FwdConfig<D, SUBS>::kSmemBytes);
}

template <int D, int SUBS>
cudaError_t run(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                const fa2dev::FwdParams& p, unsigned grid, cudaStream_t s) {
  return launch_behind(fa2dev::fa2_fwd_tc_kernel<D, true, kF16, SUBS, true>, dim3(grid), fa2dev::FwdShape<SUBS>::kThreads,
                       fa2dev::FwdConfig<D, SUBS>::kSmemBytes, s, mq, mk, mv, mo, p);
}
}  // namespace

cudaError_t prepare_window_f16() {
  cudaError_t e;
  if ((e = set_limits<64, 1>()) != cudaSuccess || (e = set_limits<64, 2>()) != cudaSuccess ||
      (e = set_limits<128, 1>()) != cudaSuccess || (e = set_limits<128, 2>()) != cudaSuccess)
    return e;
  return set_limits<256, 1>();
}

cudaError_t launch_window_f16(int d, int subs, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                               const CUtensorMap& mo, const fa2dev::FwdParams& p, unsigned grid, cudaStream_t s) {
  const auto f = d == 64 ? (subs == 1 ? run<64, 1> : run<64, 2>)
                 : d == 128 ? (subs == 1 ? run<128, 1> : run<128, 2>) : run<256, 1>;
  return f(mq, mk, mv, mo, p, grid, s);
}

}  // namespace fa2host
