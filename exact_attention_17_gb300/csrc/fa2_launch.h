// Internal: launch entry points of the kernel translation units.  Each .cu
// file instantiates one family of kernels so that they compile in parallel.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "fa2_bwd2_sm103.cuh"
#include "fa2_bwd_sm103.cuh"
#include "fa2_fwd_simt.cuh"
#include "fa2_fwd_pair_sm103.cuh"
#include "fa2_fwd_sm103.cuh"
#include "fa2_paged_sm103.cuh"

namespace fa2host {

// Launches a kernel that may start while the one before it on the stream still
// runs (when that one allows it, griddepcontrol.launch_dependents).  Every block
// waits for the one before to end (griddepcontrol.wait) before it writes, and
// before it reads what others may write, so that "complete" reaches back along the
// stream.  Kernels that read earlier: the merge of the paged attention looks up
// lengths and offsets first.  They are complete by then, because the kernel before
// it, which writes neither, lets it start only behind its own wait; a kernel that
// is to do the same has to be behind one that keeps this order.  With shared prefixes
// the launch over the sequences' own pages runs beside the groups' (which starts it behind its
// own wait, and whose results it does not touch) and waits for it at its end; the kernel that
// joins them looks up offsets and groups first, as the merge does.
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, int threads, unsigned smem, cudaStream_t s,
                          const Args&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Raise the dynamic shared-memory limit of every kernel in the unit (current device).
cudaError_t prepare_tc_d64_bf16();
cudaError_t prepare_tc_d128_bf16();
cudaError_t prepare_tc_d64_f16();
cudaError_t prepare_tc_d128_f16();
cudaError_t prepare_tc_d256_bf16();
cudaError_t prepare_tc_d256_f16();
cudaError_t prepare_simt();

// subs: query sub-tiles of 128 rows per CTA (1 or 2; head dimension 256: 1).  mo: the map the epilogue stores O (or
// the split-KV partial O) through.
#define FA2_DECLARE_TC_LAUNCH(name)                                                          \
  cudaError_t name(int subs, bool causal, const CUtensorMap& mq, const CUtensorMap& mk,      \
                   const CUtensorMap& mv, const CUtensorMap& mo, const fa2dev::FwdParams& p, \
                   unsigned grid, cudaStream_t s);
FA2_DECLARE_TC_LAUNCH(launch_tc_d64_bf16)
FA2_DECLARE_TC_LAUNCH(launch_tc_d128_bf16)
FA2_DECLARE_TC_LAUNCH(launch_tc_d64_f16)
FA2_DECLARE_TC_LAUNCH(launch_tc_d128_f16)
FA2_DECLARE_TC_LAUNCH(launch_tc_d256_bf16)
FA2_DECLARE_TC_LAUNCH(launch_tc_d256_f16)
#undef FA2_DECLARE_TC_LAUNCH
cudaError_t launch_simt(int d, bool causal, const fa2dev::SimtParams& p, dim3 grid, cudaStream_t s);

// Two-SM forward (clusters of two CTAs), head dimension 128.  mk_half: K with
// 64-row boxes; mq, mv: 128-row boxes.  grid: an even number of CTAs.
cudaError_t prepare_tc_pair_d128();
cudaError_t launch_tc_pair_d128(bool causal, bool f16, const CUtensorMap& mq, const CUtensorMap& mk_half,
                                const CUtensorMap& mv, const CUtensorMap& mo, const fa2dev::FwdParams& p,
                                unsigned grid, cudaStream_t s);

// Merge of S partial results (normalised O [S, R, d], LSE [S, R]) into O [R, d], LSE [R].
cudaError_t launch_combine(int d, const float* O_part, const float* LSE_part, int S, long long R,
                           float* O, float* LSE, cudaStream_t s);

// Backward pass (fa2_bwd.cu).
cudaError_t prepare_bwd();
// mdq: fp32 [BH][Nq][d] map of dQ, 32-column boxes, 128-byte swizzle (TMA reductions).
// f16: Q, K, V and dO are fp16 (else bf16).
cudaError_t launch_bwd(int d, bool causal, bool f16, const CUtensorMap& mq, const CUtensorMap& mk,
                       const CUtensorMap& mv, const CUtensorMap& mdo, const CUtensorMap& mdq,
                       const fa2dev::BwdParams& p, unsigned grid, cudaStream_t s);
// D_i = dO_i . O_i and LSE_i log2(e) into [BH][Nq_pad] arrays; dQ rows zeroed.
cudaError_t launch_bwd_pre(int d, bool f16, const float* O, const void* dO, const float* LSE, float* dQ,
                           float* L2, float* Dr, long long rows, int Nq, int Nq_pad, cudaStream_t s);
cudaError_t launch_zero(float* p, long long n, cudaStream_t s);

// Two-tile backward kernel (fa2_bwd2.cu), head dimension 128.  mq64, mdo64:
// 64-row boxes; mk, mv: 128-row boxes; mdq32: fp32 dQ with 32 x 32 boxes.
cudaError_t prepare_bwd2();
cudaError_t launch_bwd2(bool causal, bool f16, const CUtensorMap& mq64, const CUtensorMap& mk,
                        const CUtensorMap& mv, const CUtensorMap& mdo64, const CUtensorMap& mdq32,
                        const fa2dev::BwdParams& p, unsigned grid, cudaStream_t s);

// Windows (fa2_window_bf16.cu, fa2_window_f16.cu, fa2_bwd_window.cu).
cudaError_t prepare_window_bf16();
cudaError_t prepare_window_f16();
cudaError_t launch_window_bf16(int d, int subs, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                               const CUtensorMap& mo, const fa2dev::FwdParams& p, unsigned grid, cudaStream_t s);
cudaError_t launch_window_f16(int d, int subs, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                              const CUtensorMap& mo, const fa2dev::FwdParams& p, unsigned grid, cudaStream_t s);
cudaError_t prepare_bwd_window();
// The pre-pass of the gradients, as launch_bwd_pre (o_half: O has the input type, else fp32).
cudaError_t launch_bwd_window_pre(int d, bool f16, bool o_half, const void* O, const void* dO, const float* LSE,
                                  float* dQ, float* L2, float* Dr, long long rows, int Nq, int Nq_pad, cudaStream_t s);
cudaError_t launch_bwd_window(int d, bool f16, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                              const CUtensorMap& mdo, const CUtensorMap& mdq, const fa2dev::BwdParams& p, unsigned grid,
                              cudaStream_t s);
// Behind it: dK and dV of key blocks cut into several items, and dQ (fp32, q_elems) into the 16-bit dq_out
// unless that is null.
cudaError_t launch_bwd_window_end(int d, bool f16, const fa2dev::BwdParams& p, void* dq_out, long long q_elems,
                                  cudaStream_t s);

// Attention over a paged cache (fa2_paged_bf16.cu, fa2_paged_f16.cu): the
// partial or final results, then the merge of items cut into key ranges
// (merge_grid.x = 0: no item can be cut).
cudaError_t prepare_paged_bf16();
cudaError_t prepare_paged_f16();
cudaError_t launch_paged_bf16(int d, int subs, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                              const fa2dev::PagedParams& p, unsigned grid, dim3 merge_grid, cudaStream_t s);
cudaError_t launch_paged_f16(int d, int subs, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                             const fa2dev::PagedParams& p, unsigned grid, dim3 merge_grid, cudaStream_t s);

// The same with windows or shared prefixes (fa2_paged_ext_bf16.cu, fa2_paged_ext_f16.cu).
cudaError_t prepare_paged_ext_bf16();
cudaError_t prepare_paged_ext_f16();
cudaError_t launch_paged_ext_bf16(int d, int subs, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                  const fa2dev::PagedParams& p, unsigned grid, dim3 merge_grid, cudaStream_t s);
cudaError_t launch_paged_ext_f16(int d, int subs, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                 const fa2dev::PagedParams& p, unsigned grid, dim3 merge_grid, cudaStream_t s);
// Shared prefixes: behind the groups' launch (p0) and the sequences' own (p1), what joins their results into O
// (half_out: in the input type) and LSE (fa2_paged_prefix.cu).
cudaError_t launch_paged_join(int d, bool f16, const fa2dev::PagedParams& p0, int subs0, const fa2dev::PagedParams& p1,
                              int subs1, void* O, float* LSE, bool half_out, cudaStream_t s);

}  // namespace fa2host
