// Attention over a paged cache whose sequences share prefixes: the launches, and
// the kernel that joins a row's two results.
#include "fa2_launch.h"

namespace fa2dev {

// With (O_p, L_p) a row's result over the shared prefix and (O_o, L_o) over its
// sequence's own keys, both normalised: LSE = log(e^L_p + e^L_o), O = e^(L_p - LSE)
// O_p + e^(L_o - LSE) O_o.  A row of a sequence that shares nothing has the second alone.
// A warp takes a token's heads one after the other; whose token it is, and whether that sequence's group has a
// prefix, is looked up as the launches do.
template <int D, bool F16>
__global__ void __launch_bounds__(256) fa2_paged_join_kernel(const __grid_constant__ PagedParams p,
                                                             const float* __restrict__ O_prefix,
                                                             const float* __restrict__ LSE_prefix, void* O, float* LSE,
                                                             int half_out) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = static_cast<int>((blockIdx.x * 256ll + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  const int warps = gridDim.x * 8;
  const float* O_own = static_cast<const float*>(p.O);
  for (long long row = warp; row < static_cast<long long>(p.T) * p.Hq; row += warps) {
    const int t = static_cast<int>(row / p.Hq);
    int b = t;
    if (p.cu_q != nullptr) {   // the last sequence that begins at or before t
      int lo = 0, n = p.B;
      while (n > 1) {
        const int half = n / 2;
        if (p.cu_q[lo + half] <= t) {
          lo += half;
          n -= half;
        } else {
          n = half;
        }
      }
      b = lo;
      if (p.cu_q[b] > t || p.cu_q[b + 1] <= t) continue;   // nobody's
    }
    bool bad = false;
    const int shared = paged_shared(p, p.B, b, &bad);
    const float lo = p.LSE[row];
    float wo = 1.f, wp = 0.f, lse = lo;
    if (shared > 0) {
      const float lp = LSE_prefix[row], m = fmaxf(lo, lp);
      if (m != -INFINITY) {
        const float eo = lo == -INFINITY ? 0.f : expf(lo - m), ep = lp == -INFINITY ? 0.f : expf(lp - m);
        lse = m + logf(eo + ep);
        wo = eo / (eo + ep);
        wp = ep / (eo + ep);
      }
    }
    if (lane == 0) LSE[row] = lse;
#pragma unroll
    for (int c = lane * 4; c < D; c += 128) {
      float4 x = *reinterpret_cast<const float4*>(O_own + row * D + c);
      if (shared > 0) {
        const float4 y = *reinterpret_cast<const float4*>(O_prefix + row * D + c);
        x.x = wo * x.x + wp * y.x;
        x.y = wo * x.y + wp * y.y;
        x.z = wo * x.z + wp * y.z;
        x.w = wo * x.w + wp * y.w;
      }
      if (half_out)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(O) + row * D + c) =
            make_uint2(pack_x2<F16>(x.x, x.y), pack_x2<F16>(x.z, x.w));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(O) + row * D + c) = x;
    }
  }
}

}  // namespace fa2dev

namespace fa2host {

namespace {
template <int D, bool F16>
cudaError_t join(const fa2dev::PagedParams& p, const float* O_prefix, const float* LSE_prefix, void* O, float* LSE,
                 bool half_out, cudaStream_t s) {
  const long long rows = static_cast<long long>(p.T) * p.Hq;
  const long long blocks = (rows + 7) / 8;
  return launch_behind(fa2dev::fa2_paged_join_kernel<D, F16>, dim3(static_cast<unsigned>(blocks < 65535 ? blocks : 65535)),
                       256, 0, s, p, O_prefix, LSE_prefix, O, LSE, half_out ? 1 : 0);
}
}  // namespace

cudaError_t launch_paged_prefix(int d, bool f16, int subs0, const CUtensorMap& mq0, const CUtensorMap& mk0,
                                const CUtensorMap& mv0, const fa2dev::PagedParams& p0, dim3 merge0, int subs1,
                                const CUtensorMap& mq1, const CUtensorMap& mk1, const CUtensorMap& mv1,
                                const fa2dev::PagedParams& p1, dim3 merge1, void* O, float* LSE, bool half_out,
                                cudaStream_t s) {
  const auto launch = f16 ? launch_paged_ext_f16 : launch_paged_ext_bf16;
  const dim3 none(0);
  cudaError_t e;
  if ((e = launch(d, subs0, mq0, mk0, mv0, p0, static_cast<unsigned>(p0.ctas), none, s)) != cudaSuccess ||
      (e = launch(d, subs1, mq1, mk1, mv1, p1, static_cast<unsigned>(p1.ctas), none, s)) != cudaSuccess ||
      (e = launch(d, subs0, mq0, mk0, mv0, p0, 0, merge0, s)) != cudaSuccess ||
      (e = launch(d, subs1, mq1, mk1, mv1, p1, 0, merge1, s)) != cudaSuccess)
    return e;
  const float *o = static_cast<const float*>(p0.O), *l = p0.LSE;
  if (d == 64) return f16 ? join<64, true>(p1, o, l, O, LSE, half_out, s) : join<64, false>(p1, o, l, O, LSE, half_out, s);
  if (d == 128) return f16 ? join<128, true>(p1, o, l, O, LSE, half_out, s) : join<128, false>(p1, o, l, O, LSE, half_out, s);
  return f16 ? join<256, true>(p1, o, l, O, LSE, half_out, s) : join<256, false>(p1, o, l, O, LSE, half_out, s);
}

}  // namespace fa2host
