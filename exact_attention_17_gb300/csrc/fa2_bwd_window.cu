// Backward kernels of windows (head dimensions 64 and 128, bf16 or fp16), and the
// kernel behind them.
#include "fa2_launch.h"

namespace fa2dev {

// (No pointer of these kernels is declared restricted: the compiler would read through the cache that is not
// kept coherent, while the kernel before, behind which they are launched early, still writes.)

// Pre-pass: D_i = dO_i . O_i, LSE_i log2(e), and the row of dQ set to zero, D / 8
// lanes a query row.  Entries past Nq in each head's padded arrays are set to zero.
// Bound: bytes (O and dO read, fp32 dQ written).
template <int D, bool F16, bool O_HALF>
__global__ void __launch_bounds__(256) fa2_bwd_window_pre_kernel(const void* O, const uint16_t* dO, const float* LSE,
                                                                 float* dQ, float* L2, float* Dr, long long rows, int Nq,
                                                                 int Nq_pad) {
  constexpr int kLanes = D / 8;
  const long long r = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / kLanes;
  const int lane = threadIdx.x % kLanes;
  const bool live = r < rows;   // (every lane takes part in the shuffles)
  const long long at = (live ? r : 0) * D + lane * 8;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto wide = [](uint32_t bits) {
    return F16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(bits))) : __uint_as_float(bits << 16);
  };
  const uint4 g = *reinterpret_cast<const uint4*>(dO + at);
  const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
  float o[8];
  if constexpr (O_HALF) {
    const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(O) + at);
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = wide(e & 1 ? xw[e / 2] >> 16 : xw[e / 2] & 0xffffu);
  } else {
    const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(O) + at);
    const float4 y = *reinterpret_cast<const float4*>(static_cast<const float*>(O) + at + 4);
    o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
    o[4] = y.x; o[5] = y.y; o[6] = y.z; o[7] = y.w;
  }
  float acc = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) acc = fmaf(wide(e & 1 ? gw[e / 2] >> 16 : gw[e / 2] & 0xffffu), o[e], acc);
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  if (!live) return;
  *reinterpret_cast<float4*>(dQ + at) = make_float4(0.f, 0.f, 0.f, 0.f);
  *reinterpret_cast<float4*>(dQ + at + 4) = make_float4(0.f, 0.f, 0.f, 0.f);
  const long long bh = r / Nq, q = r - bh * Nq;
  if (lane == 0) {
    Dr[bh * Nq_pad + q] = acc;
    L2[bh * Nq_pad + q] = LSE[r] * 1.4426950408889634f;
  }
  if (q == Nq - 1) {
    for (long long pq = Nq + lane; pq < Nq_pad; pq += kLanes) {
      Dr[bh * Nq_pad + pq] = 0.f;
      L2[bh * Nq_pad + pq] = 0.f;
    }
  }
}

// dQ from fp32 to the input type (the first `dq_blocks` blocks of the grid), and sums of the
// items of the key blocks that were cut: key row, four columns a thread.
template <int D, bool F16>
__global__ void __launch_bounds__(256) fa2_bwd_window_end_kernel(const __grid_constant__ BwdParams p,
                                                                 uint2* dq_out, long long q_quads,
                                                                 int dq_blocks, long long sum_quads) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (static_cast<int>(blockIdx.x) < dq_blocks) {
    const float4* in = reinterpret_cast<const float4*>(p.dQ);
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < q_quads; i += dq_blocks * 256ll) {
      const float4 x = in[i];
      dq_out[i] = make_uint2(pack_x2<F16>(x.x, x.y), pack_x2<F16>(x.z, x.w));
    }
    return;
  }
  const long long at = (static_cast<long long>(blockIdx.x) - dq_blocks) * 256 + threadIdx.x;
  if (at >= sum_quads) return;
  constexpr int kQuads = D / 4;
  const int c = static_cast<int>(at % kQuads);
  const long long row = at / kQuads;                  // (block, head, key of the block)
  const int y = static_cast<int>(row >> 7), key_row = static_cast<int>(row & 127);
  const int jb = y / p.BH, bh = y - jb * p.BH, key = jb * 128 + key_row;
  if (key >= p.Nk) return;
  const bool with_sinks = jb < p.sink_blocks;
  const int n = with_sinks ? p.sink_parts : p.parts;
  if (n == 1) return;
  const long long slot = with_sinks ? static_cast<long long>(y) * n
                                    : static_cast<long long>(p.BH) * p.sink_blocks * p.sink_parts +
                                          (y - static_cast<long long>(p.BH) * p.sink_blocks) * n;
  const float* from = p.part + (slot * 256 + key_row) * D + c * 4;
  float4 dk = make_float4(0.f, 0.f, 0.f, 0.f), dv = dk;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float4 a = *reinterpret_cast<const float4*>(from + static_cast<long long>(i) * 256 * D);
    const float4 b = *reinterpret_cast<const float4*>(from + static_cast<long long>(i) * 256 * D + 128 * D);
    dk.x += a.x; dk.y += a.y; dk.z += a.z; dk.w += a.w;
    dv.x += b.x; dv.y += b.y; dv.z += b.z; dv.w += b.w;
  }
  const long long out = (static_cast<long long>(bh) * p.Nk + key) * kQuads + c;
  if (p.grad_half) {
    reinterpret_cast<uint2*>(p.dK)[out] = make_uint2(pack_x2<F16>(dk.x, dk.y), pack_x2<F16>(dk.z, dk.w));
    reinterpret_cast<uint2*>(p.dV)[out] = make_uint2(pack_x2<F16>(dv.x, dv.y), pack_x2<F16>(dv.z, dv.w));
  } else {
    reinterpret_cast<float4*>(p.dK)[out] = dk;
    reinterpret_cast<float4*>(p.dV)[out] = dv;
  }
}

}  // namespace fa2dev

namespace fa2host {

namespace {
template <int D, bool F16>
cudaError_t set_limits() {
  return cudaFuncSetAttribute(fa2dev::fa2_bwd_tc_kernel<D, true, F16, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              fa2dev::BwdConfig<D>::kSmemBytes);
}

template <int D, bool F16>
cudaError_t run(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo,
                const CUtensorMap& mdq, const fa2dev::BwdParams& p, unsigned grid, cudaStream_t s) {
  return launch_behind(fa2dev::fa2_bwd_tc_kernel<D, true, F16, true>, dim3(grid), fa2dev::kBwdThreads,
                       fa2dev::BwdConfig<D>::kSmemBytes, s, mq, mk, mv, mdo, mdq, p);
}

template <int D, bool F16, bool O_HALF>
cudaError_t run_pre(const void* O, const void* dO, const float* LSE, float* dQ, float* L2, float* Dr, long long rows,
                    int Nq, int Nq_pad, cudaStream_t s) {
  const long long blocks = (rows * (D / 8) + 255) / 256;
  return launch_behind(fa2dev::fa2_bwd_window_pre_kernel<D, F16, O_HALF>, dim3(static_cast<unsigned>(blocks)), 256, 0, s,
                       O, static_cast<const uint16_t*>(dO), LSE, dQ, L2, Dr, rows, Nq, Nq_pad);
}

template <int D, bool F16>
cudaError_t run_end(const fa2dev::BwdParams& p, void* dq_out, long long q_elems, cudaStream_t s) {
  const long long quads = dq_out ? q_elems / 4 : 0;
  const int dq_blocks = static_cast<int>(quads > 0 ? (quads + 2047) / 2048 < 4096 ? (quads + 2047) / 2048 : 4096 : 0);
  const int cut_blocks = p.parts > 1 ? p.key_blocks : p.sink_parts > 1 ? p.sink_blocks : 0;
  const long long sum_quads = static_cast<long long>(cut_blocks) * p.BH * 128 * (D / 4);
  const long long sum_blocks = (sum_quads + 255) / 256;
  if (dq_blocks + sum_blocks == 0) return cudaSuccess;
  if (dq_blocks + sum_blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_behind(fa2dev::fa2_bwd_window_end_kernel<D, F16>, dim3(static_cast<unsigned>(dq_blocks + sum_blocks)),
                       256, 0, s, p, static_cast<uint2*>(dq_out), quads, dq_blocks, sum_quads);
}
}  // namespace

cudaError_t prepare_bwd_window() {
  cudaError_t e;
  if ((e = set_limits<64, false>()) != cudaSuccess || (e = set_limits<64, true>()) != cudaSuccess ||
      (e = set_limits<128, false>()) != cudaSuccess)
    return e;
  return set_limits<128, true>();
}

cudaError_t launch_bwd_window_pre(int d, bool f16, bool o_half, const void* O, const void* dO, const float* LSE,
                                  float* dQ, float* L2, float* Dr, long long rows, int Nq, int Nq_pad, cudaStream_t s) {
  const auto pick = [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    return f16 ? (o_half ? run_pre<D, true, true> : run_pre<D, true, false>)
               : (o_half ? run_pre<D, false, true> : run_pre<D, false, false>);
  };
  const auto f = d == 64 ? pick(fa2dev::Int<64>{}) : pick(fa2dev::Int<128>{});
  return f(O, dO, LSE, dQ, L2, Dr, rows, Nq, Nq_pad, s);
}

cudaError_t launch_bwd_window(int d, bool f16, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                              const CUtensorMap& mdo, const CUtensorMap& mdq, const fa2dev::BwdParams& p, unsigned grid,
                              cudaStream_t s) {
  const auto f = d == 64 ? (f16 ? run<64, true> : run<64, false>) : f16 ? run<128, true> : run<128, false>;
  return f(mq, mk, mv, mdo, mdq, p, grid, s);
}

cudaError_t launch_bwd_window_end(int d, bool f16, const fa2dev::BwdParams& p, void* dq_out, long long q_elems,
                                  cudaStream_t s) {
  const auto f = d == 64 ? (f16 ? run_end<64, true> : run_end<64, false>) : f16 ? run_end<128, true> : run_end<128, false>;
  return f(p, dq_out, q_elems, s);
}

}  // namespace fa2host
