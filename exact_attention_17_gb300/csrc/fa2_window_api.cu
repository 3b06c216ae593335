// Host side of the window entry points (include/fa2.h).
#include "fa2_checks.h"
#include "fa2_launch.h"

namespace {

struct Window {
  int B, H, Hkv, Nq, Nk, d, window, sinks;
  long long BH, BHkv;
};

// Sizes and types; *empty: no rows.
int check_window(int B, int H, int Hkv, int Nq, int Nk, int d, int window, int sinks, float scale, int dtype,
                 bool backward, Window* w) {
  if (dtype != FA2_DTYPE_BF16 && dtype != FA2_DTYPE_FP16) return FA2_ERR_DTYPE;
  if (B < 0 || H < 0 || Hkv < 0 || Nq < 0 || Nk < 0 || window < 1 || sinks < 0) return FA2_ERR_SHAPE;
  w->B = B; w->H = H; w->Hkv = Hkv; w->Nq = Nq; w->Nk = Nk; w->d = d;
  // what lies beyond every key or query means the same as the last one
  w->window = window < Nq ? window : Nq > 0 ? Nq : 1;
  w->sinks = sinks < Nk ? sinks : Nk;
  w->BH = static_cast<long long>(B) * H;
  w->BHkv = static_cast<long long>(B) * Hkv;
  if (w->BH > 0x7fffffffLL) return FA2_ERR_SHAPE;
  if (H > 0 && (Hkv < 1 || H % Hkv != 0)) return FA2_ERR_SHAPE;
  if (H == 0 && Hkv > 0) return FA2_ERR_SHAPE;
  if (w->BH > 0 && Nq > 0 && Nk < 1) return FA2_ERR_SHAPE;
  if (d != 64 && d != 128 && (d != 256 || backward)) return FA2_ERR_HEADDIM;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA2_ERR_SCALE;
  return FA2_OK;
}

int tiles_of(long long n) { return static_cast<int>((n + 127) / 128); }

// How a backward call cuts its key blocks; depends on sizes and the number of SMs.
struct BackwardPlan {
  int key_blocks, sink_blocks, parts, sink_parts, chunk, sink_chunk;
  int group;                             // key/value heads whose blocks run together
  long long items;
  size_t dr_at, dq_at, part_at, bytes;   // workspace: LSE log2(e), D, dQ in fp32, parts
};

// Query tiles an item may have: a quarter of an SM's share (so that the last wave
// is short), at least eight (an item's start and end cost about three).  A block with
// sinks sees every later tile of every head, so it is cut into many; the others
// only where there are few.
constexpr int kLeastChunk = 8;

// Heads that run together: their query tiles in use (a window's, and one more for each
// other key block of the heads that runs) have Q, dO and fp32 dQ in L2, four at least;
// groups of one size, unless that is less than four.  (Window 1024, d = 128, 4096 positions,
// 16 key/value heads shared by 4 each, of which 11 fit: 16 heads together 525 us, 11 and 5
// 511, twice 8 507, 4 519, 2 536; 12 heads: 11 and 1 455, twice 6 439.5; 5 heads shared by 8:
// 4 and 1 373, 3 and 2 374.  6 heads of 8192 positions, window 2048: 5 and 1 652, 4 and 2
// 657, twice 3 666; 8 of 16384, window 4096: all 2617, 4 2579, 2 2616.)
constexpr long long kL2Bytes = 126ll << 20;
constexpr long long kLeastGroup = 4;

BackwardPlan plan_backward(const Window& w, bool grad_half, int sms) {
  BackwardPlan q;
  q.key_blocks = tiles_of(w.Nk);
  q.sink_blocks = tiles_of(w.sinks);
  const long long shared = w.H / w.Hkv, q_tiles = tiles_of(w.Nq);
  const long long row = (126ll + w.window) / 128 + 1;
  const long long list = (row < q_tiles ? row : q_tiles) * shared, sink_list = q_tiles * shared;
  const long long total = w.BHkv * ((q.key_blocks - q.sink_blocks) * list + q.sink_blocks * sink_list);
  long long c = total / (4ll * sms);
  if (c < kLeastChunk) c = kLeastChunk;
  auto cut = [&](long long n, int* parts, int* chunk) {
    const long long k = (n + c / 2) / c;
    *parts = static_cast<int>(k < 1 ? 1 : k);
    *chunk = static_cast<int>((n + *parts - 1) / *parts);
  };
  cut(list, &q.parts, &q.chunk);
  cut(sink_list, &q.sink_parts, &q.sink_chunk);
  const long long tile_bytes = shared * 128 * w.d * (2 + 2 + 4);
  const long long g = (kL2Bytes / tile_bytes - sms) / (row < q_tiles ? row : q_tiles);
  const long long fit = g < kLeastGroup ? kLeastGroup : g, groups = (w.BHkv + fit - 1) / fit;
  const long long equal = (w.BHkv + groups - 1) / groups;
  q.group = static_cast<int>(groups == 1 || equal >= kLeastGroup ? equal : fit);
  const long long sink_items = w.BHkv * q.sink_blocks * q.sink_parts;
  q.items = sink_items + w.BHkv * (q.key_blocks - q.sink_blocks) * q.parts;
  const size_t pad = static_cast<size_t>(q_tiles) * 128 * w.BH * 4;
  const long long slots = q.parts > 1 ? q.items : q.sink_parts > 1 ? sink_items : 0;
  q.dr_at = align256(pad);
  q.dq_at = q.dr_at + align256(pad);
  q.part_at = q.dq_at + (grad_half ? align256(static_cast<size_t>(w.BH) * w.Nq * w.d * 4) : 0);
  q.bytes = q.part_at + align256(static_cast<size_t>(slots) * 256 * w.d * 4);
  return q;
}

// Query sub-tiles per CTA: as for the forward pass without a window, but one (two CTAs
// per SM, whose starts and ends overlap the other's work) for short windows.  16384
// positions, 32 heads sharing 8, two sub-tiles / one: d = 128, windows of 128, 1024 and 4096:
// 146 / 114, 281 / 277 and 663 / 797 us; d = 64: 127 / 91, 254 / 214 and 592 / 590, 16384: 1197 / 1259.
// d = 256 has TMEM for one: windows of 1024 and 4096 610 and 1815 us (870 and 1063 TFLOP/s of what is seen).
int sub_tiles(const Window& w, int sms) {
  if (w.Nq <= 128 || w.d == 256 || w.window <= (w.d == 64 ? 4096 : 1024)) return 1;
  return (static_cast<long long>(w.Nq) + 255) / 256 * w.BH < 2ll * sms ? 1 : 2;
}

}  // namespace

extern "C" int fa2_forward_window(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H,
                                  int Hkv, int Nq, int Nk, int d, int window, int sinks, float scale, int qkv_dtype,
                                  int o_dtype, fa2_stream_t stream) {
  if (o_dtype != FA2_DTYPE_FP32 && o_dtype != qkv_dtype) return FA2_ERR_DTYPE;
  Window w;
  int rc = check_window(B, H, Hkv, Nq, Nk, d, window, sinks, scale, qkv_dtype, false, &w);
  if (rc != FA2_OK) return rc;
  if (w.BH == 0 || Nq == 0) return FA2_OK;
  if (!Q || !K || !V || !O || !LSE) return FA2_ERR_NULL;
  if (misaligned(Q, 15) || misaligned(K, 15) || misaligned(V, 15) || misaligned(O, 15) || misaligned(LSE, 3))
    return FA2_ERR_ALIGN;
  if ((rc = fa2host::require_device()) != FA2_OK) return rc;
  const bool f16 = qkv_dtype == FA2_DTYPE_FP16, o_half = o_dtype != FA2_DTYPE_FP32;
  const long long q_elems = w.BH * Nq * d, kv_elems = w.BHkv * Nk * d;
  if (!range_ok(Q, q_elems, 2) || !range_ok(K, kv_elems, 2) || !range_ok(V, kv_elems, 2) ||
      !range_ok(O, q_elems, o_half ? 2 : 4) || !range_ok(LSE, w.BH * Nq, 4))
    return FA2_ERR_MEMORY;
  const int sms = fa2host::device_sms(), subs = sub_tiles(w, sms);
  const long long blocks = (static_cast<long long>(Nq) + 128 * subs - 1) / (128 * subs);
  if (blocks * w.BH > 0x7fffffffLL) return FA2_ERR_SHAPE;
  CUtensorMap mq, mk, mv, mo;
  const int bh = static_cast<int>(w.BH), bhkv = static_cast<int>(w.BHkv);
  if (!fa2host::encode_heads(&mq, Q, d, Nq, bh, f16) || !fa2host::encode_heads(&mk, K, d, Nk, bhkv, f16) ||
      !fa2host::encode_heads(&mv, V, d, Nk, bhkv, f16) ||
      !fa2host::encode_heads_out(&mo, O, d, Nq, w.BH, o_half ? 2 : 4, f16))
    return FA2_ERR_SHAPE;
  fa2dev::FwdParams p = {};
  p.O = static_cast<float*>(O);
  p.LSE = LSE;
  p.Nq = Nq;
  p.Nk = Nk;
  p.BH = bh;
  p.q_blocks = static_cast<int>(blocks);
  p.scale_log2 = scale * kLog2e;
  p.status = fa2host::device_status_word();
  if (p.status == nullptr) return FA2_ERR_LAUNCH;
  p.wave = sms * (subs == 2 || d == 256 ? 1 : 2);
  p.timeout_ns = fa2host::wait_timeout_ns();
  p.num_splits = 1;
  p.tiles_per_split = tiles_of(Nk);
  p.o_half = o_half ? 1 : 0;
  p.item_group = bh;   // (a window's keys of all heads fit in L2, so one group)
  p.div_per_group = fa2host::make_fast_div(static_cast<int>(blocks * bh));
  p.div_group = fa2host::make_fast_div(bh);
  p.div_splits = fa2host::make_fast_div(1);
  p.window = w.window;
  p.sinks = w.sinks;
  p.div_shared = fa2host::make_fast_div(H / Hkv);
  const auto launch = f16 ? fa2host::launch_window_f16 : fa2host::launch_window_bf16;
  return launch(d, subs, mq, mk, mv, mo, p, static_cast<unsigned>(blocks * bh), reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? FA2_OK
             : FA2_ERR_LAUNCH;
}

extern "C" size_t fa2_backward_window_workspace_bytes(int B, int H, int Hkv, int Nq, int Nk, int d, int window,
                                                      int sinks, int grad_dtype) {
  Window w;
  if (check_window(B, H, Hkv, Nq, Nk, d, window, sinks, 1.f, FA2_DTYPE_BF16, true, &w) != FA2_OK || w.BH == 0 ||
      Nq == 0)
    return 0;
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return plan_backward(w, grad_dtype != FA2_DTYPE_FP32, sms).bytes;
}

extern "C" int fa2_backward_window(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                                   const float* LSE, void* dQ, void* dK, void* dV, int B, int H, int Hkv, int Nq, int Nk,
                                   int d, int window, int sinks, float scale, int qkv_dtype, int o_dtype,
                                   int grad_dtype, void* workspace, size_t workspace_size, fa2_stream_t stream) {
  if ((o_dtype != FA2_DTYPE_FP32 && o_dtype != qkv_dtype) || (grad_dtype != FA2_DTYPE_FP32 && grad_dtype != qkv_dtype))
    return FA2_ERR_DTYPE;
  Window w;
  int rc = check_window(B, H, Hkv, Nq, Nk, d, window, sinks, scale, qkv_dtype, true, &w);
  if (rc != FA2_OK) return rc;
  if (w.BH == 0 || (Nq == 0 && Nk == 0)) return FA2_OK;
  if (!dK || !dV || (Nq > 0 && (!Q || !K || !V || !O || !dO || !LSE || !dQ || !workspace))) return FA2_ERR_NULL;
  if (misaligned(Q, 15) || misaligned(K, 15) || misaligned(V, 15) || misaligned(O, 15) || misaligned(dO, 15) ||
      misaligned(dQ, 15) || misaligned(dK, 15) || misaligned(dV, 15) || misaligned(LSE, 3) || misaligned(workspace, 255))
    return FA2_ERR_ALIGN;
  if ((rc = fa2host::require_device()) != FA2_OK) return rc;
  const bool f16 = qkv_dtype == FA2_DTYPE_FP16, o_half = o_dtype != FA2_DTYPE_FP32, half = grad_dtype != FA2_DTYPE_FP32;
  const long long q_elems = w.BH * Nq * d, kv_elems = w.BHkv * Nk * d;
  const int grad = half ? 2 : 4;
  if (!range_ok(dK, kv_elems, grad) || !range_ok(dV, kv_elems, grad)) return FA2_ERR_MEMORY;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (Nq == 0) {   // no query sees any key
    return cudaMemsetAsync(dK, 0, kv_elems * grad, s) == cudaSuccess &&
                   cudaMemsetAsync(dV, 0, kv_elems * grad, s) == cudaSuccess
               ? FA2_OK
               : FA2_ERR_LAUNCH;
  }
  const BackwardPlan plan = plan_backward(w, half, fa2host::device_sms());
  if (!range_ok(Q, q_elems, 2) || !range_ok(K, kv_elems, 2) || !range_ok(V, kv_elems, 2) ||
      !range_ok(O, q_elems, o_half ? 2 : 4) || !range_ok(dO, q_elems, 2) || !range_ok(LSE, w.BH * Nq, 4) ||
      !range_ok(dQ, q_elems, grad) || workspace_size < plan.bytes || !fa2host::device_memory_ok(workspace, plan.bytes))
    return FA2_ERR_MEMORY;
  if (plan.items > 0x7fffffffLL || (w.BH * Nq * 32 + 255) / 256 > 0x7fffffffLL) return FA2_ERR_SHAPE;
  char* ws = static_cast<char*>(workspace);
  float* dq = half ? reinterpret_cast<float*>(ws + plan.dq_at) : static_cast<float*>(dQ);
  CUtensorMap mq, mk, mv, mdo, mdq;
  const int bh = static_cast<int>(w.BH), bhkv = static_cast<int>(w.BHkv);
  if (!fa2host::encode_heads(&mq, Q, d, Nq, bh, f16) || !fa2host::encode_heads(&mk, K, d, Nk, bhkv, f16) ||
      !fa2host::encode_heads(&mv, V, d, Nk, bhkv, f16) || !fa2host::encode_heads(&mdo, dO, d, Nq, bh, f16) ||
      !fa2host::encode_heads_f32(&mdq, dq, d, Nq, bh))
    return FA2_ERR_SHAPE;
  fa2dev::BwdParams p = {};
  p.dQ = dq;
  p.dK = static_cast<float*>(dK);
  p.dV = static_cast<float*>(dV);
  float* L2 = reinterpret_cast<float*>(ws);
  float* Dr = reinterpret_cast<float*>(ws + plan.dr_at);
  p.L2 = L2;
  p.Dr = Dr;
  p.Nq = Nq;
  p.Nk = Nk;
  p.Nq_pad = tiles_of(Nq) * 128;
  p.BH = bhkv;
  p.key_blocks = plan.key_blocks;
  p.item_group = plan.group;
  p.scale = scale;
  p.scale_log2 = scale * kLog2e;
  p.status = fa2host::device_status_word();
  if (p.status == nullptr) return FA2_ERR_LAUNCH;
  p.timeout_ns = fa2host::wait_timeout_ns();
  p.window = w.window;
  p.sinks = w.sinks;
  p.shared = H / Hkv;
  p.sink_blocks = plan.sink_blocks;
  p.parts = plan.parts;
  p.sink_parts = plan.sink_parts;
  p.chunk = plan.chunk;
  p.sink_chunk = plan.sink_chunk;
  p.part = reinterpret_cast<float*>(ws + plan.part_at);
  p.grad_half = half ? 1 : 0;
  if (fa2host::launch_bwd_window_pre(d, f16, o_half, O, dO, LSE, dq, L2, Dr, w.BH * Nq, Nq, p.Nq_pad, s) != cudaSuccess ||
      fa2host::launch_bwd_window(d, f16, mq, mk, mv, mdo, mdq, p, static_cast<unsigned>(plan.items), s) != cudaSuccess ||
      fa2host::launch_bwd_window_end(d, f16, p, half ? dQ : nullptr, q_elems, s) != cudaSuccess)
    return FA2_ERR_LAUNCH;
  return FA2_OK;
}

extern "C" int fa2_check_window_plan(int B, int H, int Hkv, int Nq, int Nk, int d, int window, int sinks, int sm_count,
                                     int* plan) {
  Window w;
  const int rc = check_window(B, H, Hkv, Nq, Nk, d, window, sinks, 1.f, FA2_DTYPE_BF16, false, &w);
  if (rc != FA2_OK) return rc;
  if (w.BH == 0 || Nq == 0 || sm_count < 1) return FA2_ERR_SHAPE;
  if (!plan) return FA2_ERR_NULL;
  const BackwardPlan q = plan_backward(w, false, sm_count);
  plan[0] = sub_tiles(w, sm_count);
  plan[1] = q.group;
  plan[2] = q.parts;
  plan[3] = q.sink_parts;
  return FA2_OK;
}
