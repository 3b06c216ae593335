// Host side of the normed rotary entry points (include/fa2.h).
#include "fa2_checks.h"
#include "fa2_launch.h"
#include "fa2_norm.h"

namespace {

// Rows [B, H, N, d] of a call; strides {batch, head, token}, those of single steps set to 0.
struct Rows {
  const void* p;
  long long s[3];
  long long extent;
};

int check_array(const void* p, const long long* strides, const long long (&sizes)[3], int d, int elem, bool written,
                Rows* out) {
  out->p = p;
  for (int i = 0; i < 3; ++i) {
    out->s[i] = sizes[i] > 1 ? strides[i] : 0;
    // reading the same row twice is fine, writing it twice is not
    if (out->s[i] < 0 || out->s[i] > kMaxStride || (written && sizes[i] > 1 && out->s[i] < d)) return FA2_ERR_SHAPE;
  }
  if (misaligned(p, elem - 1)) return FA2_ERR_ALIGN;
  if (written && !rows_apart(sizes, out->s, d)) return FA2_ERR_SHAPE;
  out->extent = extent(sizes, out->s, d);
  return out->extent < 0 ? FA2_ERR_SHAPE : FA2_OK;
}

bool vectors(const Rows& a, int elem) {
  bool ok = !misaligned(a.p, 15);
  for (int i = 0; i < 3; ++i) ok = ok && a.s[i] * elem % 16 == 0;
  return ok;
}

// in place, or apart: never shifted against each other
bool apart(const Rows& y, const Rows& x, int elem) {
  if (x.p == y.p && x.s[0] == y.s[0] && x.s[1] == y.s[1] && x.s[2] == y.s[2]) return true;
  const char *x0 = static_cast<const char*>(x.p), *y0 = static_cast<const char*>(y.p);
  return x0 >= y0 + y.extent * elem || y0 >= x0 + x.extent * elem;
}

bool bytes_apart(const void* a, long long na, const void* b, long long nb) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return x >= y + nb || y >= x + na;
}

struct NormCall {
  int B, H, N, d;
  const void* weight;
  int weight_dtype;
  float eps;
  const void* positions;
  int positions_int64;
  long long positions_batch_stride;
  const double* inv_freq;
  int rotary_dim, interleaved;
  float mscale;
  int transposed, dtype;
};

int check_call(const NormCall& c) {
  if (c.dtype != FA2_DTYPE_BF16 && c.dtype != FA2_DTYPE_FP16 && c.dtype != FA2_DTYPE_FP32) return FA2_ERR_DTYPE;
  if (c.B < 0 || c.H < 0 || c.N < 0) return FA2_ERR_SHAPE;
  if (c.d != 64 && c.d != 128 && c.d != 256) return FA2_ERR_HEADDIM;
  int rc = check_norm(c.weight_dtype, c.dtype, c.eps);
  if (rc != FA2_OK) return rc;
  return check_rotary(c.inv_freq, c.rotary_dim, c.d, c.mscale);
}

int check_small(const NormCall& c, long long ps) {
  if (ps < 0 || ps > kMaxStride) return FA2_ERR_SHAPE;
  if (!c.weight || !c.positions) return FA2_ERR_NULL;
  return misaligned(c.weight, c.weight_dtype == FA2_DTYPE_FP32 ? 3 : 1) ||
                 misaligned(c.positions, c.positions_int64 ? 7 : 3)
             ? FA2_ERR_ALIGN
             : FA2_OK;
}

bool small_in_memory(const NormCall& c, long long ps) {
  const long long pos_sizes[1] = {c.B}, pos_strides[1] = {ps};
  return range_ok(c.weight, c.d, c.weight_dtype == FA2_DTYPE_FP32 ? 4 : 2) &&
         range_ok(c.positions, extent(pos_sizes, pos_strides, c.N), c.positions_int64 ? 8 : 4) &&
         (c.rotary_dim == 0 || range_ok(c.inv_freq, c.rotary_dim / 2, 8));
}

fa2dev::NormParams params_of(const NormCall& c, const Rows& x, const Rows& y, long long ps) {
  fa2dev::NormParams p = {};
  p.r.x = x.p;
  p.r.y = const_cast<void*>(y.p);
  p.r.positions = c.positions;
  p.r.pos64 = c.positions_int64 != 0;
  p.r.pos_batch = ps;
  p.r.N = c.N;
  p.r.x_batch = x.s[0]; p.r.x_head = x.s[1]; p.r.x_token = x.s[2];
  p.r.y_batch = y.s[0]; p.r.y_head = y.s[1]; p.r.y_token = y.s[2];
  p.r.inv_freq = c.inv_freq;
  p.r.d = c.d;
  p.r.r = c.rotary_dim;
  p.r.interleaved = c.interleaved != 0;
  p.r.transposed = c.transposed;
  p.r.mscale = c.mscale;
  p.r.total_tokens = static_cast<long long>(c.B) * c.N;
  p.r.total_rows = c.H;
  p.weight = c.weight;
  p.weight32 = c.weight_dtype == FA2_DTYPE_FP32;
  p.eps = c.eps;
  return p;
}

}  // namespace

extern "C" int fa2_norm_rope(const void* X, const long long* x_strides, void* Y, const long long* y_strides, int B,
                             int H, int N, int d, const void* weight, int weight_dtype, float eps,
                             const void* positions, int positions_int64, long long positions_batch_stride,
                             const double* inv_freq, int rotary_dim, int interleaved, float mscale, int dtype,
                             fa2_stream_t stream) {
  const NormCall c = {B, H, N, d, weight, weight_dtype, eps, positions, positions_int64, positions_batch_stride,
                      inv_freq, rotary_dim, interleaved, mscale, 0, dtype};
  int rc = check_call(c);
  if (rc != FA2_OK) return rc;
  if (B == 0 || H == 0 || N == 0) return FA2_OK;
  if (!X || !Y || !x_strides || !y_strides) return FA2_ERR_NULL;
  const int elem = dtype == FA2_DTYPE_FP32 ? 4 : 2;
  const long long sizes[3] = {B, H, N}, ps = B > 1 ? positions_batch_stride : 0;
  Rows x, y;
  if ((rc = check_small(c, ps)) != FA2_OK || (rc = check_array(X, x_strides, sizes, d, elem, false, &x)) != FA2_OK ||
      (rc = check_array(Y, y_strides, sizes, d, elem, true, &y)) != FA2_OK)
    return rc;
  if ((rc = fa2host::require_device()) != FA2_OK) return rc;
  if (!range_ok(X, x.extent, elem) || !range_ok(Y, y.extent, elem) || !small_in_memory(c, ps) || !apart(y, x, elem))
    return FA2_ERR_MEMORY;
  const bool wide = wide_norm(rotary_dim, interleaved != 0, elem) && vectors(x, elem) && vectors(y, elem);
  return fa2host::launch_norm_rope(params_of(c, x, y, ps), false, dtype, wide, fa2host::device_sms(),
                                   reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA2_OK
             : FA2_ERR_LAUNCH;
}

extern "C" size_t fa2_norm_rope_backward_workspace_bytes(int d) {
  if (d != 64 && d != 128 && d != 256) return 0;
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return align256(static_cast<size_t>(sms) * fa2host::kNormGradBlocksPerSm * d * 4);
}

extern "C" int fa2_norm_rope_backward(const void* dY, const long long* dy_strides, const void* X,
                                      const long long* x_strides, void* dX, const long long* dx_strides, int B, int H,
                                      int N, int d, const void* weight, int weight_dtype, float eps,
                                      const void* positions, int positions_int64, long long positions_batch_stride,
                                      const double* inv_freq, int rotary_dim, int interleaved, float mscale, int dtype,
                                      float* dweight, void* workspace, size_t workspace_size, fa2_stream_t stream) {
  const NormCall c = {B, H, N, d, weight, weight_dtype, eps, positions, positions_int64, positions_batch_stride,
                      inv_freq, rotary_dim, interleaved, mscale, 1, dtype};
  int rc = check_call(c);
  if (rc != FA2_OK) return rc;
  if (!dweight) return FA2_ERR_NULL;
  if (misaligned(dweight, 3)) return FA2_ERR_ALIGN;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0 || H == 0 || N == 0) {   // a sum over no rows
    if ((rc = fa2host::require_device()) != FA2_OK) return rc;
    if (!range_ok(dweight, d, 4)) return FA2_ERR_MEMORY;
    return fa2host::launch_zero(dweight, d, s) == cudaSuccess ? FA2_OK : FA2_ERR_LAUNCH;
  }
  if (!dY || !X || !dX || !dy_strides || !x_strides || !dx_strides || !workspace) return FA2_ERR_NULL;
  const int elem = dtype == FA2_DTYPE_FP32 ? 4 : 2;
  const long long sizes[3] = {B, H, N}, ps = B > 1 ? positions_batch_stride : 0;
  Rows g, x, y;
  if ((rc = check_small(c, ps)) != FA2_OK || (rc = check_array(dY, dy_strides, sizes, d, elem, false, &g)) != FA2_OK ||
      (rc = check_array(X, x_strides, sizes, d, elem, false, &x)) != FA2_OK ||
      (rc = check_array(dX, dx_strides, sizes, d, elem, true, &y)) != FA2_OK)
    return rc;
  if (misaligned(workspace, 255)) return FA2_ERR_ALIGN;
  if ((rc = fa2host::require_device()) != FA2_OK) return rc;
  const int sms = fa2host::device_sms();
  const size_t need = static_cast<size_t>(sms) * fa2host::kNormGradBlocksPerSm * d * 4;
  if (!range_ok(dY, g.extent, elem) || !range_ok(X, x.extent, elem) || !range_ok(dX, y.extent, elem) ||
      !range_ok(dweight, d, 4) || !small_in_memory(c, ps) || workspace_size < need ||
      !fa2host::device_memory_ok(workspace, need) || !apart(y, g, elem) || !apart(y, x, elem) ||
      !bytes_apart(dweight, d * 4ll, dX, y.extent * elem) || !bytes_apart(dweight, d * 4ll, workspace, need) ||
      !bytes_apart(workspace, need, dX, y.extent * elem))
    return FA2_ERR_MEMORY;
  fa2dev::NormParams p = params_of(c, x, y, ps);
  p.dy = dY;
  p.dy_batch = g.s[0]; p.dy_head = g.s[1]; p.dy_token = g.s[2];
  p.partial = static_cast<float*>(workspace);
  const bool wide = wide_norm(rotary_dim, interleaved != 0, elem) && vectors(g, elem) && vectors(x, elem) &&
                    vectors(y, elem);
  return fa2host::launch_norm_rope_grad(p, dweight, dtype, wide, sms, s) == cudaSuccess ? FA2_OK : FA2_ERR_LAUNCH;
}
