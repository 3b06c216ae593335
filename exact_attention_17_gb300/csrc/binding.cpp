// The short way from torch tensors to the paged-cache entry points of libfa2.so.
//
// A small call spends more time in Python (reading attributes, ctypes
// conversions: 10-20 us) than on the GPU.  Each function here takes the
// arguments of its namesake in paged.py, checks them, allocates the outputs on
// the current stream and makes the C call.  It answers None for anything that is
// not plain -- a wrong type or shape, another device than the current one -- and
// then paged.py goes its own, longer way, which also says what is wrong; it
// answers a number where the library returned a status.
//
// The library's functions are handed over as addresses (init), so that this
// module and ctypes use one and the same loaded library.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <vector>

#include "fa2.h"

namespace {

decltype(&fa2_forward_paged) forward_paged_fn;
decltype(&fa2_forward_paged_workspace_bytes) workspace_bytes_fn;
decltype(&fa2_rope) rope_fn;
decltype(&fa2_append_paged) append_fn;
decltype(&fa2_pages_workspace_bytes) pages_workspace_fn;
decltype(&fa2_pages_reserve) reserve_fn;
decltype(&fa2_pages_fork) fork_fn;
decltype(&fa2_pages_free) free_fn;
decltype(&fa2_pages_compact) compact_fn;
decltype(&fa2_pages_copy) copy_fn;
decltype(&fa2_append_paged_norm) append_norm_fn;
decltype(&fa2_norm_rope) norm_fn;
decltype(&fa2_norm_rope_backward) norm_backward_fn;
decltype(&fa2_norm_rope_backward_workspace_bytes) norm_workspace_fn;
decltype(&fa2_forward_paged_window) paged_window_fn;
decltype(&fa2_forward_paged_prefix) paged_prefix_fn;
decltype(&fa2_forward_paged_prefix_workspace_bytes) prefix_workspace_fn;
decltype(&fa2_forward_window) window_fn;
decltype(&fa2_backward_window) window_backward_fn;
decltype(&fa2_backward_window_workspace_bytes) window_workspace_fn;

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

int type_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return FA2_DTYPE_BF16;
    case at::kHalf: return FA2_DTYPE_FP16;
    case at::kFloat: return FA2_DTYPE_FP32;
    default: return -1;
  }
}

// An int32 tensor on `device`, rows dense.
bool ints(const at::Tensor* t, c10::IntArrayRef shape, at::Device device) {
  return t && t->scalar_type() == at::kInt && t->device() == device && t->sizes() == shape &&
         (shape.back() <= 1 || t->stride(-1) == 1);
}

bool fits_int(c10::IntArrayRef sizes) {
  for (int64_t n : sizes)
    if (n > 0x7fffffff) return false;
  return true;
}

fa2_stream_t stream_of(at::Device d) {
  return reinterpret_cast<fa2_stream_t>(c10::cuda::getCurrentCUDAStream(d.index()).stream());
}

bool current(at::Device d) { return d.is_cuda() && d.index() == c10::cuda::current_device(); }

at::Tensor make(c10::IntArrayRef shape, at::ScalarType type, at::Device d) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(d));
}

PyObject* none() { Py_RETURN_NONE; }

PyObject* result(int rc, at::Tensor&& t) { return rc == FA2_OK ? THPVariable_Wrap(std::move(t)) : PyLong_FromLong(rc); }

// C++ exceptions become the Python exceptions that torch's own functions raise
// (torch.OutOfMemoryError, where a server may free pages and go on).
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

template <typename F>
int call(F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc;
}

// The cache's description from (k_pages, v_pages, page_table, kv_lens).
bool cache_of(PyObject* const* a, fa2_paged_cache* c, at::Device* device) {
  const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *table = tensor(a[2]), *lens = tensor(a[3]);
  if (!k || !v || !table || !lens || k->dim() != 4 || table->dim() != 2 || !current(k->device())) return false;
  const int type = type_code(*k);
  if ((type != FA2_DTYPE_BF16 && type != FA2_DTYPE_FP16) || k->stride(3) != 1 || v->scalar_type() != k->scalar_type() ||
      v->sizes() != k->sizes() || v->strides() != k->strides() || v->device() != k->device())
    return false;
  *device = k->device();
  if (!ints(table, table->sizes(), *device) || !ints(lens, {table->size(0)}, *device) || !fits_int(k->sizes()) ||
      !fits_int(table->sizes()) || k->size(1) == 0)   // (no heads: callers divide by them)
    return false;
  c->k_pages = k->data_ptr();
  c->v_pages = v->data_ptr();
  c->num_pages = static_cast<int>(k->size(0));
  c->kv_heads = static_cast<int>(k->size(1));
  c->page_size = static_cast<int>(k->size(2));
  c->d = static_cast<int>(k->size(3));
  c->page_stride = k->stride(0);
  c->head_stride = k->stride(1);
  c->slot_stride = k->stride(2);
  c->dtype = type;
  c->page_table = static_cast<const int*>(table->data_ptr());
  c->table_stride = table->stride(0);
  c->table_width = static_cast<int>(table->size(1));
  c->B = static_cast<int>(table->size(0));
  c->kv_lens = static_cast<const int*>(lens->data_ptr());
  return true;
}

// cu_q's pointer (null for None); false when it is not as it should be
bool offsets_of(PyObject* o, int B, int64_t T, at::Device device, const int** out) {
  *out = nullptr;
  if (o == Py_None) return T == B;
  const at::Tensor* t = tensor(o);
  if (!ints(t, {B + 1ll}, device)) return false;
  *out = static_cast<const int*>(t->data_ptr());
  return true;
}

// [T, H, d] rows of a type, last dimension dense
bool rows(const at::Tensor* t, int64_t T, int64_t H, int64_t d, at::ScalarType type, at::Device device) {
  return t && t->dim() == 3 && t->size(0) == T && t->size(1) == H && t->size(2) == d && t->scalar_type() == type &&
         t->device() == device && t->stride(2) == 1 && fits_int(t->sizes());
}

bool frequencies(PyObject* o, at::Device device, int64_t d, const double** out, int* rotary) {
  *out = nullptr;
  *rotary = 0;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (!t || t->scalar_type() != at::kDouble || t->dim() != 1 || !t->is_contiguous() || t->device() != device ||
      2 * t->size(0) > d)
    return false;
  *out = static_cast<const double*>(t->data_ptr());
  *rotary = static_cast<int>(2 * t->size(0));
  return true;
}

PyObject* pair_of(at::Tensor&& a, at::Tensor&& b) {
  PyObject* pair = PyTuple_New(2);
  if (!pair) return nullptr;
  PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(std::move(a)));
  PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(std::move(b)));
  return pair;
}

// A norm's weights of the rows' type or fp32 (null for None); *code: their type, left as it is for None
bool weights(PyObject* o, int64_t d, at::ScalarType type, at::Device device, const void** out, int* code) {
  *out = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (!t || (t->scalar_type() != type && t->scalar_type() != at::kFloat) || t->dim() != 1 || t->size(0) != d ||
      !t->is_contiguous() || t->device() != device)
    return false;
  const int own = type_code(*t);
  if (*code >= 0 && *code != own) return false;
  *code = own;
  *out = t->data_ptr();
  return true;
}

// The queries of an attention call over a cache: (q, k_pages, v_pages, page_table, kv_lens, cu_q, ...).
struct Queries {
  fa2_paged_cache c;
  at::Device device = at::Device(at::kCPU);
  const at::Tensor* q;
  int T, Hq;
  const int* cu;
};

bool queries_of(PyObject* const* a, Queries* x) {
  x->q = tensor(a[0]);
  if (!x->q || x->q->dim() != 3 || !cache_of(a + 1, &x->c, &x->device)) return false;
  const int64_t T = x->q->size(0), Hq = x->q->size(1);
  if (!rows(x->q, T, Hq, x->c.d, x->c.dtype == FA2_DTYPE_BF16 ? at::kBFloat16 : at::kHalf, x->device) ||
      Hq % x->c.kv_heads != 0 || !offsets_of(a[5], x->c.B, T, x->device, &x->cu))
    return false;
  x->T = static_cast<int>(T);
  x->Hq = static_cast<int>(Hq);
  return true;
}

// 1/sqrt(d) rounded to fp32 for None; sets a Python error where it is no number.
double scale_of(PyObject* o, int64_t d) {
  return o == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(d))) : PyFloat_AsDouble(o);
}

// Outputs and workspace, and the call: f(O, LSE, workspace, its size, stream)
template <typename F>
PyObject* attend(const Queries& x, size_t size, F f) {
  at::Tensor o = make(x.q->sizes(), x.q->scalar_type(), x.device), lse = make({x.T, x.Hq}, at::kFloat, x.device);
  at::Tensor ws = make({static_cast<int64_t>(size > 0 ? size : 1)}, at::kByte, x.device);
  const fa2_stream_t s = stream_of(x.device);
  const int rc = call([&] { return f(o.data_ptr(), static_cast<float*>(lse.data_ptr()), ws.data_ptr(), size, s); });
  if (rc != FA2_OK) return PyLong_FromLong(rc);
  return pair_of(std::move(o), std::move(lse));
}

// (q, k_pages, v_pages, page_table, kv_lens, cu_q, causal, scale)
PyObject* forward_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Queries x;
    if (n != 8 || !queries_of(a, &x)) return none();
    const int causal = PyObject_IsTrue(a[6]);
    const double scale = scale_of(a[7], x.c.d);
    if (causal < 0 || PyErr_Occurred()) return nullptr;
    return attend(x, workspace_bytes_fn(x.c.B, x.T, x.Hq, x.c.kv_heads, x.c.d, x.cu != nullptr),
                  [&](void* o, float* lse, void* ws, size_t size, fa2_stream_t s) {
                    return forward_paged_fn(&x.c, x.q->data_ptr(), x.q->stride(0), x.q->stride(1), o, lse, x.cu, x.T,
                                            x.Hq, causal, static_cast<float>(scale), x.c.dtype, ws, size, s);
                  });
  });
}

// (q, k_pages, v_pages, page_table, kv_lens, cu_q, window, sinks, scale); window and sinks fit C ints
PyObject* forward_paged_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Queries x;
    if (n != 9 || !queries_of(a, &x)) return none();
    const long window = PyLong_AsLong(a[6]), sinks = PyLong_AsLong(a[7]);
    const double scale = scale_of(a[8], x.c.d);
    if (PyErr_Occurred()) return nullptr;
    return attend(x, workspace_bytes_fn(x.c.B, x.T, x.Hq, x.c.kv_heads, x.c.d, x.cu != nullptr),
                  [&](void* o, float* lse, void* ws, size_t size, fa2_stream_t s) {
                    return paged_window_fn(&x.c, x.q->data_ptr(), x.q->stride(0), x.q->stride(1), o, lse, x.cu, x.T,
                                           x.Hq, static_cast<int>(window), static_cast<int>(sinks),
                                           static_cast<float>(scale), x.c.dtype, ws, size, s);
                  });
  });
}

// (q, k_pages, v_pages, page_table, kv_lens, cu_q, cu_groups, prefix_lens, causal, scale)
PyObject* forward_paged_prefix(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Queries x;
    if (n != 10 || !queries_of(a, &x)) return none();
    const at::Tensor *first = tensor(a[6]), *lens = tensor(a[7]);
    if (!lens || lens->dim() != 1 || lens->size(0) < 1 || !fits_int(lens->sizes()) || !ints(lens, lens->sizes(), x.device) ||
        !ints(first, {lens->size(0) + 1}, x.device))
      return none();
    const int groups = static_cast<int>(lens->size(0)), causal = PyObject_IsTrue(a[8]);
    const double scale = scale_of(a[9], x.c.d);
    if (causal < 0 || PyErr_Occurred()) return nullptr;
    return attend(x, prefix_workspace_fn(x.c.B, groups, x.T, x.Hq, x.c.kv_heads, x.c.d, x.cu != nullptr),
                  [&](void* o, float* lse, void* ws, size_t size, fa2_stream_t s) {
                    return paged_prefix_fn(&x.c, x.q->data_ptr(), x.q->stride(0), x.q->stride(1), o, lse, x.cu, x.T,
                                           x.Hq, static_cast<const int*>(first->data_ptr()),
                                           static_cast<const int*>(lens->data_ptr()), groups, causal,
                                           static_cast<float>(scale), x.c.dtype, ws, size, s);
                  });
  });
}

// The arguments of the window calls: q [B, H, Nq, d], k and v [B, Hkv, Nk, d], dense.
struct Windowed {
  const at::Tensor *q, *k, *v;
  int B, H, Hkv, Nq, Nk, d, code;
  long window, sinks;
};

bool dense(const at::Tensor* t, c10::IntArrayRef shape, at::ScalarType type, at::Device device) {
  return t && t->sizes() == shape && t->scalar_type() == type && t->device() == device && t->is_contiguous();
}

bool windowed(PyObject* q, PyObject* k, PyObject* v, PyObject* window, PyObject* sinks, Windowed* x) {
  x->q = tensor(q);
  x->k = tensor(k);
  x->v = tensor(v);
  if (!x->q || !x->k || !x->v || x->q->dim() != 4 || x->k->dim() != 4 || !current(x->q->device())) return false;
  x->code = type_code(*x->q);
  const at::ScalarType type = x->q->scalar_type();
  if ((x->code != FA2_DTYPE_BF16 && x->code != FA2_DTYPE_FP16) || !fits_int(x->q->sizes()) || !fits_int(x->k->sizes()) ||
      x->k->size(0) != x->q->size(0) || x->k->size(3) != x->q->size(3) ||
      !dense(x->q, x->q->sizes(), type, x->q->device()) || !dense(x->k, x->k->sizes(), type, x->q->device()) ||
      !dense(x->v, x->k->sizes(), type, x->q->device()))
    return false;
  x->B = static_cast<int>(x->q->size(0));
  x->H = static_cast<int>(x->q->size(1));
  x->Nq = static_cast<int>(x->q->size(2));
  x->d = static_cast<int>(x->q->size(3));
  x->Hkv = static_cast<int>(x->k->size(1));
  x->Nk = static_cast<int>(x->k->size(2));
  x->window = PyLong_AsLong(window);
  x->sinks = PyLong_AsLong(sinks);
  return x->Hkv > 0 && x->H % x->Hkv == 0;
}

// (q, k, v, window, sinks, scale, half): half: O of q's type instead of fp32
PyObject* forward_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Windowed x;
    if (n != 7 || !windowed(a[0], a[1], a[2], a[3], a[4], &x)) return PyErr_Occurred() ? nullptr : none();
    const int half = PyObject_IsTrue(a[6]);
    const double scale = scale_of(a[5], x.d);
    if (half < 0 || PyErr_Occurred()) return nullptr;
    const at::Device device = x.q->device();
    at::Tensor o = make(x.q->sizes(), half ? x.q->scalar_type() : at::kFloat, device);
    at::Tensor lse = make(x.q->sizes().slice(0, 3), at::kFloat, device);
    const fa2_stream_t s = stream_of(device);
    const int rc = call([&] {
      return window_fn(x.q->data_ptr(), x.k->data_ptr(), x.v->data_ptr(), o.data_ptr(),
                       static_cast<float*>(lse.data_ptr()), x.B, x.H, x.Hkv, x.Nq, x.Nk, x.d,
                       static_cast<int>(x.window), static_cast<int>(x.sinks), static_cast<float>(scale), x.code,
                       half ? x.code : static_cast<int>(FA2_DTYPE_FP32), s);
    });
    if (rc != FA2_OK) return PyLong_FromLong(rc);
    return pair_of(std::move(o), std::move(lse));
  });
}

// (q, k, v, o, lse, do, window, sinks, scale, half): half: gradients of q's type instead of fp32
PyObject* backward_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Windowed x;
    if (n != 10 || !windowed(a[0], a[1], a[2], a[6], a[7], &x)) return PyErr_Occurred() ? nullptr : none();
    const at::Tensor *o = tensor(a[3]), *lse = tensor(a[4]), *g = tensor(a[5]);
    const at::Device device = x.q->device();
    const at::ScalarType type = x.q->scalar_type();
    if (!o || (o->scalar_type() != at::kFloat && o->scalar_type() != type) ||
        !dense(o, x.q->sizes(), o->scalar_type(), device) || !dense(lse, x.q->sizes().slice(0, 3), at::kFloat, device) ||
        !dense(g, x.q->sizes(), type, device))
      return none();
    const int half = PyObject_IsTrue(a[9]);
    const double scale = scale_of(a[8], x.d);
    if (half < 0 || PyErr_Occurred()) return nullptr;
    const at::ScalarType kind = half ? type : at::kFloat;
    const int code = half ? x.code : static_cast<int>(FA2_DTYPE_FP32);
    const int window = static_cast<int>(x.window), sinks = static_cast<int>(x.sinks);
    const size_t size = window_workspace_fn(x.B, x.H, x.Hkv, x.Nq, x.Nk, x.d, window, sinks, code);
    at::Tensor dq = make(x.q->sizes(), kind, device), dk = make(x.k->sizes(), kind, device);
    at::Tensor dv = make(x.k->sizes(), kind, device);
    at::Tensor ws = make({static_cast<int64_t>(size > 0 ? size : 1)}, at::kByte, device);
    const fa2_stream_t s = stream_of(device);
    const int rc = call([&] {
      return window_backward_fn(x.q->data_ptr(), x.k->data_ptr(), x.v->data_ptr(), o->data_ptr(), g->data_ptr(),
                                static_cast<const float*>(lse->data_ptr()), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                x.B, x.H, x.Hkv, x.Nq, x.Nk, x.d, window, sinks, static_cast<float>(scale), x.code,
                                type_code(*o), code, ws.data_ptr(), size, s);
    });
    if (rc != FA2_OK) return PyLong_FromLong(rc);
    PyObject* three = PyTuple_New(3);
    if (!three) return nullptr;
    PyTuple_SET_ITEM(three, 0, THPVariable_Wrap(std::move(dq)));
    PyTuple_SET_ITEM(three, 1, THPVariable_Wrap(std::move(dk)));
    PyTuple_SET_ITEM(three, 2, THPVariable_Wrap(std::move(dv)));
    return three;
  });
}

// (k, v, k_pages, v_pages, page_table, kv_lens, cu_q, q, inv_freq, interleaved, mscale, q_weight, k_weight, eps)
PyObject* append_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    fa2_paged_cache c;
    at::Device device(at::kCPU);
    const at::Tensor *k = n == 14 ? tensor(a[0]) : nullptr, *v = n == 14 ? tensor(a[1]) : nullptr;
    const at::Tensor* q = k ? tensor(a[7]) : nullptr;
    if (!k || !v || !q || k->dim() != 3 || q->dim() != 3 || !cache_of(a + 2, &c, &device)) return none();
    const int64_t T = k->size(0), Hq = q->size(1);
    const at::ScalarType type = c.dtype == FA2_DTYPE_BF16 ? at::kBFloat16 : at::kHalf;
    const int* cu;
    const double* freq;
    int rotary;
    if (!rows(k, T, c.kv_heads, c.d, type, device) || !rows(v, T, c.kv_heads, c.d, type, device) ||
        !rows(q, T, Hq, c.d, type, device) || !offsets_of(a[6], c.B, T, device, &cu) ||
        !frequencies(a[8], device, c.d, &freq, &rotary))
      return none();
    const int interleaved = PyObject_IsTrue(a[9]);
    const double mscale = PyFloat_AsDouble(a[10]);
    const void *q_weight, *k_weight;
    int code = -1;
    if (!weights(a[11], c.d, type, device, &q_weight, &code) || !weights(a[12], c.d, type, device, &k_weight, &code))
      return none();
    const double eps = PyFloat_AsDouble(a[13]);
    if (interleaved < 0 || PyErr_Occurred()) return nullptr;
    at::Tensor out = make(q->sizes(), type, device);
    const long long ks[2] = {k->stride(0), k->stride(1)}, vs[2] = {v->stride(0), v->stride(1)};
    const long long qs[2] = {q->stride(0), q->stride(1)}, os[2] = {out.stride(0), out.stride(1)};
    const fa2_stream_t s = stream_of(device);
    const int rc = call([&] {
      if (q_weight || k_weight)
        return append_norm_fn(&c, k->data_ptr(), ks, v->data_ptr(), vs, q->data_ptr(), qs, out.data_ptr(), os,
                              static_cast<int>(Hq), cu, static_cast<int>(T), q_weight, k_weight, code,
                              static_cast<float>(eps), freq, rotary, interleaved, static_cast<float>(mscale), s);
      return append_fn(&c, k->data_ptr(), ks, v->data_ptr(), vs, q->data_ptr(), qs, out.data_ptr(), os,
                       static_cast<int>(Hq), cu, static_cast<int>(T), freq, rotary, interleaved,
                       static_cast<float>(mscale), s);
    });
    return result(rc, std::move(out));
  });
}

// Rows of heads, [B, H, N, d] or packed [T, H, d], with their positions.
struct Heads {
  int64_t B, H, N, d;
  long long s[3];   // {batch, head, token}
  const void* positions;
  int wide;
  long long batch_stride;
};

void strides_of(const at::Tensor& x, long long (&s)[3]) {
  const bool packed = x.dim() == 3;
  s[0] = packed ? 0 : x.stride(0);
  s[1] = x.stride(1);
  s[2] = packed ? x.stride(0) : x.stride(2);
}

bool heads_of(const at::Tensor* x, const at::Tensor* pos, Heads* h) {
  if (!x || !pos || (x->dim() != 3 && x->dim() != 4) || !current(x->device()) || type_code(*x) < 0 ||
      x->stride(-1) != 1 || !fits_int(x->sizes()))
    return false;
  const bool packed = x->dim() == 3;
  h->B = packed ? 1 : x->size(0);
  h->H = x->size(1);
  h->N = packed ? x->size(0) : x->size(2);
  h->d = x->size(-1);
  strides_of(*x, h->s);
  h->wide = pos->scalar_type() == at::kLong;
  if ((!h->wide && pos->scalar_type() != at::kInt) || pos->device() != x->device() ||
      !(pos->sizes() == c10::IntArrayRef({h->N}) || pos->sizes() == c10::IntArrayRef({h->B, h->N})) ||
      (h->N > 1 && pos->stride(-1) != 1))
    return false;
  h->positions = pos->data_ptr();
  h->batch_stride = pos->dim() == 2 ? pos->stride(0) : 0;
  return true;
}

// (x, positions, inv_freq, interleaved, mscale, transposed)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *x = n == 6 ? tensor(a[0]) : nullptr, *pos = x ? tensor(a[1]) : nullptr;
    Heads h;
    const double* freq;
    int rotary;
    if (!heads_of(x, pos, &h) || !frequencies(a[2], x->device(), h.d, &freq, &rotary)) return none();
    const int interleaved = PyObject_IsTrue(a[3]), transposed = PyObject_IsTrue(a[5]);
    const double mscale = PyFloat_AsDouble(a[4]);
    if (interleaved < 0 || transposed < 0 || PyErr_Occurred()) return nullptr;
    at::Tensor y = make(x->sizes(), x->scalar_type(), x->device());
    long long ys[3];
    strides_of(y, ys);
    const fa2_stream_t s = stream_of(x->device());
    const int rc = call([&] {
      return rope_fn(x->data_ptr(), h.s, y.data_ptr(), ys, static_cast<int>(h.B), static_cast<int>(h.H),
                     static_cast<int>(h.N), static_cast<int>(h.d), h.positions, h.wide, h.batch_stride, freq, rotary,
                     interleaved, static_cast<float>(mscale), transposed, type_code(*x), s);
    });
    return result(rc, std::move(y));
  });
}

// (x, weight, positions, inv_freq, eps, interleaved, mscale)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *x = n == 7 ? tensor(a[0]) : nullptr, *pos = x ? tensor(a[2]) : nullptr;
    Heads h;
    const double* freq;
    const void* weight;
    int rotary, code = -1;
    if (!heads_of(x, pos, &h) || !weights(a[1], h.d, x->scalar_type(), x->device(), &weight, &code) || !weight ||
        !frequencies(a[3], x->device(), h.d, &freq, &rotary))
      return none();
    const double eps = PyFloat_AsDouble(a[4]), mscale = PyFloat_AsDouble(a[6]);
    const int interleaved = PyObject_IsTrue(a[5]);
    if (interleaved < 0 || PyErr_Occurred()) return nullptr;
    at::Tensor y = make(x->sizes(), x->scalar_type(), x->device());
    long long ys[3];
    strides_of(y, ys);
    const fa2_stream_t s = stream_of(x->device());
    const int rc = call([&] {
      return norm_fn(x->data_ptr(), h.s, y.data_ptr(), ys, static_cast<int>(h.B), static_cast<int>(h.H),
                     static_cast<int>(h.N), static_cast<int>(h.d), weight, code, static_cast<float>(eps), h.positions,
                     h.wide, h.batch_stride, freq, rotary, interleaved, static_cast<float>(mscale), type_code(*x), s);
    });
    return result(rc, std::move(y));
  });
}

// (dy, x, weight, positions, inv_freq, eps, interleaved, mscale)
PyObject* norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *dy = n == 8 ? tensor(a[0]) : nullptr, *x = dy ? tensor(a[1]) : nullptr;
    const at::Tensor* pos = x ? tensor(a[3]) : nullptr;
    Heads h;
    const double* freq;
    const void* weight;
    int rotary, code = -1;
    if (!heads_of(x, pos, &h) || dy->scalar_type() != x->scalar_type() || dy->sizes() != x->sizes() ||
        dy->device() != x->device() || dy->stride(-1) != 1 ||
        !weights(a[2], h.d, x->scalar_type(), x->device(), &weight, &code) || !weight ||
        !frequencies(a[4], x->device(), h.d, &freq, &rotary))
      return none();
    const double eps = PyFloat_AsDouble(a[5]), mscale = PyFloat_AsDouble(a[7]);
    const int interleaved = PyObject_IsTrue(a[6]);
    if (interleaved < 0 || PyErr_Occurred()) return nullptr;
    at::Tensor dx = make(x->sizes(), x->scalar_type(), x->device()), dw = make({h.d}, at::kFloat, x->device());
    const size_t size = norm_workspace_fn(static_cast<int>(h.d));
    at::Tensor ws = make({static_cast<int64_t>(size > 0 ? size : 1)}, at::kByte, x->device());
    long long gs[3], ys[3];
    strides_of(*dy, gs);
    strides_of(dx, ys);
    const fa2_stream_t s = stream_of(x->device());
    const int rc = call([&] {
      return norm_backward_fn(dy->data_ptr(), gs, x->data_ptr(), h.s, dx.data_ptr(), ys, static_cast<int>(h.B),
                              static_cast<int>(h.H), static_cast<int>(h.N), static_cast<int>(h.d), weight, code,
                              static_cast<float>(eps), h.positions, h.wide, h.batch_stride, freq, rotary, interleaved,
                              static_cast<float>(mscale), type_code(*x), static_cast<float*>(dw.data_ptr()),
                              ws.data_ptr(), size, s);
    });
    if (rc != FA2_OK) return PyLong_FromLong(rc);
    return pair_of(std::move(dx), std::move(dw));
  });
}

// (page_table, lens, refs)
bool tables_of(PyObject* const* a, int page_size, fa2_page_tables* t, at::Device* device) {
  const at::Tensor *table = tensor(a[0]), *lens = tensor(a[1]), *refs = tensor(a[2]);
  if (!table || !lens || !refs || table->dim() != 2 || refs->dim() != 1 || !current(table->device())) return false;
  *device = table->device();
  if (!ints(table, table->sizes(), *device) || !ints(lens, {table->size(0)}, *device) ||
      !ints(refs, refs->sizes(), *device) || !fits_int(table->sizes()) || !fits_int(refs->sizes()))
    return false;
  t->page_table = static_cast<int*>(table->data_ptr());
  t->table_stride = table->stride(0);
  t->table_width = static_cast<int>(table->size(1));
  t->B = static_cast<int>(table->size(0));
  t->lens = static_cast<int*>(lens->data_ptr());
  t->refs = static_cast<int*>(refs->data_ptr());
  t->num_pages = static_cast<int>(refs->size(0));
  t->page_size = page_size;
  return true;
}

// One tensor [..., P, Hkv, S, d] whose pages are dense in that order
bool pools_of(PyObject* o, fa2_page_pools* d, std::vector<void*>* planes, int* page_size, at::Device* device) {
  const at::Tensor* t = tensor(o);
  if (!t || t->dim() < 4 || !current(t->device()) || !fits_int(t->sizes())) return false;
  const int64_t hd = t->size(-1), S = t->size(-2), H = t->size(-3);
  if (t->stride(-1) != 1 || t->stride(-2) != hd || t->stride(-3) != S * hd) return false;
  const int64_t size = t->element_size();
  planes->assign(1, t->data_ptr());
  for (int64_t i = 0; i + 4 < t->dim(); ++i) {
    std::vector<void*> next;
    for (void* p : *planes)
      for (int64_t x = 0; x < t->size(i); ++x) {
        if (next.size() > 256) return false;
        next.push_back(static_cast<char*>(p) + x * t->stride(i) * size);
      }
    planes->swap(next);
  }
  d->planes = planes->data();
  d->num_planes = static_cast<int>(planes->size());
  d->num_pages = static_cast<int>(t->size(-4));
  d->page_stride = t->stride(-4) * size;
  d->page_bytes = H * S * hd * size;
  *page_size = static_cast<int>(S);
  *device = t->device();
  return true;
}

// length of a dense 1-D int32 list, -1 when it is none
int64_t list(const at::Tensor* t, at::Device device) {
  return t && t->dim() == 1 && ints(t, t->sizes(), device) && fits_int(t->sizes()) ? t->size(0) : -1;
}

at::Tensor pages_workspace(int pages, int n, at::Device d, size_t* size) {
  *size = pages_workspace_fn(pages, n);
  return make({static_cast<int64_t>(*size > 0 ? *size : 1)}, at::kByte, d);
}

// An int32 tensor [1] that the workspace follows in the same allocation (an
// allocation costs a small call about two microseconds).
at::Tensor answer_and_workspace(int pages, int n, at::Device d, char** ws, size_t* size) {
  constexpr int64_t kAnswerBytes = 256;
  *size = pages_workspace_fn(pages, n);
  at::Tensor t = make({(kAnswerBytes + static_cast<int64_t>(*size)) / 4}, at::kInt, d);
  *ws = static_cast<char*>(t.data_ptr()) + kAnswerBytes;
  t.unsafeGetTensorImpl()->set_sizes_contiguous({1});
  return t;
}

int* int_ptr(const at::Tensor& t) { return static_cast<int*>(t.data_ptr()); }

// (page_table, lens, refs, add, page_size)
PyObject* pages_reserve(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    fa2_page_tables t;
    at::Device device(at::kCPU);
    if (n != 5 || !PyLong_Check(a[4])) return none();
    const long page = PyLong_AsLong(a[4]);
    if (PyErr_Occurred()) return nullptr;
    if (page < 1 || page > 0x7fffffff || !tables_of(a, static_cast<int>(page), &t, &device)) return none();
    const at::Tensor* add = tensor(a[3]);
    if (list(add, device) != t.B) return none();
    size_t size;
    char* ws;
    at::Tensor missing = answer_and_workspace(t.num_pages, 0, device, &ws, &size);
    const fa2_stream_t s = stream_of(device);
    const int rc = call([&] { return reserve_fn(&t, int_ptr(*add), int_ptr(missing), ws, size, s); });
    return result(rc, std::move(missing));
  });
}

// (page_table, lens, refs, src, dst, pools)
PyObject* pages_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    fa2_page_tables t;
    fa2_page_pools d;
    std::vector<void*> planes;
    int page = 0;
    at::Device device(at::kCPU), there(at::kCPU);
    if (n != 6 || !pools_of(a[5], &d, &planes, &page, &there) || !tables_of(a, page, &t, &device) || there != device ||
        d.num_pages != t.num_pages)
      return none();
    const at::Tensor *src = tensor(a[3]), *dst = tensor(a[4]);
    const int64_t count = list(src, device);
    if (count < 0 || list(dst, device) != count) return none();
    size_t size;
    char* ws;
    at::Tensor missing = answer_and_workspace(t.num_pages, static_cast<int>(count), device, &ws, &size);
    const fa2_stream_t s = stream_of(device);
    const int rc = call([&] {
      return fork_fn(&t, &d, int_ptr(*src), int_ptr(*dst), static_cast<int>(count), int_ptr(missing), ws, size, s);
    });
    return result(rc, std::move(missing));
  });
}

// (page_table, lens, refs, seqs): True, a status, or None
PyObject* pages_free(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    fa2_page_tables t;
    at::Device device(at::kCPU);
    if (n != 4 || !tables_of(a, 16, &t, &device)) return none();
    const at::Tensor* seqs = tensor(a[3]);
    const int64_t count = list(seqs, device);
    if (count < 0) return none();
    const fa2_stream_t s = stream_of(device);
    const int rc = call([&] { return free_fn(&t, int_ptr(*seqs), static_cast<int>(count), s); });
    if (rc != FA2_OK) return PyLong_FromLong(rc);
    Py_RETURN_TRUE;
  });
}

// (page_table, lens, refs, pools)
PyObject* pages_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    fa2_page_tables t;
    fa2_page_pools d;
    std::vector<void*> planes;
    int page = 0;
    at::Device device(at::kCPU), there(at::kCPU);
    if (n != 4 || !pools_of(a[3], &d, &planes, &page, &there) || !tables_of(a, page, &t, &device) || there != device ||
        d.num_pages != t.num_pages)
      return none();
    size_t size;
    at::Tensor ws = pages_workspace(t.num_pages, 0, device, &size), moved = make({t.num_pages}, at::kInt, device);
    const fa2_stream_t s = stream_of(device);
    const int rc = call([&] { return compact_fn(&t, &d, int_ptr(moved), ws.data_ptr(), size, s); });
    return result(rc, std::move(moved));
  });
}

// (pools, src, dst): True, a status, or None
PyObject* pages_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    fa2_page_pools d;
    std::vector<void*> planes;
    int page = 0;
    at::Device device(at::kCPU);
    if (n != 3 || !pools_of(a[0], &d, &planes, &page, &device)) return none();
    const at::Tensor *src = tensor(a[1]), *dst = tensor(a[2]);
    const int64_t count = list(src, device);
    if (count < 0 || list(dst, device) != count) return none();
    size_t size;
    at::Tensor ws = pages_workspace(0, static_cast<int>(count), device, &size);
    const fa2_stream_t s = stream_of(device);
    const int rc =
        call([&] { return copy_fn(&d, int_ptr(*src), int_ptr(*dst), static_cast<int>(count), ws.data_ptr(), size, s); });
    if (rc != FA2_OK) return PyLong_FromLong(rc);
    Py_RETURN_TRUE;
  });
}

// init(addresses): those of the library's functions, in this order
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void** to[] = {reinterpret_cast<void**>(&forward_paged_fn), reinterpret_cast<void**>(&workspace_bytes_fn),
                 reinterpret_cast<void**>(&rope_fn), reinterpret_cast<void**>(&append_fn),
                 reinterpret_cast<void**>(&pages_workspace_fn), reinterpret_cast<void**>(&reserve_fn),
                 reinterpret_cast<void**>(&fork_fn), reinterpret_cast<void**>(&free_fn),
                 reinterpret_cast<void**>(&compact_fn), reinterpret_cast<void**>(&copy_fn),
                 reinterpret_cast<void**>(&append_norm_fn), reinterpret_cast<void**>(&norm_fn),
                 reinterpret_cast<void**>(&norm_backward_fn), reinterpret_cast<void**>(&norm_workspace_fn),
                 reinterpret_cast<void**>(&paged_window_fn), reinterpret_cast<void**>(&paged_prefix_fn),
                 reinterpret_cast<void**>(&prefix_workspace_fn), reinterpret_cast<void**>(&window_fn),
                 reinterpret_cast<void**>(&window_backward_fn), reinterpret_cast<void**>(&window_workspace_fn)};
  constexpr Py_ssize_t count = sizeof to / sizeof to[0];
  if (n != count) {
    PyErr_SetString(PyExc_ValueError, "init takes one address for each function");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < count; ++i) {
    void* p = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
    *to[i] = p;
  }
  Py_RETURN_NONE;
}

#define FA2_METHOD(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {FA2_METHOD(init),          FA2_METHOD(forward_paged), FA2_METHOD(append_paged),
                         FA2_METHOD(rope),          FA2_METHOD(pages_reserve), FA2_METHOD(pages_fork),
                         FA2_METHOD(pages_free),    FA2_METHOD(pages_compact), FA2_METHOD(pages_copy),
                         FA2_METHOD(norm_rope),     FA2_METHOD(norm_rope_backward),
                         FA2_METHOD(forward_paged_window), FA2_METHOD(forward_paged_prefix),
                         FA2_METHOD(forward_window), FA2_METHOD(backward_window),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
