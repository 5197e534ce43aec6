// The host side of the attention operators' usual calls, as a Python extension: checks, allocations
// and the C ABI call. These calls are short on the GPU (3 to 20 us), and from Python the
// same steps took 14 to 30 us of host time, most of it in some sixty small Python and ctypes steps.
//
// Every function takes its arguments in order and returns its result, the status (an int) of a call
// that the C ABI refused, or None for anything that is not a plain call (another stream, tensors of
// the wrong kind, ...): the caller then takes its own way, which checks step by step, says what
// is wrong, and makes the call if nothing is.
#include <torch/csrc/autograd/python_variable.h>
#include <torch/extension.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <climits>

#include "sa_sketch.h"

namespace {

using at::Tensor;

// Arguments of a call; `ok` turns false at the first one that is not as it should be.
struct Args {
  PyObject* const* v;
  bool ok = true;
  c10::Device dev{c10::kCPU};

  bool need(bool c) {
    ok = ok && c;
    return ok;
  }
  bool none(int i) const { return v[i] == Py_None; }
  const Tensor* tensor(int i) {  // (exactly a Tensor: what a subclass means is for Python)
    if (!need(THPVariable_CheckExact(v[i]))) return nullptr;
    return &THPVariable_Unpack(v[i]);
  }
  const Tensor* first(int i, int dim) {  // the tensor whose device is the call's
    const Tensor* t = tensor(i);
    if (!t || !need(t->is_cuda() && t->dim() == dim)) return nullptr;
    dev = t->device();
    return t;
  }
  const Tensor* on(int i, at::ScalarType kind, at::IntArrayRef shape) {  // contiguous
    const Tensor* t = tensor(i);
    if (!t || !need(t->scalar_type() == kind && t->device() == dev && t->sizes() == shape && t->is_contiguous()))
      return nullptr;
    return t;
  }
  void* optional(int i, at::ScalarType kind, at::IntArrayRef shape) {
    if (none(i)) return nullptr;
    const Tensor* t = on(i, kind, shape);
    return t ? t->data_ptr() : nullptr;
  }
  // [n, heads, d] bf16 whose rows may be strided; the rows' distance
  const Tensor* heads(int i, int64_t n, int64_t h, int64_t d, int64_t* stride) {
    const Tensor* t = tensor(i);
    if (!t || !need(t->dim() == 3 && t->scalar_type() == at::kBFloat16 && t->device() == dev && t->size(0) == n &&
                    t->size(1) == h && t->size(2) == d))
      return nullptr;
    need(t->stride(2) == 1 && (t->stride(1) == d || h == 1));
    *stride = n > 1 ? t->stride(0) : h * d;
    return t;
  }
  int64_t integer(int i, int64_t lo, int64_t hi) {
    if (!need(PyLong_CheckExact(v[i]))) return 0;
    int overflow = 0;
    const long long x = PyLong_AsLongLongAndOverflow(v[i], &overflow);
    need(overflow == 0 && x >= lo && x <= hi);
    return x;
  }
  float scale(int i, int64_t d) {
    if (none(i)) return (float)std::pow((double)d, -0.5);
    if (!need(PyFloat_CheckExact(v[i]))) return 0.f;
    return (float)PyFloat_AS_DOUBLE(v[i]);
  }
};

// (at::empty without the dispatcher, half its time)
Tensor empty(at::IntArrayRef shape, at::ScalarType kind, c10::Device dev) {
  return at::detail::empty_cuda(shape, kind, dev, std::nullopt);
}

// Result dictionary; the names are interned once.
struct Result {
  PyObject* d = PyDict_New();
  void set(PyObject* name, const Tensor& t) {
    PyObject* x = THPVariable_Wrap(t);
    if (!x || PyDict_SetItem(d, name, x) < 0) PyErr_Clear();
    Py_XDECREF(x);
  }
};
PyObject *kOut, *kLse, *kRest, *kWs, *kDQ, *kDK, *kDV, *kSlots, *kNewOffsets, *kSeqLens, *kFreeUsed;

// A given workspace, or a new one of `bytes`.
bool workspace(Args& a, int i, size_t bytes, Tensor* ws) {
  if (!a.none(i)) {
    const Tensor* t = a.tensor(i);
    if (!t || !a.need(t->device() == a.dev && t->is_contiguous())) return false;  // (nbytes of them are there)
    *ws = *t;
    return true;
  }
  if (!a.need(bytes > 0)) return false;
  *ws = empty({(int64_t)bytes}, at::kByte, a.dev);
  return true;
}

PyObject* finish(int st, Result& r) {
  if (st == SA_OK) return r.d;
  Py_DECREF(r.d);
  return PyLong_FromLong(st);
}

// Without the GIL, on the device of the call and its current stream.
template <typename F>
int run(F&& f, c10::Device dev) {
  int st;
  void* s = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  Py_BEGIN_ALLOW_THREADS;
  st = f(s);
  Py_END_ALLOW_THREADS;
  return st;
}

struct Cross {
  const Tensor *Q, *qo, *K, *V, *ko;
  const uint8_t* mask;
  int64_t n_q, H, d, n_kv, Hkv, qs, ks, vs;
  int R;
  // arguments 0-5: Q, q_offsets, K, V, kv_offsets, key_mask
  bool read(Args& a) {
    if (!(Q = a.first(0, 3)) || !(K = a.tensor(2)) || !a.need(K->dim() == 3)) return false;
    n_q = Q->size(0), H = Q->size(1), d = Q->size(2), n_kv = K->size(0), Hkv = K->size(1);
    a.heads(0, n_q, H, d, &qs);
    a.heads(2, n_kv, Hkv, d, &ks);
    V = a.heads(3, n_kv, Hkv, d, &vs);
    if (!a.need(Hkv > 0 && H > 0 && H % Hkv == 0 && H <= INT_MAX) || !(qo = a.tensor(1)) ||
        !a.need(qo->dim() == 1 && qo->numel() >= 1 && qo->numel() <= INT_MAX))
      return false;
    R = (int)(qo->numel() - 1);
    a.on(1, at::kLong, {R + 1});
    ko = a.on(4, at::kLong, {R + 1});
    mask = nullptr;
    if (a.ok && !a.none(5)) {
      const Tensor* m = a.tensor(5);
      if (m) mask = (const uint8_t*)a.optional(5, m->scalar_type() == at::kByte ? at::kByte : at::kBool, {n_kv});
    }
    return a.ok;
  }
};

// (Q, q_offsets, K, V, kv_offsets, key_mask, scale, want_rest, ws)
PyObject* cross_forward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a{v};
  Cross c;
  if (n != 9 || !c.read(a)) Py_RETURN_NONE;
  const float scale = a.scale(6, c.d);
  if (!a.ok) Py_RETURN_NONE;
  c10::cuda::OptionalCUDAGuard guard(a.dev);
  Tensor ws;
  if (!workspace(a, 8, a.none(8) ? sa_cross_attn_workspace_size(c.R, c.n_q, c.n_kv, (int)c.H, (int)c.Hkv, (int)c.d, 0) : 0,
                 &ws))
    Py_RETURN_NONE;
  const bool want_rest = v[7] != Py_False;
  const Tensor out = empty({c.n_q, c.H, c.d}, at::kBFloat16, a.dev), lse = empty({c.n_q, c.H}, at::kFloat, a.dev);
  Tensor rest;
  if (want_rest) rest = empty({c.n_q, c.H, c.d}, at::kBFloat16, a.dev);
  const int st = run([&](void* s) {
    return sa_cross_attn_forward(c.Q->data_ptr(), c.qs, (const int64_t*)c.qo->data_ptr(), c.R, c.n_q, (int)c.H, (int)c.d,
                                 c.K->data_ptr(), c.ks, c.V->data_ptr(), c.vs, (const int64_t*)c.ko->data_ptr(), c.n_kv,
                                 (int)c.Hkv, c.mask, scale, out.data_ptr(), want_rest ? rest.data_ptr() : nullptr,
                                 (float*)lse.data_ptr(), ws.data_ptr(), ws.nbytes(), s);
  }, a.dev);
  Result r;
  r.set(kOut, out);
  r.set(kLse, lse);
  if (want_rest) r.set(kRest, rest);
  r.set(kWs, ws);
  return finish(st, r);
  END_HANDLE_TH_ERRORS
}

// (Q, q_offsets, K, V, kv_offsets, key_mask, scale, out, lse, rest, dout, ws)
PyObject* cross_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a{v};
  Cross c;
  if (n != 12 || !c.read(a)) Py_RETURN_NONE;
  const float scale = a.scale(6, c.d);
  const Tensor* out = a.on(7, at::kBFloat16, {c.n_q, c.H, c.d});
  const Tensor* lse = a.on(8, at::kFloat, {c.n_q, c.H});
  void* rest = a.optional(9, at::kBFloat16, {c.n_q, c.H, c.d});
  const Tensor* dout = a.on(10, at::kBFloat16, {c.n_q, c.H, c.d});
  if (!a.ok) Py_RETURN_NONE;
  c10::cuda::OptionalCUDAGuard guard(a.dev);
  Tensor ws;
  if (!workspace(a, 11, a.none(11) ? sa_cross_attn_workspace_size(c.R, c.n_q, c.n_kv, (int)c.H, (int)c.Hkv, (int)c.d, 1) : 0,
                 &ws))
    Py_RETURN_NONE;
  const Tensor dQ = empty({c.n_q, c.H, c.d}, at::kBFloat16, a.dev), dK = empty({c.n_kv, c.Hkv, c.d}, at::kBFloat16, a.dev),
               dV = empty({c.n_kv, c.Hkv, c.d}, at::kBFloat16, a.dev);
  const int st = run([&](void* s) {
    return sa_cross_attn_backward(c.Q->data_ptr(), c.qs, (const int64_t*)c.qo->data_ptr(), c.R, c.n_q, (int)c.H,
                                  (int)c.d, c.K->data_ptr(), c.ks, c.V->data_ptr(), c.vs,
                                  (const int64_t*)c.ko->data_ptr(), c.n_kv, (int)c.Hkv, c.mask, scale, out->data_ptr(),
                                  rest, (const float*)lse->data_ptr(), dout->data_ptr(), dQ.data_ptr(), dK.data_ptr(),
                                  dV.data_ptr(), ws.data_ptr(), ws.nbytes(), s);
  }, a.dev);
  Result r;
  r.set(kDQ, dQ);
  r.set(kDK, dK);
  r.set(kDV, dV);
  r.set(kWs, ws);
  return finish(st, r);
  END_HANDLE_TH_ERRORS
}

// (cached_lens, new_lens, free_pages, block_table, page_size, n_slots, free_used, ws)
PyObject* page_tables(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a{v};
  const Tensor* cached = n == 8 ? a.first(0, 1) : nullptr;
  if (!cached || !a.need(cached->numel() <= INT_MAX)) Py_RETURN_NONE;
  const int64_t R = cached->numel();
  const Tensor *free_pages = a.tensor(2), *table = a.tensor(3);
  if (!a.ok || !a.need(free_pages->dim() == 1 && table->dim() == 2 && table->size(1) <= INT_MAX)) Py_RETURN_NONE;
  const int64_t n_free = free_pages->numel(), max_pages = table->size(1);
  a.on(0, at::kInt, {R});
  const Tensor* fresh = a.on(1, at::kInt, {R});
  a.on(2, at::kInt, {n_free});
  a.on(3, at::kInt, {R, max_pages});
  const int64_t page = a.integer(4, 0, INT_MAX), n_slots = a.integer(5, 0, LLONG_MAX);
  void* used = a.optional(6, at::kLong, {1});
  if (!a.ok) Py_RETURN_NONE;
  c10::cuda::OptionalCUDAGuard guard(a.dev);
  Tensor ws;
  if (!workspace(a, 7, 256, &ws)) Py_RETURN_NONE;
  const Tensor slots = empty({n_slots}, at::kLong, a.dev), offsets = empty({R + 1}, at::kLong, a.dev),
               lens = empty({R}, at::kInt, a.dev), used_out = empty({1}, at::kLong, a.dev);
  const int st = run([&](void* s) {
    return sa_page_tables((const int32_t*)cached->data_ptr(), (const int32_t*)fresh->data_ptr(), (int)R, (int)page,
                          (const int32_t*)free_pages->data_ptr(), n_free, (const int64_t*)used,
                          (int32_t*)table->data_ptr(), (int)max_pages, n_slots, (int64_t*)slots.data_ptr(),
                          (int64_t*)offsets.data_ptr(), (int32_t*)lens.data_ptr(), (int64_t*)used_out.data_ptr(),
                          ws.data_ptr(), ws.nbytes(), s);
  }, a.dev);
  Result r;
  r.set(kSlots, slots);
  r.set(kNewOffsets, offsets);
  r.set(kSeqLens, lens);
  r.set(kFreeUsed, used_out);
  r.set(kWs, ws);
  return finish(st, r);
  END_HANDLE_TH_ERRORS
}

// A paged cache: K, V, k_scales, v_scales at arguments i ...
struct Cache {
  const Tensor *K, *V;
  void *ks = nullptr, *vs = nullptr;
  int64_t n_pages, Hkv, page, d;
  int format;
  bool read(Args& a, int i) {
    if (!(K = a.tensor(i)) || !a.need(K->dim() == 4)) return false;
    const bool fp8 = K->scalar_type() == at::kFloat8_e4m3fn;
    format = fp8 ? SA_CODEC_FP8 : SA_CODEC_BF16;
    const at::ScalarType kind = fp8 ? at::kFloat8_e4m3fn : at::kBFloat16;
    n_pages = K->size(0), Hkv = K->size(1), page = K->size(2), d = K->size(3);
    a.on(i, kind, {n_pages, Hkv, page, d});
    V = a.on(i + 1, kind, {n_pages, Hkv, page, d});
    a.need(a.none(i + 2) == !fp8 && a.none(i + 3) == !fp8);
    if (!a.need(Hkv <= INT_MAX && page <= INT_MAX && d <= INT_MAX)) return false;
    ks = a.optional(i + 2, at::kFloat, {n_pages, Hkv, page});
    vs = a.optional(i + 3, at::kFloat, {n_pages, Hkv, page});
    return a.ok;
  }
};

// (K, V, slots, cache K, cache V, k_scales, v_scales) -> status
PyObject* paged_append(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a{v};
  const Tensor* K = n == 7 ? a.first(0, 3) : nullptr;
  Cache c;
  if (!K || !c.read(a, 3)) Py_RETURN_NONE;
  const int64_t rows = K->size(0);
  int64_t ks = 0, vs = 0;
  a.heads(0, rows, c.Hkv, c.d, &ks);
  const Tensor* V = a.heads(1, rows, c.Hkv, c.d, &vs);
  const Tensor* slots = a.on(2, at::kLong, {rows});
  if (!a.ok) Py_RETURN_NONE;
  c10::cuda::OptionalCUDAGuard guard(a.dev);
  return PyLong_FromLong(run([&](void* s) {
    return sa_paged_append(K->data_ptr(), ks, V->data_ptr(), vs, (const int64_t*)slots->data_ptr(), rows, (int)c.Hkv,
                           (int)c.d, c.format, c.K->data_ptr(), c.V->data_ptr(), (float*)c.ks, (float*)c.vs, c.n_pages,
                           (int)c.page, s);
  }, a.dev));
  END_HANDLE_TH_ERRORS
}

// (Q, cache K, cache V, k_scales, v_scales, block_table, seq_lens, window, scale, ws)
PyObject* paged_attention(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a{v};
  const Tensor* Q = n == 10 ? a.first(0, 3) : nullptr;
  Cache c;
  if (!Q || !c.read(a, 1)) Py_RETURN_NONE;
  const int64_t R = Q->size(0), H = Q->size(1);
  int64_t qs = 0;
  a.heads(0, R, H, c.d, &qs);
  const Tensor* table = a.tensor(5);
  if (!a.need(c.Hkv > 0 && H > 0 && H % c.Hkv == 0 && H <= INT_MAX && R <= INT_MAX) ||
      !a.need(table->dim() == 2 && table->size(1) <= INT_MAX))
    Py_RETURN_NONE;
  const int64_t max_pages = table->size(1);
  a.on(5, at::kInt, {R, max_pages});
  const Tensor* lens = a.on(6, at::kInt, {R});
  const int64_t window = a.integer(7, LLONG_MIN, LLONG_MAX);
  const float scale = a.scale(8, c.d);
  if (!a.ok) Py_RETURN_NONE;
  c10::cuda::OptionalCUDAGuard guard(a.dev);
  Tensor ws;
  if (!workspace(a, 9, a.none(9) ? sa_paged_attn_workspace_size((int)R, (int)H, (int)c.Hkv, (int)c.d) : 0, &ws))
    Py_RETURN_NONE;
  const Tensor out = empty({R, H, c.d}, at::kBFloat16, a.dev), lse = empty({R, H}, at::kFloat, a.dev);
  const int st = run([&](void* s) {
    return sa_paged_attn(Q->data_ptr(), qs, (int)R, (int)H, (int)c.d, c.K->data_ptr(), c.V->data_ptr(),
                         (const float*)c.ks, (const float*)c.vs, c.format, c.n_pages, (int)c.page, (int)c.Hkv,
                         (const int32_t*)table->data_ptr(), (int)max_pages, (const int32_t*)lens->data_ptr(), window,
                         scale, out.data_ptr(), (float*)lse.data_ptr(), ws.data_ptr(), ws.nbytes(), s);
  }, a.dev);
  Result r;
  r.set(kOut, out);
  r.set(kLse, lse);
  r.set(kWs, ws);
  return finish(st, r);
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
#define SA_CALL(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
    SA_CALL(cross_forward), SA_CALL(cross_backward), SA_CALL(page_tables), SA_CALL(paged_append),
    SA_CALL(paged_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  struct { PyObject** to; const char* name; } names[] = {
      {&kOut, "out"}, {&kLse, "lse"}, {&kRest, "rest"}, {&kWs, "_ws"}, {&kDQ, "dQ"}, {&kDK, "dK"}, {&kDV, "dV"},
      {&kSlots, "slots"}, {&kNewOffsets, "new_offsets"}, {&kSeqLens, "seq_lens"}, {&kFreeUsed, "free_used"}};
  for (auto& x : names)
    if (!(*x.to = PyUnicode_InternFromString(x.name))) return nullptr;
  return PyModule_Create(&kModule);
}
