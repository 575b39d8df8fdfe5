// The serving calls from Python without the interpreter's share: a call on small
// tensors takes the GPU 2 to 9 us, and checking its arguments, allocating its
// outputs and passing 10 to 20 arguments through ctypes took Python 8 to 13.
//
// Each function takes the address of the C entry point (of whichever build of
// the library is selected) and the call's arguments, does what the function of
// the same name in binding.py does for arguments that are all right, and returns
// its results. It returns None, before anything is enqueued, for anything else:
// binding.py then finds what is wrong and says it. A status of the C call other
// than AWQ_OK comes back as an int.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "../../include/awq.h"

namespace {

// A strided CUDA tensor of the current device, or NULL.
struct Here {
  int dev = -1;
  const at::Tensor* operator()(PyObject* o) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided) return nullptr;
    if (dev < 0) dev = c10::cuda::current_device();
    return t.get_device() == dev ? &t : nullptr;
  }
  awq_stream_t stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

bool is(const at::Tensor* t, at::ScalarType type, int64_t dim) {
  return t && t->scalar_type() == type && t->dim() == dim && t->is_contiguous();
}
// bf16 or fp16 of so many axes, the last one contiguous
bool rows(const at::Tensor* t, int64_t dim, awq_dtype& code) {
  if (!t || t->dim() != dim || (t->stride(dim - 1) != 1 && t->size(dim - 1) > 1)) return false;
  if (t->scalar_type() != at::kBFloat16 && t->scalar_type() != at::kHalf) return false;
  code = t->scalar_type() == at::kHalf ? AWQ_DTYPE_F16 : AWQ_DTYPE_BF16;
  return true;
}
// elements from one entry of an axis to the next (the stride of a single entry means nothing)
int64_t pitch(const at::Tensor* t, int64_t axis) { return t->size(axis) > 1 ? t->stride(axis) : 0; }
bool cache_of(const at::Tensor* t, const awq_kv4cfg& c) {
  if (c.group < 1 || c.head_dim < 1 || c.page_size < 1 || !is(t, at::kInt, 3)) return false;
  return t->size(1) == c.n_kv_heads &&
         t->size(2) * 4 == (int64_t)c.page_size * (c.head_dim + 8 * (c.head_dim / c.group));
}

at::Tensor fresh(at::IntArrayRef size, const at::Tensor& like, at::ScalarType type) {
  return at::empty(size, like.options().dtype(type));
}

template <typename F>
F* entry(PyObject* o) {
  return reinterpret_cast<F*>(PyLong_AsVoidPtr(o));
}
// The C call without the interpreter's lock, which comes back whatever happens.
// What may throw (a tensor's data_ptr() does where it has no storage, inside
// torch.func's transforms for one) is evaluated before: arguments are values here.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F, typename... A>
awq_status run(PyObject* address, A... arg) {
  F* f = entry<F>(address);
  Unlocked unlocked;
  return f(arg...);
}

PyObject* none() {
  PyErr_Clear();
  Py_RETURN_NONE;
}
PyObject* pair(awq_status st, at::Tensor a, at::Tensor b) {
  if (st != AWQ_OK) return PyLong_FromLong(st);
  PyObject *x = THPVariable_Wrap(std::move(a)), *y = THPVariable_Wrap(std::move(b));
  PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// (entry, X, s or None, mode with s)
PyObject* quantize_int8(PyObject* const* arg) {
  Here here;
  const at::Tensor *X = here(arg[1]), *s = arg[2] == Py_None ? nullptr : here(arg[2]);
  awq_dtype code;
  if (!rows(X, 2, code)) return none();
  const int64_t n = X->size(0), d = X->size(1);
  if (n == 0) return none();
  if (arg[2] != Py_None && !(is(s, at::kFloat, 1) && s->size(0) == d)) return none();
  const auto mode = s ? (awq_scale_mode)PyLong_AsLong(arg[3]) : AWQ_SCALE_NONE;
  at::Tensor q = fresh({n, d}, *X, at::kChar), step = fresh({n}, *X, at::kFloat);
  const int64_t ld = n > 1 ? X->stride(0) : d > 8 ? d : 8;
  const awq_status st = run<decltype(awq_quantize_int8)>(
      arg[0], X->data_ptr(), code, ld, s ? (const float*)s->data_ptr() : nullptr, mode, n, d, (int8_t*)q.data_ptr(),
      (float*)step.data_ptr(), here.stream());
  return pair(st, std::move(q), std::move(step));
}

// (entry, xq, x_step, wq, w_step, bias or None, fp16 output, workspace: the error word)
PyObject* w8a8_gemm(PyObject* const* arg) {
  Here here;
  const at::Tensor *x = here(arg[1]), *dx = here(arg[2]), *w = here(arg[3]), *dw = here(arg[4]), *ws = here(arg[7]);
  const at::Tensor* bias = arg[5] == Py_None ? nullptr : here(arg[5]);
  if (!is(x, at::kChar, 2) || !is(w, at::kChar, 2) || !is(dx, at::kFloat, 1) || !is(dw, at::kFloat, 1) || !is(ws, at::kByte, 1))
    return none();
  const int64_t n = x->size(0), d_in = x->size(1), d_out = w->size(0);
  if (n == 0 || w->size(1) != d_in || dx->size(0) != n || dw->size(0) != d_out) return none();
  if (arg[5] != Py_None && !(is(bias, at::kFloat, 1) && bias->size(0) == d_out)) return none();
  const bool f16 = arg[6] == Py_True;
  at::Tensor y = fresh({n, d_out}, *x, f16 ? at::kHalf : at::kBFloat16);
  const awq_status st = run<decltype(awq_w8a8_gemm)>(
      arg[0], (const int8_t*)x->data_ptr(), (const float*)dx->data_ptr(), (const int8_t*)w->data_ptr(),
      (const float*)dw->data_ptr(), bias ? (const float*)bias->data_ptr() : nullptr,
      f16 ? AWQ_DTYPE_F16 : AWQ_DTYPE_BF16, n, d_out, d_in, y.data_ptr(), ws->data_ptr(), (size_t)ws->numel(),
      here.stream());
  return st != AWQ_OK ? PyLong_FromLong(st) : THPVariable_Wrap(std::move(y));
}

// (entry, k, v, slots, cache, address of the cfg): 0, a status or None
PyObject* kv4_append(PyObject* const* arg) {
  Here here;
  const at::Tensor *k = here(arg[1]), *v = here(arg[2]), *slots = here(arg[3]), *cache = here(arg[4]);
  const awq_kv4cfg cfg = *static_cast<const awq_kv4cfg*>(PyLong_AsVoidPtr(arg[5]));
  awq_dtype code, code_v;
  if (!rows(k, 3, code) || !rows(v, 3, code_v) || code != code_v || k->sizes() != v->sizes()) return none();
  const int64_t T = k->size(0);
  if (k->size(1) != cfg.n_kv_heads || k->size(2) != cfg.head_dim || !is(slots, at::kInt, 1) || slots->size(0) != T ||
      !cache_of(cache, cfg))
    return none();
  return PyLong_FromLong(run<decltype(awq_kv4_append)>(
      arg[0], k->data_ptr(), v->data_ptr(), code, T, pitch(k, 0), pitch(k, 1), pitch(v, 0), pitch(v, 1),
      (const int32_t*)slots->data_ptr(), cache->data_ptr(), cache->size(0), &cfg, here.stream()));
}

// (entry, cache, slots, address of the cfg, fp16 outputs)
PyObject* kv4_gather(PyObject* const* arg) {
  Here here;
  const at::Tensor *cache = here(arg[1]), *slots = here(arg[2]);
  const awq_kv4cfg cfg = *static_cast<const awq_kv4cfg*>(PyLong_AsVoidPtr(arg[3]));
  if (!cache_of(cache, cfg) || !is(slots, at::kInt, 1)) return none();
  const bool f16 = arg[4] == Py_True;
  const int64_t T = slots->size(0);
  const at::ScalarType type = f16 ? at::kHalf : at::kBFloat16;
  at::Tensor k = fresh({T, cfg.n_kv_heads, cfg.head_dim}, *cache, type), v = fresh({T, cfg.n_kv_heads, cfg.head_dim}, *cache, type);
  const awq_status st = run<decltype(awq_kv4_gather)>(
      arg[0], cache->data_ptr(), cache->size(0), (const int32_t*)slots->data_ptr(), T, &cfg, k.data_ptr(), v.data_ptr(),
      f16 ? AWQ_DTYPE_F16 : AWQ_DTYPE_BF16, here.stream());
  return pair(st, std::move(k), std::move(v));
}

// (entry, entry of the workspace's size, q, cache, table, lens, address of the cfg, q_start or None, max_q or None,
//  scale or None, lse)
PyObject* kv4_attention(PyObject* const* arg) {
  Here here;
  const at::Tensor *q = here(arg[2]), *cache = here(arg[3]), *table = here(arg[4]), *lens = here(arg[5]);
  const awq_kv4cfg cfg = *static_cast<const awq_kv4cfg*>(PyLong_AsVoidPtr(arg[6]));
  const at::Tensor* start = arg[7] == Py_None ? nullptr : here(arg[7]);
  awq_dtype code;
  if (!rows(q, 3, code) || q->size(2) != cfg.head_dim || !cache_of(cache, cfg) || !is(lens, at::kInt, 1) || !is(table, at::kInt, 2))
    return none();
  const int64_t T = q->size(0), heads = q->size(1), D = q->size(2), batch = lens->size(0);
  if (T == 0 || table->size(0) != batch) return none();
  if (arg[7] == Py_None ? T != batch : !(is(start, at::kInt, 1) && start->size(0) == batch + 1 && arg[8] != Py_None))
    return none();
  if ((arg[8] != Py_None && !PyLong_CheckExact(arg[8])) || (arg[9] != Py_None && !PyFloat_CheckExact(arg[9]))) return none();
  const long long max_q = arg[8] == Py_None ? 1 : PyLong_AsLongLong(arg[8]);
  if (max_q == -1 && PyErr_Occurred()) return none();
  const double scale = arg[9] == Py_None ? 1.0 / std::sqrt((double)D) : PyFloat_AS_DOUBLE(arg[9]);
  const bool with_lse = arg[10] == Py_True;
  const size_t need = entry<decltype(awq_kv4_attention_workspace_size)>(arg[1])(batch, heads, max_q, &cfg);
  at::Tensor out = fresh({T, heads, D}, *q, q->scalar_type()), ws = fresh({need > 256 ? (int64_t)need : 256}, *q, at::kByte), lse;
  if (with_lse) lse = fresh({T, heads}, *q, at::kFloat);
  const awq_status st = run<decltype(awq_kv4_attention)>(
      arg[0], q->data_ptr(), code, pitch(q, 0), pitch(q, 1), T, heads, start ? (const int32_t*)start->data_ptr() : nullptr,
      max_q, cache->data_ptr(), cache->size(0), (const int32_t*)table->data_ptr(), table->size(1),
      (const int32_t*)lens->data_ptr(), batch, (float)scale, &cfg, out.data_ptr(),
      with_lse ? (float*)lse.data_ptr() : nullptr, ws.data_ptr(), (size_t)ws.numel(), here.stream());
  if (with_lse) return pair(st, std::move(out), std::move(lse));
  return st != AWQ_OK ? PyLong_FromLong(st) : THPVariable_Wrap(std::move(out));
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected", N);
    return nullptr;
  }
  try {
    return F(arg);
  } catch (...) {  // (an allocation that failed, a tensor without storage: the long way says so)
    return none();
  }
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<quantize_int8, 4>("quantize_int8"),   method<w8a8_gemm, 8>("w8a8_gemm"),
                         method<kv4_append, 6>("kv4_append"),         method<kv4_gather, 5>("kv4_gather"),
                         method<kv4_attention, 11>("kv4_attention"),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "awq_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_awq_calls(void) { return PyModule_Create(&module); }
