// Python calls of the paged-cache attention (coli_attn.h).  A serving loop makes one of these calls per layer and step, and
// their small forms run for a few microseconds on the GPU, so the checks of the tensors, the new output and the
// call itself are here and not in Python.  Everything else of the binding is in attn.py.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "coli_attn.h"

namespace {

// what attn.py keeps of an engine (a ctypes structure with the same fields)
struct Engine {
  coli_attn* handle;
  int32_t n_q, n_kv, head_dim, dtype, device;
  float scale;
};

// what it keeps of a batch
struct Batch {
  coli_attn_batch batch;
  int32_t device;
};

struct Error {};  // the Python exception is set

[[noreturn]] void fail(const char* format, const char* what) {
  PyErr_Format(PyExc_ValueError, format, what);
  throw Error();
}

template <class T>
T* pointer(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Error();
  return static_cast<T*>(p);
}

// the batch of a call, whose tensors have to be on the engine's device
const coli_attn_batch& batch(PyObject* o, const Engine& e) {
  const Batch& b = *pointer<Batch>(o);
  if (b.device != e.device) fail("%s on the engine's device", "the batch's tensors are");
  return b.batch;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Error();
  return v;
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) fail("%s: a tensor", what);
  return THPVariable_Unpack(o);
}

// [n_tokens, heads, head_dim] of the engine's type on its device, a token's heads contiguous -> the token stride
int64_t heads(const at::Tensor& t, const Engine& e, int32_t n, const coli_attn_batch& b, const char* what) {
  const auto type = e.dtype == COLI_ATTN_BF16 ? at::kBFloat16 : at::kHalf;
  if (t.dim() != 3 || t.size(0) != b.n_tokens || t.size(1) != n || t.size(2) != e.head_dim || t.scalar_type() != type ||
      !t.is_cuda() || t.get_device() != e.device)
    fail("%s: [n_tokens, heads, head_dim] of the engine's type on its device", what);
  if (t.stride(2) != 1 || (n > 1 && t.stride(1) != e.head_dim)) fail("%s: a token's heads are contiguous", what);
  return b.n_tokens > 1 ? t.stride(0) : (int64_t)n * e.head_dim;
}

const int32_t* int32s(PyObject* o, const Engine& e, const char* what) {
  const at::Tensor& t = tensor(o, what);
  if (t.dim() != 1 || t.scalar_type() != at::kInt || (t.numel() > 1 && t.stride(0) != 1) || !t.is_cuda() ||
      t.get_device() != e.device)
    fail("%s: a contiguous 1-dimensional int32 tensor on the engine's device", what);
  return static_cast<const int32_t*>(t.data_ptr());
}

float* log_sums(PyObject* o, const Engine& e, const coli_attn_batch& b) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "lse");
  if (t.dim() != 2 || t.size(0) != b.n_tokens || t.size(1) != e.n_q || t.scalar_type() != at::kFloat || !t.is_cuda() ||
      t.get_device() != e.device || !t.is_contiguous())
    fail("%s: contiguous float32 [n_tokens, n_q]", "lse");
  return static_cast<float*>(t.data_ptr());
}

// the stream of a call: the current one (None), or a handle
c10::cuda::CUDAStream stream_of(PyObject* o, const Engine& e) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(e.device);
  const auto handle = (cudaStream_t)PyLong_AsVoidPtr(o);
  if (!handle && PyErr_Occurred()) throw Error();
  if (!handle || handle == cudaStreamLegacy) return c10::cuda::getDefaultCUDAStream(e.device);
  return c10::cuda::getStreamFromExternal(handle, e.device);
}

// The caller's output or a new one, in memory of the call's stream: what an earlier owner of the same memory has queued on
// another one may not have run when the call does.
at::Tensor output(PyObject* o, const at::Tensor& like, const Engine& e, const coli_attn_batch& b, int64_t* stride,
                  const c10::cuda::CUDAStream& stream, bool current) {
  if (o != Py_None) {
    const at::Tensor& t = tensor(o, "out");
    *stride = heads(t, e, e.n_q, b, "out");
    return t;
  }
  *stride = (int64_t)e.n_q * e.head_dim;
  c10::cuda::OptionalCUDAStreamGuard guard;
  if (!current) guard.reset_stream(stream);
  return at::empty({b.n_tokens, e.n_q, e.head_dim}, like.options());
}

// the result of a call: its output, or its status where it is not COLI_OK
PyObject* result(int status, const at::Tensor* out) {
  if (status != COLI_OK) return PyLong_FromLong(status);
  if (!out) Py_RETURN_NONE;
  return THPVariable_Wrap(*out);
}

template <class F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F body) {
  if (have != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return body();
  } catch (const Error&) {
    return nullptr;
  } catch (const std::exception& x) {  // an allocation that failed
    PyErr_SetString(PyExc_RuntimeError, x.what());
    return nullptr;
  }
}

// append(engine, cache, batch, k, v, q, q_out, pos_base, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    const Engine& e = *pointer<Engine>(a[0]);
    const auto* kv = pointer<coli_attn_kv>(a[1]);
    const coli_attn_batch& b = batch(a[2], e);
    const at::Tensor &k = tensor(a[3], "k"), &v = tensor(a[4], "v");
    const int64_t ks = heads(k, e, e.n_kv, b, "k"), vs = heads(v, e, e.n_kv, b, "v");
    const int32_t* base = a[7] == Py_None ? nullptr : int32s(a[7], e, "pos_base");
    const auto stream = stream_of(a[8], e);
    if (a[5] == Py_None)
      return result(coli_attn_append(e.handle, kv, &b, nullptr, 0, k.data_ptr(), ks, v.data_ptr(), vs, nullptr, 0, base,
                                     stream.stream()),
                    nullptr);
    const at::Tensor& q = tensor(a[5], "q");
    const int64_t qs = heads(q, e, e.n_q, b, "q");
    int64_t os;
    const at::Tensor out = output(a[6], q, e, b, &os, stream, a[8] == Py_None);
    return result(coli_attn_append(e.handle, kv, &b, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
                                   out.data_ptr(), os, base, stream.stream()),
                  &out);
  });
}

// window(engine, cache, batch, q, window, sinks, scale, out, lse, stream)
PyObject* window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const Engine& e = *pointer<Engine>(a[0]);
    const auto* kv = pointer<coli_attn_kv>(a[1]);
    const coli_attn_batch& b = batch(a[2], e);
    const at::Tensor& q = tensor(a[3], "q");
    const int64_t qs = heads(q, e, e.n_q, b, "q");
    int64_t w = integer(a[4]), s = integer(a[5]);
    w = w < -1 ? -1 : w > INT32_MAX ? INT32_MAX : w;
    s = s < -1 ? -1 : s > INT32_MAX ? INT32_MAX : s;
    const float scale = a[6] == Py_None ? e.scale : (float)PyFloat_AsDouble(a[6]);
    if (PyErr_Occurred()) throw Error();
    float* lse = log_sums(a[8], e, b);
    int64_t os;
    const auto stream = stream_of(a[9], e);
    const at::Tensor out = output(a[7], q, e, b, &os, stream, a[9] == Py_None);
    return result(coli_attn_window(e.handle, kv, &b, q.data_ptr(), qs, (int)w, (int)s, scale, out.data_ptr(), os, lse,
                                   stream.stream()),
                  &out);
  });
}

// prefix(engine, cache, batch, prefix_table, prefix_len, q, scale, out, lse, stream)
PyObject* prefix(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const Engine& e = *pointer<Engine>(a[0]);
    const auto* kv = pointer<coli_attn_kv>(a[1]);
    const coli_attn_batch& b = batch(a[2], e);
    const int32_t *table = int32s(a[3], e, "prefix_table"), *len = int32s(a[4], e, "prefix_len");
    const int64_t pages = THPVariable_Unpack(a[3]).size(0);
    if (THPVariable_Unpack(a[4]).numel() < 1 || pages > INT32_MAX) fail("%s: one entry", "prefix_len");
    const at::Tensor& q = tensor(a[5], "q");
    const int64_t qs = heads(q, e, e.n_q, b, "q");
    const float scale = a[6] == Py_None ? e.scale : (float)PyFloat_AsDouble(a[6]);
    if (PyErr_Occurred()) throw Error();
    float* lse = log_sums(a[8], e, b);
    int64_t os;
    const auto stream = stream_of(a[9], e);
    const at::Tensor out = output(a[7], q, e, b, &os, stream, a[9] == Py_None);
    return result(coli_attn_prefix(e.handle, kv, &b, table, (int)pages, len, q.data_ptr(), qs, scale, out.data_ptr(), os,
                                   lse, stream.stream()),
                  &out);
  });
}

PyMethodDef methods[] = {
    {"append", (PyCFunction)(void (*)())append, METH_FASTCALL, nullptr},
    {"window", (PyCFunction)(void (*)())window, METH_FASTCALL, nullptr},
    {"prefix", (PyCFunction)(void (*)())prefix, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_py", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_py() { return PyModule_Create(&module); }
