// marshal.cpp -- the Python binding's calls of a decode step, whose kernels take a few microseconds:
// tensors become the C entry points' descriptors here, by their C++ accessors. Through ctypes the descriptors of
// one attention call took 10 us to fill, more than its kernel runs for a short sequence. Argument
// marshalling only, as in api.py, which wraps these functions: each returns the library's status.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>
#include <initializer_list>

#include "mxgemm.h"

namespace {

struct TypeError : std::exception {
  const char* text;
  explicit TypeError(const char* t) : text(t) {}
  const char* what() const noexcept override { return text; }
};
struct PythonError : std::exception {};  // already set
struct Refused : std::exception {  // with a status of the library
  int status;
  explicit Refused(int s) : status(s) {}
};

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw TypeError("a torch tensor was expected");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  return v;
}

int narrow(PyObject* o, int status) {  // a number that is no int is refused with this status
  int past = 0;
  const int64_t v = PyLong_AsLongLongAndOverflow(o, &past);
  if (v == -1 && !past && PyErr_Occurred()) throw PythonError();
  if (past || v < INT_MIN || v > INT_MAX) throw Refused(status);
  return (int)v;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return v;
}

template <typename T>
T* address(PyObject* o) {  // of a structure that the caller keeps; None: NULL
  return o == Py_None ? nullptr : reinterpret_cast<T*>((uintptr_t)integer(o));
}

bool is_int(int64_t n) { return n <= INT_MAX; }

// A [tokens][heads][dim] tensor, dim contiguous. False: another shape.
bool heads(const at::Tensor& t, mx_heads* h) {
  if (t.dim() != 3 || (t.stride(2) != 1 && t.size(2) > 1) || !is_int(t.size(0)) || !is_int(t.size(1)) || !is_int(t.size(2))) return false;
  *h = mx_heads{t.data_ptr(), (int)t.size(1), t.stride(0), t.stride(1)};
  return true;
}

// Whether the tensor's elements are format f's: of its size (a wrong one would be read past its end), and where they are
// floating ones, of its type. Whole numbers of that size stand for their bits.
bool fits(const at::Tensor& t, int f) {
  const at::ScalarType s = t.scalar_type();
  if (t.element_size() != (f == MX_F32 ? 4 : 2)) return false;
  return !at::isFloatingType(s) || s == (f == MX_F32 ? at::kFloat : f == MX_BF16 ? at::kBFloat16 : at::kHalf);
}

// The address of a dense int32 tensor of this shape; None: NULL.
bool ints(PyObject* o, at::IntArrayRef shape, const int32_t** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor& t = tensor(o);
  if (t.scalar_type() != at::kInt || t.sizes() != shape || !t.is_contiguous()) return false;
  *p = static_cast<const int32_t*>(t.data_ptr());
  return true;
}

bool table_of(PyObject* o, mxkv_table* table) {
  const at::Tensor& t = tensor(o);
  if (t.dim() != 2 || t.scalar_type() != at::kInt || !t.is_contiguous() || !is_int(t.size(0)) || !is_int(t.size(1))) return false;
  *table = mxkv_table{static_cast<const int32_t*>(t.data_ptr()), (int)t.size(0), (int)t.size(1)};
  return true;
}

// The last check before a call: every tensor that a kernel will read is one that the GPU can (None and addresses pass). `host`: whether
// one of a descriptor that the caller keeps is not.
void on_gpu(PyObject* host, std::initializer_list<PyObject*> tensors) {
  bool ok = host != Py_True;
  for (PyObject* o : tensors) {
    if (!THPVariable_Check(o)) continue;
    const at::Tensor& t = THPVariable_Unpack(o);
    ok = ok && (t.is_cuda() || t.numel() == 0 || t.is_pinned());
  }
  if (!ok) throw TypeError("a tensor on the GPU was expected");
}

void* stream_of(PyObject* o) {  // None: torch's current stream
  if (o != Py_None) return address<void>(o);
  static PyObject* current = nullptr;  // torch's own function of a device's current stream, kept for good
  if (!current) {
    PyObject* m = PyImport_ImportModule("torch._C");
    current = m ? PyObject_GetAttrString(m, "_cuda_getCurrentRawStream") : nullptr;
    Py_XDECREF(m);
    if (!current) throw PythonError();
  }
  const c10::impl::VirtualGuardImpl gpu(c10::DeviceType::CUDA);
  PyObject* device = PyLong_FromLong(gpu.getDevice().index());
  PyObject* handle = device ? PyObject_CallOneArg(current, device) : nullptr;
  Py_XDECREF(device);
  if (!handle) throw PythonError();
  void* stream = PyLong_AsVoidPtr(handle);
  Py_DECREF(handle);
  if (PyErr_Occurred()) throw PythonError();
  return stream;
}

template <typename F>
int unlocked(F call) {
  PyThreadState* state = PyEval_SaveThread();
  const int status = call();
  PyEval_RestoreThread(state);
  return status;
}

// (f, rope, x, out, positions, inverse, stream, host)
int rope(PyObject* const* a) {
  const at::Tensor &x = tensor(a[2]), &out = tensor(a[3]);
  mx_heads hx, ho;
  const int32_t* positions;
  if (!heads(x, &hx) || !heads(out, &ho) || x.sizes() != out.sizes() || !ints(a[4], x.sizes().slice(0, 1), &positions)) return MX_ERR_SHAPE;
  const int f = narrow(a[0], MX_ERR_FORMAT), tokens = (int)x.size(0), dim = (int)x.size(2), inverse = integer(a[5]) != 0;
  if (!fits(x, f) || !fits(out, f)) return MX_ERR_FORMAT;
  const mxrope* r = address<mxrope>(a[1]);
  on_gpu(a[7], {a[2], a[3], a[4]});
  void* stream = stream_of(a[6]);
  return unlocked([&] { return mxrope_run(f, r, tokens, dim, &hx, &ho, positions, inverse, stream); });
}

// (cache, f, k, v, positions, table, seq, rope, q, q_out, stream, host)
int append(PyObject* const* a) {
  const mxkv_cache* cache = address<mxkv_cache>(a[0]);
  mx_heads h[4];
  bool given[4];
  const int f = narrow(a[1], MX_ERR_FORMAT);
  const int64_t n = tensor(a[2]).dim() == 3 ? tensor(a[2]).size(0) : -1;
  const int place[4] = {2, 3, 8, 9};
  for (int i = 0; i < 4; i++) {
    given[i] = i < 2 || a[place[i]] != Py_None;
    if (!given[i]) continue;
    const at::Tensor& t = tensor(a[place[i]]);
    if (!heads(t, &h[i]) || t.size(0) != n || t.size(2) != cache->dim) return MX_ERR_SHAPE;
    if (!fits(t, f)) return MX_ERR_FORMAT;
  }
  const int32_t *positions, *seq;
  mxkv_table table;
  if (!table_of(a[5], &table) || !ints(a[4], {n}, &positions) || !ints(a[6], {n}, &seq)) return MX_ERR_SHAPE;
  const mxrope* r = address<mxrope>(a[7]);
  on_gpu(a[11], {a[2], a[3], a[4], a[5], a[6], a[8], a[9]});
  void* stream = stream_of(a[10]);
  return unlocked([&] {
    return mxkv_append_run(cache, f, (int)n, &h[0], &h[1], positions, seq, &table, r, given[2] ? &h[2] : nullptr, given[3] ? &h[3] : nullptr, stream);
  });
}

// (cache, f, q, out, table, lengths, max_len, scale, lse, starts, window, softcap, workspace, workspace_bytes, stream,
//  host)
int attention(PyObject* const* a) {
  const mxkv_cache* cache = address<mxkv_cache>(a[0]);
  const at::Tensor &q = tensor(a[2]), &out = tensor(a[3]);
  mx_heads hq, ho;
  mxkv_table table;
  if (!heads(q, &hq) || !heads(out, &ho) || q.sizes() != out.sizes() || q.size(2) != cache->dim) return MX_ERR_SHAPE;
  const int64_t n = q.size(0);
  const int32_t *lengths, *starts;
  if (!table_of(a[4], &table) || table.seqs != n || !ints(a[5], {n}, &lengths) || !ints(a[9], {n}, &starts)) return MX_ERR_SHAPE;
  float* lse = nullptr;
  if (a[8] != Py_None) {
    const at::Tensor& t = tensor(a[8]);
    if (t.sizes() != q.sizes().slice(0, 2) || !t.is_contiguous() || t.scalar_type() != at::kFloat) return MX_ERR_SHAPE;
    lse = static_cast<float*>(t.data_ptr());
  }
  void* workspace = nullptr;
  size_t bytes = 0;
  if (THPVariable_Check(a[12])) {
    const at::Tensor& t = tensor(a[12]);
    if (!t.is_contiguous()) return MX_ERR_SHAPE;
    workspace = t.data_ptr(), bytes = t.nbytes();
  } else {
    workspace = address<void>(a[12]);
  }
  if (a[13] != Py_None) {
    const int64_t given = integer(a[13]);
    if (given < 0 || (THPVariable_Check(a[12]) && (size_t)given > bytes)) return MX_ERR_SHAPE;
    bytes = (size_t)given;
  }
  const int f = narrow(a[1], MX_ERR_FORMAT), max_len = narrow(a[6], MX_ERR_SHAPE);
  if (!fits(q, f) || !fits(out, f)) return MX_ERR_FORMAT;
  const mxattn_opts opts = {(float)number(a[7]), (float)number(a[11]), narrow(a[10], MX_ERR_SHAPE)};
  on_gpu(a[15], {a[2], a[3], a[4], a[5], a[8], a[9], a[12]});
  void* stream = stream_of(a[14]);
  return unlocked([&] {
    return mxattn_decode_run(cache, f, &hq, &ho, lse, &table, lengths, starts, max_len, &opts, workspace, bytes, stream);
  });
}

// (layers, n_layers, pairs, stream, host)
int copy(PyObject* const* a) {
  const mxkv_cache* layers = address<mxkv_cache>(a[0]);
  const at::Tensor& t = tensor(a[2]);
  const int32_t* pairs;
  if (t.dim() != 2 || !is_int(t.size(0)) || !ints(a[2], {t.size(0), 2}, &pairs)) return MX_ERR_SHAPE;
  const int n_layers = narrow(a[1], MX_ERR_SHAPE), n = (int)t.size(0);
  on_gpu(a[4], {a[2]});
  void* stream = stream_of(a[3]);
  return unlocked([&] { return mxkv_copy_run(layers, n_layers, pairs, n, stream); });
}

template <int (*F)(PyObject* const*), int COUNT>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t count) {
  if (count != COUNT) {
    PyErr_Format(PyExc_TypeError, "%d arguments were expected", COUNT);
    return nullptr;
  }
  try {
    return PyLong_FromLong(F(args));
  } catch (const TypeError& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const Refused& e) {
    return PyLong_FromLong(e.status);
  } catch (const PythonError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <int (*F)(PyObject* const*), int COUNT>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, COUNT>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<rope, 8>("rope"), method<append, 12>("append"), method<attention, 16>("attention"), method<copy, 5>("copy"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__marshal() { return PyModule_Create(&module); }
