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

// A [rows][dim] tensor, dim contiguous. False: another shape.
bool matrix(const at::Tensor& t, mx_rows* m) {
  if (t.dim() != 2 || (t.stride(1) != 1 && t.size(1) > 1) || !is_int(t.size(0)) || !is_int(t.size(1))) return false;
  // a single row has no stride of its own: that of its whole 16-byte pieces
  const int64_t unit = 16 / t.element_size(), whole = (t.size(1) + unit - 1) / unit * unit;
  *m = mx_rows{t.data_ptr(), t.size(0) > 1 ? t.stride(0) : whole};
  return true;
}

// Whether a dense tensor of this type and shape stands here; None: NULL.
template <typename T>
bool dense(PyObject* o, at::IntArrayRef shape, at::ScalarType type, T** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor& t = tensor(o);
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous()) return false;
  *p = static_cast<T*>(t.data_ptr());
  return true;
}

// A workspace (tensor, address or None) and its size, None: the tensor's own. False: a size that the tensor does not have.
bool workspace_of(PyObject* o, PyObject* size, void** p, size_t* bytes) {
  *bytes = 0;
  if (THPVariable_Check(o)) {
    const at::Tensor& t = tensor(o);
    if (!t.is_contiguous()) return false;
    *p = t.data_ptr(), *bytes = t.nbytes();
  } else {
    *p = address<void>(o);
  }
  if (size == Py_None) return true;
  const int64_t given = integer(size);
  if (given < 0 || (THPVariable_Check(o) && (size_t)given > *bytes)) return false;
  *bytes = (size_t)given;
  return true;
}

// (cache, f, q, out, table, lengths, max_len, first, shared, max_shared, scale, lse, softcap, workspace, workspace_bytes, stream, host)
int prefix(PyObject* const* a) {
  const mxkv_cache* cache = address<mxkv_cache>(a[0]);
  const at::Tensor &q = tensor(a[2]), &out = tensor(a[3]), &first = tensor(a[7]), &shared = tensor(a[8]);
  mx_heads hq, ho;
  mxkv_table table;
  mxattn_groups groups;
  if (!heads(q, &hq) || !heads(out, &ho) || q.sizes() != out.sizes() || q.size(2) != cache->dim) return MX_ERR_SHAPE;
  const int64_t n = q.size(0);
  const int32_t* lengths;
  if (!table_of(a[4], &table) || table.seqs != n || !ints(a[5], {n}, &lengths)) return MX_ERR_SHAPE;
  if (shared.dim() != 1 || !is_int(shared.size(0)) || !ints(a[7], {shared.size(0) + 1}, &groups.first) || !ints(a[8], shared.sizes(), &groups.shared))
    return MX_ERR_SHAPE;
  groups.count = (int)shared.size(0), groups.max_shared = narrow(a[9], MX_ERR_SHAPE);
  float* lse;
  void* workspace;
  size_t bytes;
  if (!dense(a[11], q.sizes().slice(0, 2), at::kFloat, &lse) || !workspace_of(a[13], a[14], &workspace, &bytes)) return MX_ERR_SHAPE;
  const int f = narrow(a[1], MX_ERR_FORMAT), max_len = narrow(a[6], MX_ERR_SHAPE);
  if (!fits(q, f) || !fits(out, f)) return MX_ERR_FORMAT;
  const mxattn_opts opts = {(float)number(a[10]), (float)number(a[12]), 0};
  on_gpu(a[16], {a[2], a[3], a[4], a[5], a[7], a[8], a[11], a[13]});
  void* stream = stream_of(a[15]);
  return unlocked([&] {
    return mxattn_prefix_run(cache, f, &hq, &ho, lse, &table, lengths, &groups, max_len, &opts, workspace, bytes, stream);
  });
}

at::ScalarType type_of(int f) { return f == MX_F32 ? at::kFloat : f == MX_BF16 ? at::kBFloat16 : at::kHalf; }

// Bytes that stand for format f: of its type, or whole numbers of 8 bits.
bool holds(const at::Tensor& t, int f) {
  const at::ScalarType s = t.scalar_type();
  if (f == MX_F16 || f == MX_BF16 || f == MX_F32) return s == type_of(f);
  if (t.element_size() != 1 || s == at::kBool) return false;
  return !at::isFloatingType(s) || (f == MX_E4M3 && s == at::kFloat8_e4m3fn) || (f == MX_E5M2 && s == at::kFloat8_e5m2);
}

// The scales of rows in fmt, as norm and quantisation write them.
int scales_of(PyObject* o, int fmt, const at::Tensor& out, void** p) {
  *p = nullptr;
  if (o == Py_None) return MX_OK;
  const at::Tensor& t = tensor(o);
  const bool block = fmt == MX_E4M3 || fmt == MX_E5M2;
  if (!t.is_contiguous() || t.dim() != (block ? 2 : 1) || t.size(0) != out.size(0) || (block && t.size(1) != out.size(1) / 32)) return MX_ERR_SHAPE;
  if (block ? t.element_size() != 1 || (at::isFloatingType(t.scalar_type()) && t.scalar_type() != at::kFloat8_e8m0fnu) : t.scalar_type() != at::kFloat)
    return MX_ERR_FORMAT;
  *p = t.data_ptr();
  return MX_OK;
}

// (f, x, out, scales, fmt, weight, eps, residual, total, stream)
int norm(PyObject* const* a) {
  const int f = narrow(a[0], MX_ERR_FORMAT), fmt = narrow(a[4], MX_ERR_FORMAT);
  const at::Tensor &x = tensor(a[1]), &out = tensor(a[2]);
  mx_rows m[4];
  const int place[4] = {1, 2, 7, 8};
  for (int i = 0; i < 4; i++) {
    if (a[place[i]] == Py_None) continue;
    const at::Tensor& t = tensor(a[place[i]]);
    if (!matrix(t, &m[i]) || t.sizes() != x.sizes()) return MX_ERR_SHAPE;
    if (!holds(t, i == 1 ? fmt : f)) return MX_ERR_FORMAT;
  }
  void *scales, *weight = nullptr;
  if (int s = scales_of(a[3], fmt, out, &scales)) return s;
  if (a[5] != Py_None) {
    const at::Tensor& t = tensor(a[5]);
    if (!holds(t, f)) return MX_ERR_FORMAT;
    if (t.dim() != 1 || t.size(0) != x.size(1) || !t.is_contiguous()) return MX_ERR_SHAPE;
    weight = t.data_ptr();
  }
  const float eps = (float)number(a[6]);
  on_gpu(Py_False, {a[1], a[2], a[3], a[5], a[7], a[8]});
  void* stream = stream_of(a[9]);
  return unlocked([&] {
    return mxnorm_run(f, (int)x.size(0), (int)x.size(1), &m[0], a[7] == Py_None ? nullptr : &m[2], a[8] == Py_None ? nullptr : &m[3], weight, eps, fmt,
                      &m[1], scales, stream);
  });
}

// (f, x, out, scales, fmt, stream)
int quant(PyObject* const* a) {
  const int f = narrow(a[0], MX_ERR_FORMAT), fmt = narrow(a[4], MX_ERR_FORMAT);
  const at::Tensor &x = tensor(a[1]), &out = tensor(a[2]);
  mx_rows mx, mo;
  if (!matrix(x, &mx) || !matrix(out, &mo) || out.sizes() != x.sizes()) return MX_ERR_SHAPE;
  if (!holds(x, f) || !holds(out, fmt)) return MX_ERR_FORMAT;
  void* scales;
  if (int s = scales_of(a[3], fmt, out, &scales)) return s;
  on_gpu(Py_False, {a[1], a[2], a[3]});
  void* stream = stream_of(a[5]);
  return unlocked([&] { return mxquant_rows_run(f, (int)x.size(0), (int)x.size(1), &mx, fmt, &mo, scales, stream); });
}

// Whether every row's last 16-byte piece lies within the tensor's memory.
bool whole_pieces(const at::Tensor& t, const mx_rows& m) {
  if (t.numel() == 0) return true;
  const int64_t last = t.storage_offset() + (t.size(0) - 1) * m.stride + (t.size(1) + 15) / 16 * 16;
  return last <= (int64_t)t.storage().nbytes();
}

// (A, SA, B, SB, C, fc, bias, flags, workspace, workspace_bytes, stream)
int gemm_i8(PyObject* const* a) {
  const at::Tensor &A = tensor(a[0]), &B = tensor(a[2]), &C = tensor(a[4]);
  const int fc = narrow(a[5], MX_ERR_FORMAT);
  const int64_t flags = integer(a[7]);
  mx_rows ma, mb, mc;
  if (!matrix(A, &ma) || !matrix(B, &mb) || !matrix(C, &mc)) return MX_ERR_SHAPE;
  if (A.size(1) != B.size(1) || C.size(0) != A.size(0) || C.size(1) != B.size(0)) return MX_ERR_SHAPE;
  if (!holds(A, MX_INT8) || !holds(B, MX_INT8) || A.scalar_type() == at::kByte || B.scalar_type() == at::kByte) return MX_ERR_FORMAT;
  if ((fc != MX_F16 && fc != MX_BF16 && fc != MX_F32) || !holds(C, fc) || flags < 0 || flags > INT_MAX) return MX_ERR_FORMAT;
  if (!whole_pieces(A, ma) || !whole_pieces(B, mb)) return MX_ERR_SHAPE;
  float *sa, *sb;
  void *bias, *workspace;
  size_t bytes;
  if (!dense(a[1], A.sizes().slice(0, 1), at::kFloat, &sa) || !dense(a[3], B.sizes().slice(0, 1), at::kFloat, &sb)) return MX_ERR_SHAPE;
  if (a[6] != Py_None && !holds(tensor(a[6]), fc)) return MX_ERR_FORMAT;
  if (!dense(a[6], B.sizes().slice(0, 1), type_of(fc), &bias) || !workspace_of(a[8], a[9], &workspace, &bytes)) return MX_ERR_SHAPE;
  on_gpu(Py_False, {a[0], a[1], a[2], a[3], a[4], a[6], a[8]});
  void* stream = stream_of(a[10]);
  return unlocked([&] {
    return mxgemm_i8_run((int)A.size(0), (int)B.size(0), (int)A.size(1), &ma, sa, &mb, sb, bias, fc, &mc, (unsigned)flags, workspace, bytes, stream);
  });
}

// (page_size, table, lengths, wants, free, n_free, offsets, seq, positions, slots, status, kept, lengths_out, n_free_out, stream)
int step(PyObject* const* a) {
  mxkv_step s = {};
  const at::Tensor &table = tensor(a[1]), &free = tensor(a[4]);
  if (table.dim() != 2 || table.scalar_type() != at::kInt || !table.is_contiguous() || !is_int(table.size(0)) || !is_int(table.size(1))) return MX_ERR_SHAPE;
  if (free.dim() != 1 || !is_int(free.size(0))) return MX_ERR_SHAPE;
  const int64_t n = table.size(0), more = n + 1, one = 1;
  const int64_t room = a[7] == Py_None ? 0 : tensor(a[7]).numel();
  if (!is_int(room)) return MX_ERR_SHAPE;
  s.seqs = (int)n, s.cols = (int)table.size(1), s.page_size = narrow(a[0], MX_ERR_SHAPE), s.pages = (int)free.size(0), s.max_tokens = (int)room;
  s.table = static_cast<int32_t*>(table.data_ptr());
  int32_t *lengths, *wants, *kept, *n_free;
  if (!dense(a[2], {n}, at::kInt, &lengths) || !dense(a[3], {n}, at::kInt, &wants) || !dense(a[11], {n}, at::kInt, &kept) ||
      !dense(a[4], free.sizes(), at::kInt, &s.free_pages) || !dense(a[5], {one}, at::kInt, &n_free) || !dense(a[6], {more}, at::kInt, &s.offsets) ||
      !dense(a[7], {room}, at::kInt, &s.seq) || !dense(a[8], {room}, at::kInt, &s.positions) || !dense(a[9], {room}, at::kInt, &s.slots) ||
      !dense(a[10], {one}, at::kInt, &s.status) || !dense(a[12], {n}, at::kInt, &s.lengths_out) || !dense(a[13], {one}, at::kInt, &s.n_free_out))
    return MX_ERR_SHAPE;
  s.lengths = lengths, s.wants = wants, s.kept = kept, s.n_free = n_free;
  if (!s.lengths_out) s.lengths_out = lengths;
  if (!s.n_free_out) s.n_free_out = n_free;
  on_gpu(Py_False, {a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11], a[12], a[13]});
  void* stream = stream_of(a[14]);
  return unlocked([&] { return mxkv_step_run(&s, stream); });
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
                         method<norm, 10>("norm"), method<quant, 6>("quant"), method<gemm_i8, 11>("gemm_i8"), method<step, 15>("step"), method<prefix, 17>("prefix"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__marshal() { return PyModule_Create(&module); }
