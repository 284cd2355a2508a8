// The Python binding's common case in C++: a call's tensors are checked as the Python code checks
// them, and the C function is called: 3.1 us a call (kv_rotary, kv_quant_write and kv_quant_read of 64
// to 513 rows), 9.4 to 10.3 with the checks in Python and ctypes.  Anything out of the ordinary
// returns None, and the Python code, which has the error messages, does the call.
#include <torch/csrc/autograd/python_variable.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "kvevict.h"

namespace {

// Thrown where the Python code shall look at the call.
struct NotOrdinary {};

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw NotOrdinary();
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.layout() != at::kStrided) throw NotOrdinary();
  return t;
}

struct Call {
  int device;
  void* stream;

  explicit Call(PyObject* stream_arg) {
    device = c10::cuda::current_device();
    if (stream_arg == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    } else if (PyLong_Check(stream_arg)) {
      stream = PyLong_AsVoidPtr(stream_arg);
      if (PyErr_Occurred()) {
        PyErr_Clear();
        throw NotOrdinary();
      }
    } else {
      throw NotOrdinary();
    }
  }
  // A contiguous tensor of the type with at least `count` entries; None is null.
  void* buf(PyObject* o, at::ScalarType type, int64_t count) const {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    if (t.scalar_type() != type || t.get_device() != device || t.numel() < count ||
        !t.is_contiguous())
      throw NotOrdinary();
    return t.data_ptr();
  }
  // Rows of `row` elements, each contiguous: their number and the stride between them.
  void* rows(PyObject* o, at::ScalarType type, int64_t row, int64_t* n, int64_t* stride) const {
    const at::Tensor& t = tensor(o);
    if (t.scalar_type() != type || t.get_device() != device || t.dim() < 2) throw NotOrdinary();
    *n = t.size(0);
    if (t.numel() != *n * row) throw NotOrdinary();
    int64_t step = 1;
    for (int64_t k = t.dim() - 1; k > 0; --k) {
      if (t.size(k) > 1 && t.stride(k) != step) throw NotOrdinary();
      step *= t.size(k);
    }
    *stride = *n > 1 ? t.stride(0) : row;
    if (*stride < row) throw NotOrdinary();
    return t.data_ptr();
  }
  // A page pool of codes: pages of `inner` bytes, dense, `apart` bytes apart.
  void* pool(PyObject* o, int format, int64_t inner, int64_t pages, int64_t apart) const {
    const at::Tensor& t = tensor(o);
    const at::ScalarType type = t.scalar_type();
    if (format == KV_E4M3 ? type != at::kFloat8_e4m3fn && type != at::kByte : type != at::kChar)
      throw NotOrdinary();
    if (t.get_device() != device || t.dim() < 1) throw NotOrdinary();
    const int64_t n = t.size(0);
    if (n < pages || t.numel() != n * inner) throw NotOrdinary();
    int64_t step = 1;
    for (int64_t k = t.dim() - 1; k > 0; --k) {
      if (t.size(k) > 1 && t.stride(k) != step) throw NotOrdinary();
      step *= t.size(k);
    }
    if (pages > 1 && t.stride(0) != apart) throw NotOrdinary();
    return t.data_ptr();
  }
  void* work(PyObject* o, size_t* bytes) const {
    const at::Tensor& t = tensor(o);
    if (t.get_device() != device || !t.is_contiguous()) throw NotOrdinary();
    *bytes = t.nbytes();
    return t.data_ptr();
  }
};

at::ScalarType row_type(int dtype) {
  if (dtype == KV_BF16) return at::kBFloat16;
  if (dtype == KV_F32) return at::kFloat;
  throw NotOrdinary();
}
int number(PyObject* o) {
  const long v = PyLong_Check(o) ? PyLong_AsLong(o) : -1;
  if (v < 0 || v > 1 << 20) {
    PyErr_Clear();
    throw NotOrdinary();
  }
  return (int)v;
}
// The bytes of a ctypes structure.
template <typename S>
S structure(PyObject* o) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    throw NotOrdinary();
  }
  S s;
  const bool ok = b.len == (Py_ssize_t)sizeof(S);
  if (ok) memcpy(&s, b.buf, sizeof(S));
  PyBuffer_Release(&b);
  if (!ok) throw NotOrdinary();
  return s;
}
struct Quant {
  kv_paged_shape s;
  int format;
  int64_t heads, row, inner, apart, blocks;
  Quant(PyObject* shape, PyObject* fmt) : s(structure<kv_paged_shape>(shape)), format(number(fmt)) {
    // (what the C function refuses is its own to refuse; nothing may divide by zero or overflow here)
    if (s.tables <= 0 || s.hkv <= 0 || s.hkv > 256 || s.hq <= 0 || s.hq > 1 << 16 || s.d <= 0 ||
        s.d > 256 || s.page <= 0 || s.page > 256 || s.num_pages <= 0 || s.num_pages > INT32_MAX ||
        s.seqs < 0 || s.max_pages <= 0)
      throw NotOrdinary();
    heads = s.hkv / s.tables;
    row = heads * s.d;
    inner = row * s.page;
    apart = s.page_stride != 0 ? s.page_stride : inner;
    blocks = s.num_pages * heads * (s.page / KV_QUANT_BLOCK);
  }
};

decltype(&kv_quant_write) quant_write_fn;
decltype(&kv_quant_read) quant_read_fn;
decltype(&quant_decode_attn) quant_decode_fn;
decltype(&kv_rotary) rotary_fn;

template <typename F>
PyObject* ordinary(F call) {
  int status;
  try {
    status = call();
  } catch (...) {
    Py_RETURN_NONE;
  }
  return PyLong_FromLong(status);
}

// shape, format, k, v, slot_map, n_rows, k_pages, v_pages, k_scale, v_scale, ws, stream
PyObject* write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary([&]() -> int {
    if (n != 12) throw NotOrdinary();
    const Quant q(a[0], a[1]);
    const Call c(a[11]);
    const at::ScalarType type = row_type(q.s.dtype);
    int64_t rows, stride, rows_v, stride_v;
    void* k = c.rows(a[2], type, q.row, &rows, &stride);
    void* v = c.rows(a[3], type, q.row, &rows_v, &stride_v);
    if (rows != rows_v || stride != stride_v) throw NotOrdinary();
    size_t bytes;
    void* ws = c.work(a[10], &bytes);
    return quant_write_fn(&q.s, q.format, k, v, stride, (int64_t*)c.buf(a[4], at::kLong, rows),
                          rows, (int64_t*)c.buf(a[5], at::kLong, 1),
                          c.pool(a[6], q.format, q.inner, q.s.num_pages, q.apart),
                          c.pool(a[7], q.format, q.inner, q.s.num_pages, q.apart),
                          (float*)c.buf(a[8], at::kFloat, q.blocks),
                          (float*)c.buf(a[9], at::kFloat, q.blocks), ws, bytes, c.stream);
  });
}
// shape, format, k_pages, v_pages, k_scale, v_scale, slot_map, n_rows, k, v, ws, stream
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary([&]() -> int {
    if (n != 12) throw NotOrdinary();
    const Quant q(a[0], a[1]);
    const Call c(a[11]);
    const at::ScalarType type = row_type(q.s.dtype);
    int64_t rows, stride, rows_v, stride_v;
    void* k = c.rows(a[8], type, q.row, &rows, &stride);
    void* v = c.rows(a[9], type, q.row, &rows_v, &stride_v);
    if (rows != rows_v || stride != stride_v) throw NotOrdinary();
    size_t bytes;
    void* ws = c.work(a[10], &bytes);
    return quant_read_fn(&q.s, q.format, c.pool(a[2], q.format, q.inner, q.s.num_pages, q.apart),
                         c.pool(a[3], q.format, q.inner, q.s.num_pages, q.apart),
                         (float*)c.buf(a[4], at::kFloat, q.blocks),
                         (float*)c.buf(a[5], at::kFloat, q.blocks),
                         (int64_t*)c.buf(a[6], at::kLong, rows), rows,
                         (int64_t*)c.buf(a[7], at::kLong, 1), k, v, stride, ws, bytes, c.stream);
  });
}
// shape, format, q, k_new, v_new, cu_add, slot_map, k_pages, v_pages, k_scale, v_scale,
// block_table, lens, softmax_scale, out, ws, stream
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary([&]() -> int {
    if (n != 17) throw NotOrdinary();
    const Quant q(a[0], a[1]);
    const Call c(a[16]);
    const at::ScalarType type = row_type(q.s.dtype);
    const int64_t tables = (int64_t)q.s.seqs * q.s.tables, d = q.s.d;
    const int64_t nq = (int64_t)q.s.seqs * q.s.hq * d, nk = (int64_t)q.s.seqs * q.s.hkv * d;
    if (!PyFloat_Check(a[13])) throw NotOrdinary();
    const int64_t slots = a[6] == Py_None ? 0 : tensor(a[6]).numel();
    size_t bytes;
    void* ws = c.work(a[15], &bytes);
    return quant_decode_fn(&q.s, q.format, c.buf(a[2], type, nq), c.buf(a[3], type, nk),
                           c.buf(a[4], type, nk), (int64_t*)c.buf(a[5], at::kLong, tables + 1),
                           (int64_t*)c.buf(a[6], at::kLong, 0), slots,
                           c.pool(a[7], q.format, q.inner, q.s.num_pages, q.apart),
                           c.pool(a[8], q.format, q.inner, q.s.num_pages, q.apart),
                           (float*)c.buf(a[9], at::kFloat, q.blocks),
                           (float*)c.buf(a[10], at::kFloat, q.blocks),
                           (int32_t*)c.buf(a[11], at::kInt, tables * q.s.max_pages),
                           (int32_t*)c.buf(a[12], at::kInt, tables),
                           (float)PyFloat_AS_DOUBLE(a[13]), c.buf(a[14], type, nq), ws, bytes,
                           c.stream);
  });
}
// shape, q, k, positions, inv_freq, q_out, k_out, n_rows, back, stream
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return ordinary([&]() -> int {
    if (n != 10) throw NotOrdinary();
    const kv_rotary_shape s = structure<kv_rotary_shape>(a[0]);
    const Call c(a[9]);
    const at::ScalarType type = row_type(s.dtype);
    if (s.hq < 0 || s.hkv < 0 || s.hq > 4096 || s.hkv > 4096 || s.d <= 0 || s.d > 256 || s.rot <= 0)
      throw NotOrdinary();
    int64_t rows = -1;
    void* p[4] = {};
    int64_t stride[4] = {};
    const int heads[4] = {s.hq, s.hkv, s.hq, s.hkv};
    PyObject* const side[4] = {a[1], a[2], a[5], a[6]};
    for (int i = 0; i < 4; ++i) {
      if (heads[i] == 0) continue;
      int64_t m;
      p[i] = c.rows(side[i], type, (int64_t)heads[i] * s.d, &m, &stride[i]);
      if (rows >= 0 && m != rows) throw NotOrdinary();
      rows = m;
    }
    if (rows < 0 || !PyBool_Check(a[8])) throw NotOrdinary();
    return rotary_fn(&s, a[8] == Py_True, p[0], stride[0], p[1], stride[1],
                     (int32_t*)c.buf(a[3], at::kInt, rows),
                     (double*)c.buf(a[4], at::kDouble, s.rot / 2), rows,
                     (int64_t*)c.buf(a[7], at::kLong, 1), p[2], stride[2], p[3], stride[3],
                     c.stream);
  });
}

// The library's functions, as addresses: write, read, decode, rotary.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* f[4];
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "four addresses are needed");
    return nullptr;
  }
  for (int i = 0; i < 4; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  quant_write_fn = reinterpret_cast<decltype(quant_write_fn)>(f[0]);
  quant_read_fn = reinterpret_cast<decltype(quant_read_fn)>(f[1]);
  quant_decode_fn = reinterpret_cast<decltype(quant_decode_fn)>(f[2]);
  rotary_fn = reinterpret_cast<decltype(rotary_fn)>(f[3]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL,
          nullptr};
}
PyMethodDef methods[] = {method<write>("kv_quant_write"), method<read>("kv_quant_read"),
                         method<decode>("quant_decode_attn"), method<rotary>("kv_rotary"),
                         method<bind>("bind"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods,
                          nullptr, nullptr, nullptr, nullptr};
}  // namespace

PyMODINIT_FUNC PyInit__fast() { return PyModule_Create(&module_def); }
