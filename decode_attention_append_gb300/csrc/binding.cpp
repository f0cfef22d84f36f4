// The Python side of the calls with rotation: tensors to pointers and strides.
//
// These calls take up to a dozen tensors, and their kernels a few microseconds: checked
// from Python, attribute by attribute, a call costs the host 9 to 13 us on a GB300
// machine's cores, and 3 to 4 here, most of it the launch.  Nothing is computed here;
// what a tensor has to be is checked and the C ABI called.  TypeError: not a tensor,
// another dtype, not on CUDA, not contiguous where it must be; ValueError: a shape or
// device that does not fit.  The calls return the library's status.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/daa.h"

namespace {

// What a call has found wrong is set as Python's error, and thrown as this.
struct Refused {};

[[noreturn]] void refuse(PyObject* kind, const char* format, const char* name, long long a = 0, long long b = 0) {
  PyErr_Format(kind, format, name, a, b);
  throw Refused{};
}

const at::Tensor& cuda_tensor(PyObject* o, const char* name, c10::ScalarType type) {
  const char* what = type == c10::kBFloat16 ? "%s must be a bf16 CUDA tensor"
                     : type == c10::kByte   ? "%s must be a uint8 CUDA tensor"
                                            : "%s must be an int32 CUDA tensor";
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, what, name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || t.scalar_type() != type || !t.is_cuda() || t.layout() != c10::kStrided)
    refuse(PyExc_TypeError, what, name);
  return t;
}

void on_device(const at::Tensor& t, const char* name, int dev) {
  if (t.get_device() != dev) refuse(PyExc_ValueError, "%s must be on cuda:%lld", name, dev);
}

// A contiguous tensor of `n` entries (any number with n < 0).
void* flat(PyObject* o, const char* name, c10::ScalarType type, int dev, int64_t n) {
  const at::Tensor& t = cuda_tensor(o, name, type);
  if (!t.is_contiguous()) refuse(PyExc_TypeError, "%s must be contiguous", name);
  on_device(t, name, dev);
  if (n >= 0 && (t.dim() != 1 || t.size(0) != n)) refuse(PyExc_ValueError, "%s must be [%lld]", name, n);
  return const_cast<void*>(t.unsafeGetTensorImpl()->data());
}

// bf16 rows [rows, heads, d] with d's values side by side; `written`: an output.
daa_rows heads_of(PyObject* o, const char* name, int dev, int64_t rows, int64_t d, bool written, int64_t& heads) {
  const at::Tensor& t = cuda_tensor(o, name, c10::kBFloat16);
  on_device(t, name, dev);
  if (t.dim() != 3 || t.size(0) != rows || t.size(2) != d)
    refuse(PyExc_ValueError, "%s must be [%lld, heads, %lld]", name, rows, d);
  if (t.stride(2) != 1) refuse(PyExc_ValueError, "%s's head_dim values must be side by side", name);
  heads = t.size(1);
  auto* impl = t.unsafeGetTensorImpl();
  return daa_rows{written ? impl->mutable_data() : const_cast<void*>(impl->data()), t.stride(0), t.stride(1)};
}

// cudaStream_t: the handle given, or the device's current stream.
void* stream_of(PyObject* o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev).stream();
  void* s = PyLong_AsVoidPtr(o);
  if (PyErr_Occurred()) throw Refused{};
  return s;
}

const daa_rope* rope_of(PyObject* o) {
  const void* p = PyLong_AsVoidPtr(o);
  if (!p) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "rope");
    throw Refused{};
  }
  return static_cast<const daa_rope*>(p);
}

float number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Refused{};
  return static_cast<float>(x);
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return;
  PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
  throw Refused{};
}

void same_heads(const char* name, int64_t heads, int64_t want, const char* as) {
  if (heads == want) return;
  PyErr_Format(PyExc_ValueError, "%s must have the heads of %s", name, as);
  throw Refused{};
}

// fn with the device current and the interpreter free for other threads.
template <class F>
PyObject* call(int dev, F&& fn) {
  daa_status st;
  {
    c10::cuda::OptionalCUDAGuard guard;
    if (c10::cuda::current_device() != dev) guard.set_index(dev);
    Py_BEGIN_ALLOW_THREADS;
    st = fn();
    Py_END_ALLOW_THREADS;
  }
  return PyLong_FromLong(st);
}

template <class F>
PyObject* guarded(F&& fn) {
  try {
    return fn();
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

int device_of(const at::Tensor& t) { return static_cast<int>(t.get_device()); }

// apply_rope(q, k, positions, rope, q_out, k_out, q_norm, k_norm, eps, stream)
PyObject* apply_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    count(n, 10);
    const at::Tensor& q = cuda_tensor(a[0], "q", c10::kBFloat16);
    const int dev = device_of(q);
    const daa_rope* rope = rope_of(a[3]);
    const int64_t rows = q.dim() == 3 ? q.size(0) : 0, d = rope->head_dim;
    int64_t hq, hk = 0, h;
    daa_rope_rows io{};
    io.q = heads_of(a[0], "q", dev, rows, d, false, hq);
    io.positions = static_cast<int32_t*>(flat(a[2], "positions", c10::kInt, dev, rows));
    io.q_out = heads_of(a[4], "q_out", dev, rows, d, true, h);
    same_heads("q_out", h, hq, "q");
    if (a[1] != Py_None) {
      io.k = heads_of(a[1], "k", dev, rows, d, false, hk);
      io.k_out = heads_of(a[5], "k_out", dev, rows, d, true, h);
      same_heads("k_out", h, hk, "k");
    } else if (a[5] != Py_None || a[7] != Py_None) {
      refuse(PyExc_ValueError, "k_out and k_norm go with %s", "k");
    }
    if (a[6] != Py_None) io.q_norm = flat(a[6], "q_norm", c10::kBFloat16, dev, d);
    if (a[7] != Py_None) io.k_norm = flat(a[7], "k_norm", c10::kBFloat16, dev, d);
    io.eps = number(a[8]);
    if (rows > INT32_MAX || hq > INT32_MAX || hk > INT32_MAX) refuse(PyExc_ValueError, "%s has too many rows or heads", "q");
    io.num_rows = static_cast<int32_t>(rows);
    void* s = stream_of(a[9], dev);
    return call(dev, [&] {
      return daa_apply_rope(rope, &io, static_cast<int32_t>(hq), static_cast<int32_t>(hk), s);
    });
  });
}

// append_rope(q, k_new, v_new, kv_pages, kv_exp, append_indptr, page_indices, kv_indptr, last_page_len, rope,
//             positions, q_out, q_norm, k_norm, eps, stream), and append_rope_q4 of the same
template <bool Q4>
PyObject* append_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    count(n, 16);
    const at::Tensor& pool = cuda_tensor(a[3], "kv_pages", Q4 ? c10::kByte : c10::kBFloat16);
    const int dev = device_of(pool);
    if (!pool.is_contiguous()) refuse(PyExc_TypeError, "%s must be contiguous", "kv_pages");
    daa_dims dims{};
    int64_t hkv;
    if (Q4) {
      if (pool.dim() != 4 || pool.size(2) != 2 || pool.size(3) % 9 != 0)
        refuse(PyExc_ValueError, "%s must be [num_pages, Hkv, 2, 9 * head_dim]", "kv_pages");
      hkv = pool.size(1);
      dims.head_dim = static_cast<int32_t>(pool.size(3) / 9);
      dims.page_size = 16;
    } else {
      if (pool.dim() != 5 || pool.size(1) != 2)
        refuse(PyExc_ValueError, "%s must be [num_pages, 2, Hkv, page_size, head_dim]", "kv_pages");
      hkv = pool.size(2);
      dims.head_dim = static_cast<int32_t>(pool.size(4));
      dims.page_size = static_cast<int32_t>(pool.size(3));
    }
    dims.num_pages = pool.size(0);
    const daa_rope* rope = rope_of(a[9]);
    const int64_t d = rope->head_dim;
    if (d != dims.head_dim) refuse(PyExc_ValueError, "%s is of another head_dim (%lld) than the pool", "rope", d);
    const at::Tensor& k = cuda_tensor(a[1], "k_new", c10::kBFloat16);
    const int64_t rows = k.dim() == 3 ? k.size(0) : 0;
    int64_t hq = hkv, h;
    daa_rope_rows io{};
    io.k = heads_of(a[1], "k_new", dev, rows, d, false, h);
    same_heads("k_new", h, hkv, "kv_pages");
    io.v = heads_of(a[2], "v_new", dev, rows, d, false, h);
    same_heads("v_new", h, hkv, "kv_pages");
    if (a[0] != Py_None) {
      io.q = heads_of(a[0], "q", dev, rows, d, false, hq);
      io.q_out = heads_of(a[11], "q_out", dev, rows, d, true, h);
      same_heads("q_out", h, hq, "q");
    } else if (a[11] != Py_None || a[12] != Py_None) {
      refuse(PyExc_ValueError, "q_out and q_norm go with %s", "q");
    }
    if (a[10] != Py_None) io.positions = static_cast<int32_t*>(flat(a[10], "positions", c10::kInt, dev, rows));
    if (a[12] != Py_None) io.q_norm = flat(a[12], "q_norm", c10::kBFloat16, dev, d);
    if (a[13] != Py_None) io.k_norm = flat(a[13], "k_norm", c10::kBFloat16, dev, d);
    io.eps = number(a[14]);
    const int64_t batch = cuda_tensor(a[5], "append_indptr", c10::kInt).numel() - 1;
    const int32_t* indptr = static_cast<int32_t*>(flat(a[5], "append_indptr", c10::kInt, dev, batch + 1));
    const int32_t* ids = static_cast<int32_t*>(flat(a[6], "page_indices", c10::kInt, dev, -1));
    const int32_t* kv_indptr = static_cast<int32_t*>(flat(a[7], "kv_indptr", c10::kInt, dev, batch + 1));
    const int32_t* last = static_cast<int32_t*>(flat(a[8], "last_page_len", c10::kInt, dev, batch < 0 ? 0 : batch));
    const int32_t* exps = nullptr;
    if (a[4] != Py_None) {
      exps = static_cast<int32_t*>(flat(a[4], "kv_exp", c10::kInt, dev, -1));
      const at::Tensor& e = THPVariable_Unpack(a[4]);
      if (e.dim() != 2 || e.size(0) != 2 || e.size(1) != hkv) refuse(PyExc_ValueError, "%s must be [2, Hkv]", "kv_exp");
    }
    if (rows > INT32_MAX || batch > INT32_MAX || hq > INT32_MAX || hkv > INT32_MAX)
      refuse(PyExc_ValueError, "%s has too many rows or heads, or append_indptr too many requests", "k_new");
    io.num_rows = static_cast<int32_t>(rows);
    dims.num_qo_heads = static_cast<int32_t>(hq);
    dims.num_kv_heads = static_cast<int32_t>(hkv);
    void* pages = pool.unsafeGetTensorImpl()->mutable_data();
    void* s = stream_of(a[15], dev);
    const int32_t requests = static_cast<int32_t>(batch);
    return call(dev, [&] {
      return Q4 ? daa_append_rope_q4(rope, &io, pages, exps, indptr, ids, kv_indptr, last, requests, dims, s)
                : daa_append_rope(rope, &io, pages, indptr, ids, kv_indptr, last, requests, dims, s);
    });
  });
}

template <class F>
PyCFunction method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef methods[] = {{"apply_rope", method(apply_rope), METH_FASTCALL, nullptr},
                         {"append_rope", method(append_rope<false>), METH_FASTCALL, nullptr},
                         {"append_rope_q4", method(append_rope<true>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
