// Python module _layer_call: argument marshalling of the layer operators.
//
// The smallest of these calls take the GPU two microseconds; read in Python and passed through
// ctypes, a call's tensors took the host five (norm of 5 rows: 7.8 us a call so, 3.0 us here).  The module reads
// shapes, strides, types and devices of the tensors, makes their device current, takes its current stream unless one
// is given, and calls the library's C functions, whose addresses the package hands it (bind).
// Refusals become the package's DAError; every check of values is the library's own.
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdint.h>
#include <string>

#include "da.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refusal {
  da_status code;
  std::string what;
};

[[noreturn]] void refuse(da_status code, const std::string& what) { throw Refusal{code, what}; }

// A Python error is set; only the way out is left.
struct PythonError {};

PyObject* error_class = nullptr;   // DAError(code, where)
decltype(&da_rms_norm) call_rms_norm = nullptr;
decltype(&da_rms_norm_i8) call_rms_norm_i8 = nullptr;
decltype(&da_quantize_i8) call_quantize_i8 = nullptr;
decltype(&da_linear_i8) call_linear_i8 = nullptr;
decltype(&da_rope) call_rope = nullptr;

const Tensor* optional(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(DA_ERR_INVALID_ARG, std::string(what) + " has to be a tensor");
  const Tensor& t = THPVariable_Unpack(o);
  if (t.is_neg()) refuse(DA_ERR_INVALID_ARG, std::string(what) + " is negated lazily (resolve_neg() makes it a plain tensor)");
  return &t;
}

const Tensor& tensor(PyObject* o, const char* what) {
  const Tensor* t = optional(o, what);
  if (!t) refuse(DA_ERR_INVALID_ARG, std::string(what) + " has to be a tensor");
  return *t;
}

void* pointer(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

da_dtype element(const Tensor& t, const char* what) {
  if (t.scalar_type() == ScalarType::BFloat16) return DA_BF16;
  if (t.scalar_type() == ScalarType::Float) return DA_F32;
  refuse(DA_ERR_DTYPE, std::string(what) + " has to be bfloat16 or float32");
}

void type(const Tensor& t, ScalarType want, const char* what) {
  if (t.scalar_type() != want) refuse(DA_ERR_DTYPE, std::string(what) + " has to be " + c10::toString(want));
}

// The row stride of a [rows, width] tensor with contiguous rows; 0 for none.
int64_t row_stride(const Tensor* t, int64_t rows, int64_t width, ScalarType want, const char* what) {
  if (!t) return 0;
  if (t->dim() != 2 || t->size(0) != rows || t->size(1) != width)
    refuse(DA_ERR_SHAPE, std::string(what) + " has to be [" + std::to_string(rows) + ", " + std::to_string(width) + "]");
  type(*t, want, what);
  if (width > 1 && t->stride(1) != 1) refuse(DA_ERR_SHAPE, std::string(what) + " needs contiguous rows");
  return rows > 1 || t->stride(0) > width ? t->stride(0) : width;
}

void vector(const Tensor* t, int64_t n, ScalarType want, const char* what) {
  if (!t) return;
  if (t->dim() != 1 || t->size(0) != n) refuse(DA_ERR_SHAPE, std::string(what) + " has to be [" + std::to_string(n) + "]");
  type(*t, want, what);
  if (n > 1 && t->stride(0) != 1) refuse(DA_ERR_SHAPE, std::string(what) + " has to be contiguous");
}

da_head_strides head_strides(const Tensor& t, const char* what) {
  if (t.dim() != 4) refuse(DA_ERR_SHAPE, std::string(what) + " has to be [B, H, N, d]");
  if (t.size(3) > 1 && t.stride(3) != 1) refuse(DA_ERR_SHAPE, std::string(what) + " needs a contiguous last dimension");
  return da_head_strides{t.stride(0), t.stride(1), t.stride(2)};
}

// The sizes of the C calls are ints where no tensor that fits a GPU can reach beyond them.
int size32(int64_t n, const char* what) {
  if (n > INT32_MAX) refuse(DA_ERR_SHAPE, std::string(what) + " is too large");
  return (int)n;
}

// The one CUDA device that holds all the tensors.
template <typename... T>
int device_of(const Tensor* first, const T*... more) {
  const int device = first->is_cuda() ? (int)first->get_device() : -1;
  bool same = device >= 0;
  for (const Tensor* t : {first, more...}) same = same && (!t || (t->is_cuda() && t->get_device() == device));
  if (!same) refuse(DA_ERR_INVALID_ARG, "tensors have to be on one CUDA device");
  return device;
}

da_stream stream_of(PyObject* o, int device) {
  if (o == Py_None) return reinterpret_cast<da_stream>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
  PyObject* raw = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : Py_NewRef(o);
  void* p = raw ? PyLong_AsVoidPtr(raw) : nullptr;
  Py_XDECREF(raw);
  if (PyErr_Occurred()) throw PythonError{};
  return static_cast<da_stream>(p);
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return (float)v;
}

// Runs `call` with the device current and without the interpreter's lock, and raises what it returns.
template <typename F>
void run(int device, F call) {
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
  da_status st;
  Py_BEGIN_ALLOW_THREADS
  st = call();
  Py_END_ALLOW_THREADS
  if (st != DA_OK) refuse(st, "");
}

// f(arguments) with refusals as DAError and C++ errors as RuntimeError; None on success.
template <typename F>
PyObject* guarded(const char* where, Py_ssize_t have, Py_ssize_t want, F f) {
  if (have != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", where, want, have);
    return nullptr;
  }
  if (!error_class) {
    PyErr_SetString(PyExc_RuntimeError, "bind() first");
    return nullptr;
  }
  try {
    f();
    Py_RETURN_NONE;
  } catch (const Refusal& r) {
    const std::string text = r.what.empty() ? where : std::string(where) + ": " + r.what;
    if (PyObject* e = PyObject_CallFunction(error_class, "is", (int)r.code, text.c_str())) {
      PyErr_SetObject(error_class, e);
      Py_DECREF(e);
    }
  } catch (const PythonError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (x, weight, out, residual, sum_out, eps, stream)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("da_rms_norm", n, 7, [&] {
    const Tensor &x = tensor(a[0], "x"), &out = tensor(a[2], "out");
    const Tensor *w = optional(a[1], "weight"), *r = optional(a[3], "residual"), *sum = optional(a[4], "sum_out");
    const int device = device_of(&x, w, &out, r, sum);
    const da_dtype dtype = element(x, "x");
    if (x.dim() != 2) refuse(DA_ERR_SHAPE, "x has to be [rows, width]");
    const int64_t rows = x.size(0), width = x.size(1);
    const ScalarType t = x.scalar_type();
    vector(w, width, t, "weight");
    const int64_t xs = row_stride(&x, rows, width, t, "x"), rs = row_stride(r, rows, width, t, "residual");
    const int64_t ss = row_stride(sum, rows, width, t, "sum_out"), os = row_stride(&out, rows, width, t, "out");
    const int width32 = size32(width, "width");
    const float eps = number(a[5]);
    const da_stream s = stream_of(a[6], device);
    run(device, [&] {
      return call_rms_norm(rows, width32, dtype, x.data_ptr(), xs, pointer(r), rs, pointer(w), eps, pointer(sum), ss, out.data_ptr(), os, s);
    });
  });
}

// (x, weight, q, scale, residual, sum_out, eps, stream)
PyObject* rms_norm_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("da_rms_norm_i8", n, 8, [&] {
    const Tensor &x = tensor(a[0], "x"), &q = tensor(a[2], "q"), &scale = tensor(a[3], "scale");
    const Tensor *w = optional(a[1], "weight"), *r = optional(a[4], "residual"), *sum = optional(a[5], "sum_out");
    const int device = device_of(&x, w, &q, &scale, r, sum);
    const da_dtype dtype = element(x, "x");
    if (x.dim() != 2) refuse(DA_ERR_SHAPE, "x has to be [rows, width]");
    const int64_t rows = x.size(0), width = x.size(1);
    const ScalarType t = x.scalar_type();
    vector(w, width, t, "weight");
    vector(&scale, rows, ScalarType::Float, "scale");
    const int64_t xs = row_stride(&x, rows, width, t, "x"), rs = row_stride(r, rows, width, t, "residual");
    const int64_t ss = row_stride(sum, rows, width, t, "sum_out"), qs = row_stride(&q, rows, width, ScalarType::Char, "q");
    const int width32 = size32(width, "width");
    const float eps = number(a[6]);
    const da_stream s = stream_of(a[7], device);
    run(device, [&] {
      return call_rms_norm_i8(rows, width32, dtype, x.data_ptr(), xs, pointer(r), rs, pointer(w), eps, pointer(sum), ss,
                              static_cast<int8_t*>(q.data_ptr()), qs, static_cast<float*>(scale.data_ptr()), s);
    });
  });
}

// (x, q, scale, stream)
PyObject* quantize_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("da_quantize_i8", n, 4, [&] {
    const Tensor &x = tensor(a[0], "x"), &q = tensor(a[1], "q"), &scale = tensor(a[2], "scale");
    const int device = device_of(&x, &q, &scale);
    const da_dtype dtype = element(x, "x");
    int64_t B = 1, H = 1, N, d;
    da_head_strides xs{0, 0, 0};
    if (x.dim() == 2) {
      N = x.size(0);
      d = x.size(1);
      xs.token = row_stride(&x, N, d, x.scalar_type(), "x");
    } else {
      xs = head_strides(x, "x");
      B = x.size(0);
      H = x.size(1);
      N = x.size(2);
      d = x.size(3);
    }
    vector(&scale, B * N, ScalarType::Float, "scale");
    const int64_t qs = row_stride(&q, B * N, H * d, ScalarType::Char, "q");
    const int b = size32(B, "x"), h = size32(H, "x"), tokens = size32(N, "x"), dim = size32(d, "x");
    const da_stream s = stream_of(a[3], device);
    run(device, [&] {
      return call_quantize_i8(b, h, tokens, dim, dtype, x.data_ptr(), &xs, static_cast<int8_t*>(q.data_ptr()), qs,
                              static_cast<float*>(scale.data_ptr()), s);
    });
  });
}

// (x, x_scale, w, w_scale, out, ws, bias, stream)
PyObject* linear_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("da_linear_i8", n, 8, [&] {
    const Tensor &x = tensor(a[0], "x"), &sx = tensor(a[1], "x_scale"), &w = tensor(a[2], "w"), &sw = tensor(a[3], "w_scale");
    const Tensor &out = tensor(a[4], "out"), &ws = tensor(a[5], "ws");
    const Tensor* bias = optional(a[6], "bias");
    const int device = device_of(&x, &sx, &w, &sw, &out, &ws, bias);
    const da_dtype dtype = element(out, "out");
    if (x.dim() != 2 || w.dim() != 2) refuse(DA_ERR_SHAPE, "x and w have to be matrices");
    const int64_t M = x.size(0), K = x.size(1), C = w.size(0);
    int64_t B = 1, H = 1, N = M, d = C;
    da_head_strides os{0, 0, 0};
    if (out.dim() == 2) {
      os.token = row_stride(&out, M, C, out.scalar_type(), "out");
    } else {
      os = head_strides(out, "out");
      B = out.size(0);
      H = out.size(1);
      N = out.size(2);
      d = out.size(3);
      if (B * N != M || H * d != C)
        refuse(DA_ERR_SHAPE, "out has to hold " + std::to_string(M) + " tokens of " + std::to_string(C) + " channels");
    }
    vector(&sx, M, ScalarType::Float, "x_scale");
    vector(&sw, C, ScalarType::Float, "w_scale");
    vector(bias, C, ScalarType::Float, "bias");
    if (!ws.is_contiguous()) refuse(DA_ERR_SHAPE, "ws has to be contiguous");
    const int64_t xs = row_stride(&x, M, K, ScalarType::Char, "x"), wstr = row_stride(&w, C, K, ScalarType::Char, "w");
    const int b = size32(B, "out"), h = size32(H, "out"), tokens = size32(N, "out"), dim = size32(d, "out"), depth = size32(K, "x");
    const da_stream s = stream_of(a[7], device);
    run(device, [&] {
      return call_linear_i8(b, tokens, h, dim, depth, static_cast<const int8_t*>(x.data_ptr()), xs, static_cast<const float*>(sx.data_ptr()),
                            static_cast<const int8_t*>(w.data_ptr()), wstr, static_cast<const float*>(sw.data_ptr()),
                            static_cast<const float*>(pointer(bias)), dtype, out.data_ptr(), &os, ws.data_ptr(), ws.nbytes(), s);
    });
  });
}

// Three whole numbers of a rope's tuple.
void triple(PyObject* o, int (&to)[3], const char* what) {
  PyObject* seq = PySequence_Fast(o, "");
  if (!seq || PySequence_Fast_GET_SIZE(seq) != 3) {
    Py_XDECREF(seq);
    PyErr_Clear();
    refuse(DA_ERR_INVALID_ARG, std::string(what) + " has to be three whole numbers");
  }
  for (int i = 0; i < 3; ++i) {
    const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
    if (PyErr_Occurred() || v < INT32_MIN || v > INT32_MAX) {
      Py_DECREF(seq);
      PyErr_Clear();
      refuse(DA_ERR_INVALID_ARG, std::string(what) + " has to be three whole numbers");
    }
    to[i] = (int)v;
  }
  Py_DECREF(seq);
}

da_rope_plan plan_of(PyObject* o) {   // (axes, grid, theta, pairing)
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) refuse(DA_ERR_INVALID_ARG, "rope has to be a Rope");
  da_rope_plan p;
  triple(PyTuple_GET_ITEM(o, 0), p.axis_dims, "axes");
  triple(PyTuple_GET_ITEM(o, 1), p.grid, "grid");
  p.theta = PyFloat_AsDouble(PyTuple_GET_ITEM(o, 2));
  if (p.theta == -1.0 && PyErr_Occurred()) throw PythonError{};
  PyObject* pairing = PyTuple_GET_ITEM(o, 3);
  if (PyUnicode_Check(pairing) && PyUnicode_CompareWithASCIIString(pairing, "adjacent") == 0) p.pairing = DA_ROPE_ADJACENT;
  else if (PyUnicode_Check(pairing) && PyUnicode_CompareWithASCIIString(pairing, "halves") == 0) p.pairing = DA_ROPE_HALVES;
  else refuse(DA_ERR_INVALID_ARG, "pairing has to be 'adjacent' or 'halves'");
  return p;
}

// (x, out, rope, positions, weight, eps, stream)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("da_rope", n, 7, [&] {
    const da_rope_plan plan = plan_of(a[2]);
    const Tensor &x = tensor(a[0], "x"), &out = tensor(a[1], "out");
    const Tensor *pos = optional(a[3], "positions"), *w = optional(a[4], "weight");
    const int device = device_of(&x, &out, pos, w);
    const da_dtype dtype = element(x, "x");
    type(out, x.scalar_type(), "out");
    const da_head_strides xs = head_strides(x, "x"), os = head_strides(out, "out");
    if (out.sizes() != x.sizes()) refuse(DA_ERR_SHAPE, "out has to be of x's shape");
    const int64_t B = x.size(0), H = x.size(1), N = x.size(2), d = x.size(3);
    int64_t pos_batch = 0, width = 0;
    if (pos) {
      type(*pos, ScalarType::Int, "positions");
      const bool one = pos->dim() == 2 && pos->size(0) == N && pos->size(1) == 3;
      const bool each = pos->dim() == 3 && pos->size(0) == B && pos->size(1) == N && pos->size(2) == 3;
      if (!(one || each) || !pos->is_contiguous())
        refuse(DA_ERR_SHAPE, "positions have to be contiguous [N, 3] or [B, N, 3]");
      pos_batch = each ? 3 * N : 0;
    }
    if (w) {
      width = w->numel();
      vector(w, width, x.scalar_type(), "weight");
    }
    const int b = size32(B, "x"), h = size32(H, "x"), tokens = size32(N, "x"), dim = size32(d, "x"), weight_width = size32(width, "weight");
    const float eps = number(a[5]);
    const da_stream s = stream_of(a[6], device);
    run(device, [&] {
      return call_rope(&plan, b, h, tokens, dim, dtype, x.data_ptr(), &xs, static_cast<const int32_t*>(pointer(pos)), pos_batch, pointer(w),
                       weight_width, eps, out.data_ptr(), &os, s);
    });
  });
}

// bind(DAError, {name: address of the C function})
PyObject* bind(PyObject*, PyObject* args) {
  PyObject *error, *calls;
  if (!PyArg_ParseTuple(args, "OO!", &error, &PyDict_Type, &calls)) return nullptr;
  auto address = [&](const char* name) {
    PyObject* v = PyDict_GetItemString(calls, name);
    return v ? PyLong_AsVoidPtr(v) : nullptr;
  };
  call_rms_norm = reinterpret_cast<decltype(call_rms_norm)>(address("da_rms_norm"));
  call_rms_norm_i8 = reinterpret_cast<decltype(call_rms_norm_i8)>(address("da_rms_norm_i8"));
  call_quantize_i8 = reinterpret_cast<decltype(call_quantize_i8)>(address("da_quantize_i8"));
  call_linear_i8 = reinterpret_cast<decltype(call_linear_i8)>(address("da_linear_i8"));
  call_rope = reinterpret_cast<decltype(call_rope)>(address("da_rope"));
  if (PyErr_Occurred()) return nullptr;
  if (!call_rms_norm || !call_rms_norm_i8 || !call_quantize_i8 || !call_linear_i8 || !call_rope) {
    PyErr_SetString(PyExc_ValueError, "an address is missing");
    return nullptr;
  }
  Py_INCREF(error);
  Py_XDECREF(error_class);
  error_class = error;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"rms_norm", (PyCFunction)(void*)rms_norm, METH_FASTCALL, nullptr},
    {"rms_norm_i8", (PyCFunction)(void*)rms_norm_i8, METH_FASTCALL, nullptr},
    {"quantize_i8", (PyCFunction)(void*)quantize_i8, METH_FASTCALL, nullptr},
    {"linear_i8", (PyCFunction)(void*)linear_i8, METH_FASTCALL, nullptr},
    {"rope", (PyCFunction)(void*)rope, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_call() { return PyModule_Create(&module); }
