// The 8-bit calls (and, in paged_calls.h, the paged ones) from Python without the interpreter: each function checks
// the tensors, allocates the outputs that were not given and calls the C ABI on
// the current stream.  A decode step makes a handful of these calls with
// microseconds of GPU work each; through ctypes a call costs the host 9 to 14
// us, most of it attribute look-ups and the making of outputs; here 3.5 to 4.7,
// of which the launch is 2.
//
// Whatever is not plainly right (a shape, a type, a stride, a device that is
// not the current one, a refused size) gives None, and nothing has been
// launched: the package's general path then handles the call or says what is
// wrong with it.  An entry point that got as far as its launch and failed
// raises, so that no call is ever made twice.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/quarot.h"

namespace {

using at::ScalarType;
using at::Tensor;

// Addresses in the library that the package has loaded, set by bind().
decltype(&quarot_quant_fp8) g_quant = nullptr;
decltype(&quarot_quant_fp8_block) g_quant_block = nullptr;
decltype(&quarot_add_rmsnorm_quant_fp8) g_norm = nullptr;
decltype(&quarot_fp8_gemm) g_gemm = nullptr;
decltype(&quarot_fp8_gated_gemm) g_gated = nullptr;

constexpr ScalarType kCode = ScalarType::Float8_e4m3fn, kScale = ScalarType::Float;

int64_t blocks(int64_t n) { return (n + 127) / 128; }

// The device of a CUDA tensor, if it is the current one; or -1.
int device_of(PyObject* o) {
  if (!THPVariable_CheckExact(o)) return -1;
  const Tensor& t = THPVariable_Unpack(o);
  return t.defined() && t.is_cuda() && t.get_device() == c10::cuda::current_device() ? int(t.get_device()) : -1;
}

// The matrix behind a Python object: a dense CUDA tensor (exactly a tensor or
// parameter) of two dimensions on the current device; or null.
const Tensor* matrix(PyObject* o, int dev) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const Tensor& t = THPVariable_Unpack(o);
  return t.defined() && t.is_cuda() && t.get_device() == dev && t.dim() == 2 && t.layout() == at::kStrided &&
                 t.is_contiguous()
             ? &t
             : nullptr;
}
bool is(const Tensor* t, ScalarType type, int64_t rows, int64_t cols) {
  return t != nullptr && t->scalar_type() == type && t->size(0) == rows && t->size(1) == cols;
}
int dtype_of(const Tensor& t) {
  return t.scalar_type() == ScalarType::Half ? QUAROT_FP16 : t.scalar_type() == ScalarType::BFloat16 ? QUAROT_BF16 : -1;
}

// An output: the given tensor, if it is of this type and shape, or a new one.
bool output(PyObject* given, ScalarType type, int64_t rows, int64_t cols, int dev, Tensor& out) {
  if (given != Py_None) {
    const Tensor* t = matrix(given, dev);
    if (!is(t, type, rows, cols)) return false;
    out = *t;
  } else {
    out = at::detail::empty_cuda({rows, cols}, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)),
                                 std::nullopt);
  }
  return true;
}
PyObject* back(PyObject* given, const Tensor& out) {
  if (given == Py_None) return THPVariable_Wrap(out);
  Py_INCREF(given);
  return given;
}
PyObject* tuple_of(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New(Py_ssize_t(items.size()));
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (t != nullptr && o != nullptr) PyTuple_SET_ITEM(t, i++, o);
    else Py_XDECREF(o);
  }
  if (t != nullptr && i != Py_ssize_t(items.size())) Py_CLEAR(t);
  return t;
}
// What a status other than OK gives.  The first three are refusals, found
// before anything is launched: None.  The others raise the module's `error`.
PyObject* refused(PyObject* module, int status, const char* where) {
  if (status == QUAROT_ERR_INVALID_ARG || status == QUAROT_ERR_UNSUPPORTED || status == QUAROT_ERR_ALIGNMENT)
    Py_RETURN_NONE;
  PyObject* type = PyObject_GetAttrString(module, "error");
  if (type == nullptr) return nullptr;
  PyObject* e = PyObject_CallFunction(type, "is", status, where);
  if (e != nullptr) PyErr_SetObject(type, e);
  Py_XDECREF(e);
  Py_DECREF(type);
  return nullptr;
}
void* stream(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }
uint8_t* u8(const Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); }
float* f32(const Tensor& t) { return static_cast<float*>(t.data_ptr()); }

// quant(x, q_out, scale_out, weights)
PyObject* quant(PyObject* module, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4 || g_quant == nullptr) Py_RETURN_NONE;
  const int dev = device_of(args[0]);
  if (dev < 0) Py_RETURN_NONE;
  const Tensor* x = matrix(args[0], dev);
  if (x == nullptr || dtype_of(*x) < 0) Py_RETURN_NONE;
  const bool weights = args[3] == Py_True;
  const int64_t M = x->size(0), d = x->size(1);
  Tensor q, s;
  if (!output(args[1], kCode, M, d, dev, q) ||
      !output(args[2], kScale, weights ? blocks(M) : blocks(d), weights ? blocks(d) : M, dev, s))
    Py_RETURN_NONE;
  const int st = (weights ? g_quant_block : g_quant)(x->data_ptr(), dtype_of(*x), M, d, d, u8(q), f32(s), stream(dev));
  if (st != QUAROT_OK) return refused(module, st, weights ? "quarot_quant_fp8_block" : "quarot_quant_fp8");
  return tuple_of({back(args[1], q), back(args[2], s)});
  END_HANDLE_TH_ERRORS
}

// norm(x, residual, weight, eps, residual_out, q_out, scale_out)
PyObject* norm(PyObject* module, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7 || g_norm == nullptr || !PyFloat_CheckExact(args[3])) Py_RETURN_NONE;
  const int dev = device_of(args[0]);
  if (dev < 0) Py_RETURN_NONE;
  const Tensor* x = matrix(args[0], dev);
  if (x == nullptr || dtype_of(*x) < 0) Py_RETURN_NONE;
  const int64_t M = x->size(0), d = x->size(1);
  const Tensor* r = nullptr;
  if (args[1] != Py_None) {
    r = matrix(args[1], dev);
    if (!is(r, x->scalar_type(), M, d)) Py_RETURN_NONE;
  }
  const void* w = nullptr;
  if (args[2] != Py_None) {
    if (!THPVariable_CheckExact(args[2])) Py_RETURN_NONE;
    const Tensor& t = THPVariable_Unpack(args[2]);
    if (!t.defined() || !t.is_cuda() || t.get_device() != dev || t.dim() != 1 || t.size(0) != d ||
        t.layout() != at::kStrided || !t.is_contiguous() || t.scalar_type() != x->scalar_type())
      Py_RETURN_NONE;
    w = t.data_ptr();
  }
  Tensor h, q, s;
  const bool has_h = r != nullptr || args[4] != Py_None;
  if ((has_h && !output(args[4], x->scalar_type(), M, d, dev, h)) || !output(args[5], kCode, M, d, dev, q) ||
      !output(args[6], kScale, blocks(d), M, dev, s))
    Py_RETURN_NONE;
  const int st = g_norm(x->data_ptr(), d, r != nullptr ? r->data_ptr() : nullptr, d, w, dtype_of(*x), M, d,
                        float(PyFloat_AS_DOUBLE(args[3])), has_h ? h.data_ptr() : nullptr, d, u8(q), f32(s), stream(dev));
  if (st != QUAROT_OK) return refused(module, st, "quarot_add_rmsnorm_quant_fp8");
  return tuple_of({back(args[5], q), back(args[6], s), has_h ? back(args[4], h) : back(args[0], *x)});
  END_HANDLE_TH_ERRORS
}

// Token codes and their scales; weight codes of K columns and their scales.
bool tokens(const Tensor* a, const Tensor* as) {
  return a != nullptr && a->scalar_type() == kCode && is(as, kScale, blocks(a->size(1)), a->size(0));
}
bool weights(const Tensor* w, const Tensor* ws, int64_t K) {
  return w != nullptr && w->scalar_type() == kCode && w->size(1) == K && is(ws, kScale, blocks(w->size(0)), blocks(K));
}

// gemm(a_q, a_scale, w_q, w_scale, y, dtype): dtype is that of an output that is not given
PyObject* gemm(PyObject* module, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 6 || g_gemm == nullptr || !PyLong_CheckExact(args[5])) Py_RETURN_NONE;
  const int dev = device_of(args[0]);
  if (dev < 0) Py_RETURN_NONE;
  const Tensor *a = matrix(args[0], dev), *as = matrix(args[1], dev), *w = matrix(args[2], dev), *ws = matrix(args[3], dev);
  if (!tokens(a, as) || !weights(w, ws, a->size(1))) Py_RETURN_NONE;
  const int64_t M = a->size(0), N = w->size(0), K = a->size(1);
  long dt = PyLong_AsLong(args[5]);
  if (args[4] != Py_None) {
    const Tensor* y = matrix(args[4], dev);
    dt = y != nullptr ? dtype_of(*y) : -1;
  }
  if (dt != QUAROT_FP16 && dt != QUAROT_BF16) Py_RETURN_NONE;
  Tensor y;
  if (!output(args[4], dt == QUAROT_FP16 ? ScalarType::Half : ScalarType::BFloat16, M, N, dev, y)) Py_RETURN_NONE;
  const int st = g_gemm(u8(*a), f32(*as), u8(*w), f32(*ws), M, N, K, y.data_ptr(), int(dt), stream(dev));
  if (st != QUAROT_OK) return refused(module, st, "quarot_fp8_gemm");
  return back(args[4], y);
  END_HANDLE_TH_ERRORS
}

// gated(a_q, a_scale, wg_q, wg_scale, wu_q, wu_scale, q_out, scale_out)
PyObject* gated(PyObject* module, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8 || g_gated == nullptr) Py_RETURN_NONE;
  const int dev = device_of(args[0]);
  if (dev < 0) Py_RETURN_NONE;
  const Tensor* t[6];
  for (int i = 0; i < 6; ++i) t[i] = matrix(args[i], dev);
  if (!tokens(t[0], t[1])) Py_RETURN_NONE;
  const int64_t M = t[0]->size(0), K = t[0]->size(1);
  if (!weights(t[2], t[3], K) || !weights(t[4], t[5], K) || t[2]->size(0) != t[4]->size(0)) Py_RETURN_NONE;
  const int64_t I = t[2]->size(0);
  Tensor q, s;
  if (!output(args[6], kCode, M, I, dev, q) || !output(args[7], kScale, blocks(I), M, dev, s)) Py_RETURN_NONE;
  const int st = g_gated(u8(*t[0]), f32(*t[1]), u8(*t[2]), f32(*t[3]), u8(*t[4]), f32(*t[5]), M, I, K, u8(q), f32(s),
                         stream(dev));
  if (st != QUAROT_OK) return refused(module, st, "quarot_fp8_gated_gemm");
  return tuple_of({back(args[6], q), back(args[7], s)});
  END_HANDLE_TH_ERRORS
}

// bind(quant, quant_block, norm, gemm, gated): the entry points' addresses
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void* p[5];
  if (n != 5) return PyErr_Format(PyExc_TypeError, "bind takes five addresses");
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred() != nullptr) return nullptr;
  }
  g_quant = reinterpret_cast<decltype(g_quant)>(p[0]);
  g_quant_block = reinterpret_cast<decltype(g_quant_block)>(p[1]);
  g_norm = reinterpret_cast<decltype(g_norm)>(p[2]);
  g_gemm = reinterpret_cast<decltype(g_gemm)>(p[3]);
  g_gated = reinterpret_cast<decltype(g_gated)>(p[4]);
  Py_RETURN_NONE;
}

#include "paged_calls.h"

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef g_methods[] = {{"bind", FAST(bind)}, {"quant", FAST(quant)}, {"norm", FAST(norm)},
                           {"gemm", FAST(gemm)}, {"gated", FAST(gated)}, {"bind_paged", FAST(bind_paged)},
                           {"rope", FAST(rope)}, {"append", FAST(append)}, {"read", FAST(read)},
                           {"attn", FAST(attn)}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fp8_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8_calls() { return PyModule_Create(&g_module); }
