// Python entry for the calls whose kernels are as short as their launch
// (rmsnorm_quantize, qgemv_*, qgemm_mx_grouped): checks the ordinary case,
// allocates the outputs and calls the C ABI on the current stream, in about
// half the host time of the same steps in Python (norm of one row 11.6 -> 5.4
// us a call with its launch, which alone takes 4).
//
// Every function returns None, with nothing launched, where anything is not
// the ordinary case (another device than the current one, a strided or
// subclassed tensor, a wrong type or shape, a size the library refuses): the
// Python path in ops.py then does the call or raises its error.  Any other
// failure is answered with the library's status as an int, which the caller
// raises: that call is not made again.
#include <Python.h>

#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/vdtq.h"

namespace {

using at::ScalarType;

// Activation kinds of gemv, as the Python caller numbers them.
enum { kBf16 = 0, kInt8 = 1, kMx8 = 2, kMx4 = 3 };

bool is_none(PyObject* o) { return o == Py_None; }

// A plain tensor on device `dev`, dense, of type t and the given sizes.
const at::Tensor* dense(PyObject* o, int dev, ScalarType t, at::IntArrayRef sizes) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& x = THPVariable_Unpack(o);
  if (!x.defined() || !x.is_cuda() || x.get_device() != dev || x.scalar_type() != t || x.sizes() != sizes ||
      !x.is_contiguous())
    return nullptr;
  return &x;
}

// A 2-D plain tensor's sizes and device, if that is the current one.
bool shape2(PyObject* o, int64_t& rows, int64_t& cols, int& dev) {
  if (!THPVariable_CheckExact(o)) return false;
  const at::Tensor& x = THPVariable_Unpack(o);
  if (!x.defined() || !x.is_cuda() || x.dim() != 2) return false;
  rows = x.size(0);
  cols = x.size(1);
  dev = (int)x.get_device();
  return dev == c10::hip::current_device();
}

at::TensorBase make(at::IntArrayRef sizes, ScalarType t, int dev) {
  return at::detail::empty_cuda(sizes, t, c10::Device(c10::DeviceType::CUDA, (c10::DeviceIndex)dev), std::nullopt);
}

void* stream(int dev) { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream(); }

// "bf16" / "f32" -> the library's code, -1 otherwise
int out_code(PyObject* o) {
  if (!PyUnicode_Check(o)) return -1;
  if (PyUnicode_CompareWithASCIIString(o, "bf16") == 0) return VDTQ_OUT_BF16;
  return PyUnicode_CompareWithASCIIString(o, "f32") == 0 ? VDTQ_OUT_F32 : -1;
}

// The caller's y or a new one; false where a given y is not the ordinary one.
bool output(PyObject* y, int64_t M, int64_t N, int out, int dev, at::TensorBase& t) {
  const ScalarType st = out == VDTQ_OUT_F32 ? ScalarType::Float : ScalarType::BFloat16;
  if (is_none(y)) {
    t = make({M, N}, st, dev);
    return true;
  }
  const at::Tensor* g = dense(y, dev, st, {M, N});
  if (!g) return false;
  t = *g;
  return true;
}

// What the Python caller makes of a status other than VDTQ_OK: a refusal
// launches nothing, and the Python path names it.
PyObject* failed(int rc) {
  if (rc == VDTQ_EINVAL || rc == VDTQ_EUNSUPPORTED) Py_RETURN_NONE;
  return PyLong_FromLong(rc);
}

PyObject* give(PyObject* y, at::TensorBase&& t) {
  if (is_none(y)) return THPVariable_Wrap(std::move(t));
  Py_INCREF(y);
  return y;
}

const void* ptr(const at::Tensor* t) { return t ? t->const_data_ptr() : nullptr; }

// gemv(kind, a_q, a_s, w_q, w_s, w_ts, bias, y, out_dtype)
PyObject* gemv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) return PyErr_Format(PyExc_TypeError, "gemv takes 9 arguments");
  const long kind = PyLong_AsLong(a[0]);
  if (kind == -1 && PyErr_Occurred()) return nullptr;
  int64_t M, K, N, w2;
  int dev, wdev;
  const int out = out_code(a[8]);
  if (out < 0 || kind < kBf16 || kind > kMx4 || !shape2(a[1], M, K, dev) || !shape2(a[3], N, w2, wdev)) Py_RETURN_NONE;
  const int64_t width = K;
  if (kind == kMx4) K *= 2;
  const bool mx = kind >= kMx8;
  const ScalarType at = kind == kBf16 ? ScalarType::BFloat16 : kind == kInt8 ? ScalarType::Char : ScalarType::Byte;
  const at::Tensor* aq = dense(a[1], dev, at, {M, width});
  const at::Tensor* wq = dense(a[3], dev, ScalarType::Byte, {N, K / 2});
  const at::Tensor* ws = dense(a[4], dev, ScalarType::Byte, {N, K / (mx ? 32 : 16)});
  if (!aq || !wq || !ws || K % (mx ? 32 : 16)) Py_RETURN_NONE;
  const at::Tensor *as = nullptr, *ts = nullptr, *bias = nullptr;
  if (kind == kInt8 && !(as = dense(a[2], dev, ScalarType::Float, {M}))) Py_RETURN_NONE;
  if (mx && !(as = dense(a[2], dev, ScalarType::Byte, {M, K / 32}))) Py_RETURN_NONE;
  if (!mx && !(ts = dense(a[5], dev, ScalarType::Float, {2}))) Py_RETURN_NONE;
  if (!is_none(a[6]) && !(bias = dense(a[6], dev, ScalarType::Float, {N}))) Py_RETURN_NONE;
  if (M > VDTQ_GEMV_MAX_ROWS) Py_RETURN_NONE;
  at::TensorBase y;
  if (!output(a[7], M, N, out, dev, y)) Py_RETURN_NONE;
  const auto wqp = static_cast<const uint8_t*>(ptr(wq)), wsp = static_cast<const uint8_t*>(ptr(ws));
  const auto tsp = static_cast<const float*>(ptr(ts)), bp = static_cast<const float*>(ptr(bias));
  void* const yp = y.mutable_data_ptr();
  int rc;
  if (kind == kBf16)
    rc = qgemv_w4a16(ptr(aq), wqp, wsp, tsp, bp, yp, N, out, M, N, K, stream(dev));
  else if (kind == kInt8)
    rc = qgemv_w4a8(static_cast<const int8_t*>(ptr(aq)), static_cast<const float*>(ptr(as)), wqp, wsp, tsp, bp, yp, N,
                    out, M, N, K, stream(dev));
  else
    rc = qgemv_mx(kind == kMx8 ? VDTQ_FMT_MXFP8 : VDTQ_FMT_MXFP4, static_cast<const uint8_t*>(ptr(aq)),
                  static_cast<const uint8_t*>(ptr(as)), wqp, wsp, bp, yp, N, out, M, N, K, stream(dev));
  if (rc != VDTQ_OK) return failed(rc);
  return give(a[7], std::move(y));
  END_HANDLE_TH_ERRORS
}

// grouped(a8, a_q, a_s, w_q, w_s, offsets, bias, y, out_dtype)
PyObject* grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) return PyErr_Format(PyExc_TypeError, "grouped takes 9 arguments");
  const bool a8 = a[0] == Py_True;
  int64_t T, K, rows, w2;
  int dev, wdev;
  const int out = out_code(a[8]);
  if (out < 0 || !shape2(a[1], T, K, dev) || !shape2(a[3], rows, w2, wdev) || !THPVariable_CheckExact(a[5])) Py_RETURN_NONE;
  const int64_t width = K;
  if (!a8) K *= 2;
  const int64_t E = THPVariable_Unpack(a[5]).numel() - 1;
  if (E < 1 || rows % E || K % 32) Py_RETURN_NONE;
  const int64_t N = rows / E;
  const at::Tensor* aq = dense(a[1], dev, ScalarType::Byte, {T, width});
  const at::Tensor* as = dense(a[2], dev, ScalarType::Byte, {T, K / 32});
  const at::Tensor* wq = dense(a[3], dev, ScalarType::Byte, {rows, K / 2});
  const at::Tensor* ws = dense(a[4], dev, ScalarType::Byte, {rows, K / 32});
  const at::Tensor* off = dense(a[5], dev, ScalarType::Int, {E + 1});
  const at::Tensor* bias = nullptr;
  if (!aq || !as || !wq || !ws || !off) Py_RETURN_NONE;
  if (!is_none(a[6]) && !(bias = dense(a[6], dev, ScalarType::Float, {E, N}))) Py_RETURN_NONE;
  at::TensorBase y;
  if (!output(a[7], T, N, out, dev, y)) Py_RETURN_NONE;
  const int rc = qgemm_mx_grouped(
      a8 ? VDTQ_FMT_MXFP8 : VDTQ_FMT_MXFP4, static_cast<const uint8_t*>(ptr(aq)), static_cast<const uint8_t*>(ptr(as)),
      static_cast<const uint8_t*>(ptr(wq)), static_cast<const uint8_t*>(ptr(ws)), static_cast<const float*>(ptr(bias)),
      static_cast<const int32_t*>(ptr(off)), E, y.mutable_data_ptr(), N, out, T, N, K, stream(dev));
  if (rc != VDTQ_OK) return failed(rc);
  return give(a[7], std::move(y));
  END_HANDLE_TH_ERRORS
}

// norm(x, weight, residual, eps, had_block, fmt, sum_out): the library's fmt
// code; returns (q, scales or None, sum or None)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7) return PyErr_Format(PyExc_TypeError, "norm takes 7 arguments");
  const double eps = PyFloat_AsDouble(a[3]);
  const long b = PyLong_AsLong(a[4]), fmt = PyLong_AsLong(a[5]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  if (b != (int)b) Py_RETURN_NONE;
  int64_t M, K;
  int dev;
  if (!shape2(a[0], M, K, dev)) Py_RETURN_NONE;
  const bool mx = fmt == VDTQ_FMT_MXFP4 || fmt == VDTQ_FMT_MXFP8;
  if ((!mx && fmt != VDTQ_FMT_INT8 && fmt != VDTQ_FMT_BF16) || K < 1 || K % (mx ? 32 : 16) || K > 16384) Py_RETURN_NONE;
  const at::Tensor* x = dense(a[0], dev, ScalarType::BFloat16, {M, K});
  const at::Tensor *w = nullptr, *res = nullptr;
  if (!x || (!is_none(a[1]) && !(w = dense(a[1], dev, ScalarType::Float, {K})))) Py_RETURN_NONE;
  if (!is_none(a[2]) && !(res = dense(a[2], dev, ScalarType::BFloat16, {M, K}))) Py_RETURN_NONE;
  at::TensorBase q, scales, sum;
  if (res) {
    if (!output(a[6], M, K, VDTQ_OUT_BF16, dev, sum)) Py_RETURN_NONE;
  } else if (!is_none(a[6])) {
    Py_RETURN_NONE;
  }
  if (fmt == VDTQ_FMT_BF16) {
    q = make({M, K}, ScalarType::BFloat16, dev);
  } else if (fmt == VDTQ_FMT_INT8) {
    q = make({M, K}, ScalarType::Char, dev);
    scales = make({M}, ScalarType::Float, dev);
  } else {
    q = make({M, fmt == VDTQ_FMT_MXFP4 ? K / 2 : K}, ScalarType::Byte, dev);
    scales = make({M, K / 32}, ScalarType::Byte, dev);
  }
  const int rc = rmsnorm_quantize(ptr(x), M, K, K, ptr(res), K, static_cast<const float*>(ptr(w)), (float)eps, (int)b,
                                  (int)fmt, res ? sum.mutable_data_ptr() : nullptr, K, q.mutable_data_ptr(),
                                  scales.defined() ? scales.mutable_data_ptr() : nullptr, stream(dev));
  if (rc != VDTQ_OK) return failed(rc);
  PyObject* pq = THPVariable_Wrap(std::move(q));
  PyObject* ps = Py_None;
  PyObject* pr = Py_None;
  if (scales.defined()) ps = THPVariable_Wrap(std::move(scales));
  else Py_INCREF(ps);
  if (res) pr = give(a[6], std::move(sum));
  else Py_INCREF(pr);
  PyObject* t = pq && ps && pr ? PyTuple_New(3) : nullptr;
  if (!t) {
    Py_XDECREF(pq);
    Py_XDECREF(ps);
    Py_XDECREF(pr);
    return nullptr;
  }
  PyTuple_SET_ITEM(t, 0, pq);
  PyTuple_SET_ITEM(t, 1, ps);
  PyTuple_SET_ITEM(t, 2, pr);
  return t;
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"gemv", (PyCFunction)(void (*)(void))gemv, METH_FASTCALL, "products of few rows"},
    {"grouped", (PyCFunction)(void (*)(void))grouped, METH_FASTCALL, "products of rows grouped by expert"},
    {"norm", (PyCFunction)(void (*)(void))norm, METH_FASTCALL, "norm and quantization"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fastcalls", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__fastcalls() { return PyModule_Create(&kModule); }
