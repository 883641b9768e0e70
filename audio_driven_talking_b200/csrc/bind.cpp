// bind.cpp - the Python binding of the microscaled operators: checks of arguments, outputs from
// torch's allocator on torch's current stream of the tensors' device, and the C calls of
// include/fh_ops.h. A call of these operators on a few rows is shorter on the GPU than in Python:
// checks and allocations there took 7 us a call beside the 4 of the C call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/core/InferenceMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>

#include "fh.h"
#include "fh_ops.h"

namespace {

PyObject *g_mx = nullptr, *g_error = nullptr;  // MXTensor and FHError
PyObject *s_data, *s_scales, *s_shape, *s_fmt, *s_mxfp8, *s_mxfp4, *s_gelu;

struct Ref {  // an owned reference
  PyObject* p;
  explicit Ref(PyObject* o) : p(o) {}
  Ref(const Ref&) = delete;
  ~Ref() { Py_XDECREF(p); }
  PyObject* give() {
    PyObject* r = p;
    p = nullptr;
    return r;
  }
};

bool type_error(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(PyExc_TypeError, fmt, ap);
  va_end(ap);
  return false;
}
bool value_error(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(PyExc_ValueError, fmt, ap);
  va_end(ap);
  return false;
}

// The library's error of a return code, as FHError(code, message)
bool library_ok(int rc) {
  if (rc == FH_OK) return true;
  Ref e(PyObject_CallFunction(g_error, "is", rc, fh_last_error()));
  if (e.p) PyErr_SetObject(g_error, e.p);
  return false;
}

// "mxfp8" or "mxfp4": the type code, else -1
int mx_code(PyObject* o) {
  if (o == s_mxfp8) return FH_MXFP8;
  if (o == s_mxfp4) return FH_MXFP4;
  if (!PyUnicode_Check(o)) return -1;
  if (PyUnicode_CompareWithASCIIString(o, "mxfp8") == 0) return FH_MXFP8;
  if (PyUnicode_CompareWithASCIIString(o, "mxfp4") == 0) return FH_MXFP4;
  return -1;
}
bool format(PyObject* o, int* code) {
  *code = mx_code(o);
  return *code >= 0 || value_error("format %R: expected one of ['mxfp4', 'mxfp8']", o);
}

bool kind_of(at::ScalarType t, const char* what, int* kind) {
  if (t == at::kFloat)
    *kind = FH_F32;
  else if (t == at::kBFloat16)
    *kind = FH_BF16;
  else
    return type_error("%s: expected float32 or bfloat16, got %s", what, c10::toString(t));
  return true;
}
bool dtype_kind(PyObject* o, const char* what, int* kind) {
  if (!THPDtype_Check(o)) return type_error("%s: expected a torch dtype, got %R", what, o);
  return kind_of(reinterpret_cast<THPDtype*>(o)->scalar_type, what, kind);
}
bool out_kind(PyObject* o, int* kind) {
  if (THPDtype_Check(o)) {
    const at::ScalarType t = reinterpret_cast<THPDtype*>(o)->scalar_type;
    if (t == at::kFloat || t == at::kBFloat16) {
      *kind = t == at::kFloat ? FH_F32 : FH_BF16;
      return true;
    }
  } else if ((*kind = mx_code(o)) >= 0) {
    return true;
  }
  return value_error("out=%R: expected torch.float32, torch.bfloat16, 'mxfp8' or 'mxfp4'", o);
}

// A CUDA tensor, on `device` where that is not negative; null with an error set. Those that torch.vmap
// and the transforms of torch.func pass on wrap another tensor and have no memory of their own.
const at::Tensor* cuda_tensor(PyObject* o, const char* what, int device = -1) {
  if (!THPVariable_Check(o)) {
    type_error("%s: expected a torch tensor", what);
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) {
    value_error("%s: expected a CUDA tensor", what);
    return nullptr;
  }
  if (device >= 0 && t.get_device() != device) {
    value_error("%s is on cuda:%d, expected cuda:%d", what, (int)t.get_device(), device);
    return nullptr;
  }
  if (!t.has_storage()) {
    value_error("%s has no storage: the operators take plain tensors, not ones that a transform wraps", what);
    return nullptr;
  }
  // forward only: what autograd would lose without a word is refused
  if ((t.requires_grad() && c10::GradMode::is_enabled()) ||
      (t._fw_grad(0).defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode())) {
    value_error("%s requires a gradient, which these operators do not give: detach it, or call them in torch.no_grad()",
                what);
    return nullptr;
  }
  return &t;
}
const at::Tensor* matrix(PyObject* o, const char* what, int device = -1) {
  const at::Tensor* t = cuda_tensor(o, what, device);
  if (!t) return nullptr;
  if (t->dim() != 2) {
    value_error("%s: expected 2 dimensions, got %d", what, (int)t->dim());
    return nullptr;
  }
  if (!t->is_contiguous()) {
    value_error("%s must be contiguous", what);
    return nullptr;
  }
  return t;
}
// sizes that the C calls take; what they refuse, they refuse
bool int_sizes(const at::Tensor& t, const char* what) {
  return (t.size(0) <= INT_MAX && t.size(1) <= INT_MAX) || value_error("%s: too large", what);
}

struct Mx {  // a microscaled operand
  const at::Tensor *data = nullptr, *scales = nullptr;
  Ref d{nullptr}, s{nullptr};  // keep them alive
  int code = 0, device = 0;
  long rows = 0, cols = 0;
};
long scale_bytes(long rows, long cols) { return (rows + 127) / 128 * ((cols + 127) / 128) * 512; }

bool mx_operand(PyObject* q, const char* what, int device, Mx* m) {
  const int is = PyObject_IsInstance(q, g_mx);
  if (is <= 0) return is < 0 ? false : type_error("%s: expected an MXTensor", what);
  Ref fmt(PyObject_GetAttr(q, s_fmt)), shape(PyObject_GetAttr(q, s_shape));
  m->d.p = PyObject_GetAttr(q, s_data);
  m->s.p = PyObject_GetAttr(q, s_scales);
  if (!fmt.p || !shape.p || !m->d.p || !m->s.p || !format(fmt.p, &m->code)) return false;
  if (!PyTuple_Check(shape.p) || PyTuple_GET_SIZE(shape.p) != 2)
    return type_error("%s.shape: expected a tuple of two, got %R", what, shape.p);
  m->rows = PyLong_AsLong(PyTuple_GET_ITEM(shape.p, 0));
  m->cols = PyLong_AsLong(PyTuple_GET_ITEM(shape.p, 1));
  if (PyErr_Occurred()) return false;
  if (m->rows < 1 || m->cols < 32 || m->cols % 32 || m->rows > INT_MAX || m->cols > INT_MAX)
    return value_error("%s: %ld x %ld is not a microscaled shape (columns: a multiple of 32)", what, m->rows, m->cols);
  char name[64];
  snprintf(name, sizeof name, "%s.data", what);
  if (!(m->data = cuda_tensor(m->d.p, name, device))) return false;
  m->device = m->data->get_device();
  const long n = m->rows * m->cols / (m->code == FH_MXFP4 ? 2 : 1), ns = scale_bytes(m->rows, m->cols);
  if (m->data->scalar_type() != at::kByte || m->data->numel() != n || !m->data->is_contiguous())
    return value_error("%s: expected %ld contiguous uint8 values", name, n);
  snprintf(name, sizeof name, "%s.scales", what);
  if (!(m->scales = cuda_tensor(m->s.p, name, m->device))) return false;
  if (m->scales->scalar_type() != at::kByte || m->scales->numel() != ns || !m->scales->is_contiguous())
    return value_error("%s: expected %ld contiguous uint8 values", name, ns);
  return true;
}

at::Tensor empty(long rows, long cols, at::ScalarType t, int device) {
  const int64_t size[2] = {rows, cols}, stride[2] = {cols, 1};
  return at::Tensor(at::detail::empty_strided_cuda(size, stride, t, at::Device(at::kCUDA, (at::DeviceIndex)device)));
}

struct Out {  // an output of the asked type
  at::Tensor data, scales;
  int kind;
  long rows, cols;
  Out(long r, long c, int k, int device) : kind(k), rows(r), cols(c) {
    if (k == FH_F32 || k == FH_BF16) {
      data = empty(r, c, k == FH_F32 ? at::kFloat : at::kBFloat16, device);
    } else {
      data = empty(r, k == FH_MXFP4 ? c / 2 : c, at::kByte, device);
      const int64_t n = scale_bytes(r, c), one = 1;
      scales = at::Tensor(at::detail::empty_strided_cuda(at::IntArrayRef(&n, 1), at::IntArrayRef(&one, 1), at::kByte,
                                                         at::Device(at::kCUDA, (at::DeviceIndex)device)));
    }
  }
  void* scale_ptr() const { return kind >= FH_MXFP8 ? scales.data_ptr() : nullptr; }
  // what the caller gets; a new reference
  PyObject* object() const {
    if (kind < FH_MXFP8) return THPVariable_Wrap(data);
    Ref d(THPVariable_Wrap(data)), s(THPVariable_Wrap(scales)), shape(Py_BuildValue("(ll)", rows, cols));
    if (!d.p || !s.p || !shape.p) return nullptr;
    PyObject* args[4] = {d.p, s.p, shape.p, kind == FH_MXFP8 ? s_mxfp8 : s_mxfp4};
    return PyObject_Vectorcall(g_mx, args, 4, nullptr);
  }
};

bool arg_count(Py_ssize_t n, Py_ssize_t want, const char* name) {
  return n == want || type_error("%s: expected %d arguments", name, (int)want);
}

// Pointers and the stream are read with the GIL held: reading them may throw, which must not happen
// between Py_BEGIN_ALLOW_THREADS and Py_END_ALLOW_THREADS.
const float* floats(const at::Tensor* t) { return t ? static_cast<const float*>(t->const_data_ptr()) : nullptr; }
void* stream_of(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

// quantize(x, fmt)
PyObject* py_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int code, kind;
  if (!arg_count(n, 2, "quantize") || !format(a[1], &code)) return nullptr;
  const at::Tensor* x = cuda_tensor(a[0], "x");
  if (!x || !kind_of(x->scalar_type(), "x", &kind)) return nullptr;
  if (x->dim() != 2 || x->stride(1) != 1) {
    value_error("x: expected 2 dimensions with contiguous rows");
    return nullptr;
  }
  if (!int_sizes(*x, "x")) return nullptr;
  const long M = x->size(0), K = x->size(1);
  const int dev = x->get_device();
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
  Out q(M, K, code, dev);
  const void* const xp = x->const_data_ptr();
  const long ldx = M > 1 ? x->stride(0) : K;
  void *const qp = q.data.data_ptr(), *const sp = q.scales.data_ptr(), *const st = stream_of(dev);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fh_op_quantize(xp, ldx, (int)M, (int)K, kind, code, qp, sp, st);
  Py_END_ALLOW_THREADS;
  return library_ok(rc) ? q.object() : nullptr;
  END_HANDLE_TH_ERRORS
}

// dequantize(q, dtype)
PyObject* py_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Mx q;
  int kind;
  if (!arg_count(n, 2, "dequantize") || !mx_operand(a[0], "q", -1, &q) || !dtype_kind(a[1], "dtype", &kind)) return nullptr;
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)q.device);
  Out out(q.rows, q.cols, kind, q.device);
  const void *const qp = q.data->const_data_ptr(), *const sp = q.scales->const_data_ptr();
  void *const op = out.data.data_ptr(), *const st = stream_of(q.device);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fh_op_dequantize(qp, sp, (int)q.rows, (int)q.cols, q.code, op, kind, st);
  Py_END_ALLOW_THREADS;
  return library_ok(rc) ? out.object() : nullptr;
  END_HANDLE_TH_ERRORS
}

// add_rms_norm(x, res, a, c, out, eps, sum_out)
PyObject* py_add_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int kind, xk, rk;
  if (!arg_count(n, 7, "add_rms_norm") || !out_kind(a[4], &kind)) return nullptr;
  const at::Tensor* x = matrix(a[0], "x");
  if (!x || !int_sizes(*x, "x")) return nullptr;
  const int dev = x->get_device();
  const at::Tensor* res = matrix(a[1], "res", dev);
  if (!res) return nullptr;
  const long M = x->size(0), D = x->size(1);
  if (!res->sizes().equals(x->sizes())) {
    value_error("res: expected shape (%ld, %ld), got (%ld, %ld)", M, D, (long)res->size(0), (long)res->size(1));
    return nullptr;
  }
  const at::Tensor* g = cuda_tensor(a[2], "a", dev);
  if (!g) return nullptr;
  if (g->scalar_type() != at::kFloat || (g->dim() != 1 && g->dim() != 2) || g->size(-1) != D || !g->is_contiguous()) {
    value_error("a: expected contiguous float32 [%ld] or [streams, %ld]", D, D);
    return nullptr;
  }
  const long streams = g->dim() == 2 ? g->size(0) : 1;
  if (streams < 1 || M % streams) {
    value_error("%ld rows do not divide into %ld streams", M, streams);
    return nullptr;
  }
  const at::Tensor* c = nullptr;
  if (a[3] != Py_None) {
    if (!(c = cuda_tensor(a[3], "c", dev))) return nullptr;
    if (c->scalar_type() != at::kFloat || !c->sizes().equals(g->sizes()) || !c->is_contiguous()) {
      value_error("c: expected a contiguous float32 tensor of a's shape");
      return nullptr;
    }
  }
  if (!kind_of(x->scalar_type(), "x", &xk) || !kind_of(res->scalar_type(), "res", &rk)) return nullptr;
  const double eps = PyFloat_AsDouble(a[5]);
  if (PyErr_Occurred()) return nullptr;
  const bool own = a[6] == Py_None;
  if (!own) {
    const at::Tensor* s = matrix(a[6], "sum_out", dev);
    if (!s) return nullptr;
    if (!s->sizes().equals(x->sizes()) || s->scalar_type() != x->scalar_type()) {
      value_error("sum_out: expected x's shape and type");
      return nullptr;
    }
    if (s->is_inference() && !c10::InferenceMode::is_enabled()) {
      value_error("sum_out: an inference tensor is written in inference mode only");
      return nullptr;
    }
  }
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
  const at::Tensor sum = own ? empty(M, D, x->scalar_type(), dev) : THPVariable_Unpack(a[6]);
  Out y(M, D, kind, dev);
  void* const tp = sum.data_ptr();
  const void *const xp = x->const_data_ptr(), *const rp = res->const_data_ptr();
  const float *const ap = floats(g), *const cp = floats(c);
  void *const yp = y.data.data_ptr(), *const sp = y.scale_ptr(), *const st = stream_of(dev);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fh_op_add_rms_norm(xp, xk, rp, rk, tp, ap, cp, streams > 1 ? D : 0, M > 0 ? (int)(M / streams) : 1, (int)M,
                          (int)D, (float)eps, kind, yp, sp, st);
  Py_END_ALLOW_THREADS;
  if (!library_ok(rc)) return nullptr;
  if (!own) sum.unsafeGetTensorImpl()->bump_version();  // autograd sees that what it saved was written
  Ref s(own ? THPVariable_Wrap(sum) : Py_NewRef(a[6])), o(y.object());
  return s.p && o.p ? PyTuple_Pack(2, s.p, o.p) : nullptr;
  END_HANDLE_TH_ERRORS
}

// linear_mx(A, W, bias, act, out)
PyObject* py_linear_mx(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int kind = FH_BF16;
  if (!arg_count(n, 5, "linear_mx") || (a[4] != Py_None && !out_kind(a[4], &kind))) return nullptr;
  const bool gelu = a[3] == s_gelu || (PyUnicode_Check(a[3]) && PyUnicode_CompareWithASCIIString(a[3], "gelu") == 0);
  if (!gelu && a[3] != Py_None) {
    value_error("act=%R: expected None or 'gelu'", a[3]);
    return nullptr;
  }
  Mx A, W;
  if (!mx_operand(a[0], "A", -1, &A) || !mx_operand(a[1], "W", A.device, &W)) return nullptr;
  if (A.code != W.code) {
    value_error("A is %s, W is %s: expected one format", A.code == FH_MXFP8 ? "mxfp8" : "mxfp4",
                W.code == FH_MXFP8 ? "mxfp8" : "mxfp4");
    return nullptr;
  }
  if (A.cols != W.cols) {
    value_error("A has %ld columns, W has %ld", A.cols, W.cols);
    return nullptr;
  }
  const long M = A.rows, N = W.rows, K = A.cols;
  const at::Tensor* bias = nullptr;
  if (a[2] != Py_None) {
    if (!(bias = cuda_tensor(a[2], "bias", A.device))) return nullptr;
    if (bias->scalar_type() != at::kFloat || bias->dim() != 1 || bias->size(0) != N || !bias->is_contiguous()) {
      value_error("bias: expected contiguous float32 [%ld]", N);
      return nullptr;
    }
  }
  if (kind >= FH_MXFP8 && N % 32) {
    value_error("%ld columns: a microscaled output needs a multiple of 32", N);
    return nullptr;
  }
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)A.device);
  Out y(M, N, kind, A.device);
  const void *const dA = A.data->const_data_ptr(), *const sA = A.scales->const_data_ptr();
  const void *const dW = W.data->const_data_ptr(), *const sW = W.scales->const_data_ptr();
  const float* const bp = floats(bias);
  void *const yp = y.data.data_ptr(), *const sp = y.scale_ptr(), *const st = stream_of(A.device);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fh_op_linear_mx(dA, sA, dW, sW, bp, (int)M, (int)N, (int)K, A.code, gelu ? FH_ACT_GELU : FH_ACT_NONE, kind, yp,
                       sp, st);
  Py_END_ALLOW_THREADS;
  return library_ok(rc) ? y.object() : nullptr;
  END_HANDLE_TH_ERRORS
}

// init(MXTensor, FHError)
PyObject* py_init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arg_count(n, 2, "init")) return nullptr;
  Py_XSETREF(g_mx, Py_NewRef(a[0]));
  Py_XSETREF(g_error, Py_NewRef(a[1]));
  Py_RETURN_NONE;
}

#define FH_DEF(name, fn, doc) {name, (PyCFunction)(void (*)(void))fn, METH_FASTCALL, doc}
PyMethodDef methods[] = {FH_DEF("init", py_init, "init(MXTensor, FHError)"),
                         FH_DEF("quantize", py_quantize, "quantize(x, fmt)"),
                         FH_DEF("dequantize", py_dequantize, "dequantize(q, dtype)"),
                         FH_DEF("add_rms_norm", py_add_rms_norm, "add_rms_norm(x, res, a, c, out, eps, sum_out)"),
                         FH_DEF("linear_mx", py_linear_mx, "linear_mx(A, W, bias, act, out)"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fhbind", "Microscaled operators of libfh.so", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__fhbind(void) {
  s_data = PyUnicode_InternFromString("data");
  s_scales = PyUnicode_InternFromString("scales");
  s_shape = PyUnicode_InternFromString("shape");
  s_fmt = PyUnicode_InternFromString("fmt");
  s_mxfp8 = PyUnicode_InternFromString("mxfp8");
  s_mxfp4 = PyUnicode_InternFromString("mxfp4");
  s_gelu = PyUnicode_InternFromString("gelu");
  return PyModule_Create(&module);
}
