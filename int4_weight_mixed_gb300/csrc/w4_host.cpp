// w4_host.cpp — the binding's per-call work for the norm and for products with
// an epilogue of their own: checks of the tensors, outputs, the call into
// libw4.  The smallest of these calls are host time: a norm of one row takes
// 1.5 us on the GPU, and the host 13.1 us a call when this work was Python's
// and ctypes', 4.6 here (a gated product of one row 16.1 and 5.4; both with
// the outputs allocated).
//
// A plain CPython extension module on torch's C++ tensors; the package's
// __init__.py documents the entry points and calls them with every argument
// in place.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/w4.h"

namespace {

// Objects of the Python module (init): the workspaces by (device, stream), the
// function that makes one, and the one that raises a library error.
PyObject *ws_cache, *make_workspace, *raise_status;

struct Bad {};  // a Python error is set

[[noreturn]] void bad(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Bad();
}
[[noreturn]] void bad_value(const std::string& what) { bad(PyExc_ValueError, what); }

// The tensor of an argument, or null for None.
const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) bad(PyExc_TypeError, std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Bad();
  return v;
}

int code_of(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return W4_F16;
    case at::kBFloat16: return W4_BF16;
    case at::kChar: return W4_S8;
    case at::kInt: return W4_S32;
    case at::kFloat8_e4m3fn: return W4_E4M3;
    default: bad(PyExc_KeyError, std::string("torch type ") + c10::toString(t));
  }
}
at::ScalarType type_of(int code) {
  switch (code) {
    case W4_F16: return at::kHalf;
    case W4_BF16: return at::kBFloat16;
    case W4_S8: return at::kChar;
    case W4_S32: return at::kInt;
    default: return at::kFloat8_e4m3fn;
  }
}

// The kernels read every array densely from its first element: each given
// tensor must be a contiguous CUDA tensor on dev.
void dense(const at::Tensor* t, c10::Device dev, const char* name) {
  if (!t) return;
  if (!t->is_cuda() || t->device() != dev)
    bad_value(std::string(name) + " must be a CUDA tensor on " + dev.str() + " (got " +
              t->device().str() + ")");
  if (!t->is_contiguous()) bad_value(std::string(name) + " must be contiguous");
}
void holds(const at::Tensor* t, int64_t n, at::ScalarType type, const char* name) {
  if (t && (t->numel() != n || t->scalar_type() != type))
    bad_value(std::string(name) + " must hold " + std::to_string(n) + " values of " +
              c10::toString(type) + " (got " + std::to_string(t->numel()) + " of " +
              c10::toString(t->scalar_type()) + ")");
}

const void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
void* out_ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// Whether dev, the tensors' device, is the current one: the library plans for
// that one and launches on it.  If not, the entry points return NotImplemented
// and the Python module calls again with dev current (a guard of torch's here
// would be the same, but could not be tried without a second GPU).
bool is_current(c10::Device dev) {
  c10::DeviceIndex now = -1;
  return c10::cuda::GetDevice(&now) == cudaSuccess && now == dev.index();
}

at::Tensor empty(c10::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

void check(int status, const char* where) {
  if (status == W4_OK) return;
  PyObject* r = PyObject_CallFunction(raise_status, "is", status, where);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, where);
  throw Bad();
}

// The argument itself where it was given, else the tensor made for it.
PyObject* result(PyObject* given, const at::Tensor& t) {
  if (given == Py_None) return THPVariable_Wrap(t);
  Py_INCREF(given);
  return given;
}

// norm(x, weight, eps, residual, out, scales, residual_out, code): code is the
// 8-bit output's type, or -1 for x's
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  try {
    if (nargs != 8) bad(PyExc_TypeError, "norm takes 8 arguments");
    const at::Tensor* x = tensor(a[0], "x");
    if (!x) bad(PyExc_TypeError, "x must be a tensor");
    const at::Tensor *weight = tensor(a[1], "weight"), *residual = tensor(a[3], "residual");
    const at::Tensor *y = tensor(a[4], "out"), *scales = tensor(a[5], "scales");
    const at::Tensor* h = tensor(a[6], "residual_out");
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred()) throw Bad();
    const int64_t code = integer(a[7]);
    const at::ScalarType dt = x->scalar_type();
    const at::ScalarType yt = code < 0 ? dt : type_of(static_cast<int>(code));
    const c10::Device dev = x->device();
    const c10::IntArrayRef shape = x->sizes();
    if (y && (y->scalar_type() != yt || y->sizes() != shape))
      bad_value(code < 0 ? "out must have x's type and shape"
                         : std::string("out must be ") + c10::toString(yt) + " of x's shape");
    if (scales && (scales->scalar_type() != at::kFloat || scales->dim() + 1 != x->dim() ||
                   scales->sizes() != shape.slice(0, shape.size() - 1)))
      bad_value("scales must be fp32, one per row of x");
    dense(x, dev, "x");
    dense(weight, dev, "weight");
    dense(residual, dev, "residual");
    dense(y, dev, "out");
    dense(scales, dev, "scales");
    dense(h, dev, "residual_out");
    if (shape.empty()) bad_value("x needs at least one dimension");
    if (dt != at::kHalf && dt != at::kBFloat16)
      bad_value(std::string("x must be fp16 or bf16 (got ") + c10::toString(dt) + ")");
    const int64_t K = shape.back(), n = x->numel();
    int64_t M = 1;
    for (size_t i = 0; i + 1 < shape.size(); ++i) M *= shape[i];
    holds(weight, K, dt, "weight");
    holds(residual, n, dt, "residual");
    holds(h, n, dt, "residual_out");
    if (!is_current(dev)) Py_RETURN_NOTIMPLEMENTED;
    at::Tensor y_new, s_new, h_new;
    if (!y) y = &(y_new = empty(shape, yt, dev));
    if (!scales && code >= 0) scales = &(s_new = empty(shape.slice(0, shape.size() - 1), at::kFloat, dev));
    if (!h && residual) h = &(h_new = empty(shape, dt, dev));
    void* const stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    const int x_code = dt == at::kHalf ? W4_F16 : W4_BF16;
    const void *px = ptr(x), *pr = ptr(residual), *pw = ptr(weight);
    void *const ph = out_ptr(h), *const py = out_ptr(y);
    float* const ps = static_cast<float*>(out_ptr(scales));
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = w4_rmsnorm(px, x_code, M, K, pr, pw, static_cast<float>(eps), ph, py,
                    code < 0 ? x_code : static_cast<int>(code), ps, stream);
    Py_END_ALLOW_THREADS
    check(st, "w4_rmsnorm");
    if (code < 0 && !residual) return result(a[4], *y);
    PyObject* t = PyTuple_New(1 + (code >= 0) + (residual != nullptr));
    if (!t) return nullptr;
    int i = 0;
    PyTuple_SET_ITEM(t, i++, result(a[4], *y));
    if (code >= 0) PyTuple_SET_ITEM(t, i++, result(a[5], *scales));
    if (residual) PyTuple_SET_ITEM(t, i++, result(a[6], *h));
    if (PyErr_Occurred()) {  // an output without a Python object
      Py_DECREF(t);
      return nullptr;
    }
    return t;
  } catch (const Bad&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// The workspace of a's stream: the cached one (whatever its size), or one of at
// least `bytes` bytes from the Python module.
at::Tensor workspace(PyObject* a, c10::Device dev, void* stream, int64_t bytes) {
  if (bytes == 0 && c10::cuda::currentStreamCaptureStatusMayInitCtx() ==
                        c10::cuda::CaptureStatus::None) {
    PyObject* key = Py_BuildValue("(iK)", static_cast<int>(dev.index()),
                                  static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(stream)));
    if (!key) throw Bad();
    PyObject* ws = PyDict_GetItemWithError(ws_cache, key);
    Py_DECREF(key);
    if (ws) return THPVariable_Unpack(ws);
    if (PyErr_Occurred()) throw Bad();
  }
  PyObject* device = PyObject_GetAttrString(a, "device");
  if (!device) throw Bad();
  PyObject* ws = PyObject_CallFunction(make_workspace, "OL", device, static_cast<long long>(bytes));
  Py_DECREF(device);
  if (!ws) throw Bad();
  at::Tensor t = THPVariable_Unpack(ws);
  Py_DECREF(ws);
  return t;
}

// The sizes and types of a product's arrays (the library sees addresses alone).
struct Product {
  const at::Tensor *a, *b, *scales, *zeros, *s_tok, *s_ch, *out, *ws, *bias, *residual;
  int64_t N, gs;
  at::ScalarType ot;  // of the output
  int gated;
  int64_t M, K, cols;
  c10::Device dev = c10::Device(c10::kCPU);

  void devices() {
    dev = a->device();
    dense(a, dev, "a");
    dense(b, dev, "b_packed");
    dense(scales, dev, "scales");
    dense(zeros, dev, "zeros");
    dense(s_tok, dev, "token_scales");
    dense(s_ch, dev, "channel_scales");
    dense(out, dev, "out");
    dense(ws, dev, "ws");
    dense(bias, dev, "bias");
    dense(residual, dev, "residual");
    if (a->dim() != 2) bad_value("a must be [M, K]");
    M = a->size(0);
    K = a->size(1);
    cols = gated ? N / 2 : N;
  }
  void sizes() const {
    const int64_t n_groups = N * (gs == -1 ? 1 : gs > 0 ? K / gs : 0);
    if (M && static_cast<int64_t>(b->nbytes()) < (N + 127) / 128 * 64 * K)
      bad_value("b_packed is smaller than the prepacked " + std::to_string(K) + " x " +
                std::to_string(N) + " weight");
    // (over no K no scale is read, however many groups the array has)
    if (scales && K) holds(scales, n_groups, scales->scalar_type(), "scales");
    if (K) holds(zeros, n_groups, ot, "zeros");
    holds(s_tok, M, at::kFloat, "token_scales");
    holds(s_ch, N, at::kFloat, "channel_scales");
    holds(bias, N, ot, "bias");
    holds(residual, M * cols, ot, "residual");
    holds(out, M * cols, ot, "out");
  }
};

// gemm(a, b_packed, wtype, N, scales, zeros, group_size, token_scales,
// channel_scales, out_code (-1: by a), out, ws, schedule, bias, act, gated,
// residual)
PyObject* gemm(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  try {
    if (nargs != 17) bad(PyExc_TypeError, "gemm takes 17 arguments");
    const at::Tensor *a = tensor(v[0], "a"), *b = tensor(v[1], "b_packed");
    if (!a || !b) bad(PyExc_TypeError, "a and b_packed must be tensors");
    const int wtype = static_cast<int>(integer(v[2]));
    const int64_t N = integer(v[3]), gs = integer(v[6]);
    const at::Tensor *scales = tensor(v[4], "scales"), *zeros = tensor(v[5], "zeros");
    const at::Tensor *s_tok = tensor(v[7], "token_scales"), *s_ch = tensor(v[8], "channel_scales");
    const int64_t out_code = integer(v[9]);
    const at::Tensor *out = tensor(v[10], "out"), *ws = tensor(v[11], "ws");
    const int schedule = static_cast<int>(integer(v[12]));
    const at::Tensor *bias = tensor(v[13], "bias"), *residual = tensor(v[16], "residual");
    const int act = static_cast<int>(integer(v[14]));
    const int gated = PyObject_IsTrue(v[15]);
    if (gated < 0) throw Bad();
    Product p{a, b, scales, zeros, s_tok, s_ch, out, ws, bias, residual, N, gs, at::kHalf, gated};
    p.devices();
    const int a_code = code_of(a->scalar_type());
    const at::ScalarType ot = out_code >= 0 ? type_of(static_cast<int>(out_code))
                              : a_code == W4_S8 || a_code == W4_E4M3 ? at::kHalf
                                                                     : a->scalar_type();
    p.ot = ot;
    p.sizes();
    if (!is_current(p.dev)) Py_RETURN_NOTIMPLEMENTED;
    const int64_t M = p.M, K = p.K;
    const c10::Device dev = p.dev;
    at::Tensor o_new;
    if (!out) out = &(o_new = empty({M, p.cols}, ot, dev));
    void* const stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    const int s_code = scales ? code_of(scales->scalar_type()) : a_code, o_code = code_of(ot);
    const void *pa = ptr(a), *pb = ptr(b), *ps = ptr(scales), *pz = ptr(zeros);
    const void *pbias = ptr(bias), *pr = ptr(residual);
    const float *pt = static_cast<const float*>(ptr(s_tok)), *pc = static_cast<const float*>(ptr(s_ch));
    void* const po = out_ptr(out);
    // The library checks the workspace against its plan before it launches
    // anything: the stream's cached one is tried as it is, and the size asked
    // for when it is too small.
    at::Tensor w_new;
    int st;
    for (int64_t bytes = 0;;
         bytes = static_cast<int64_t>(w4_gemm_workspace_size(M, N, K, a_code, gs))) {
      if (!ws) w_new = workspace(v[0], dev, stream, bytes);
      const at::Tensor& w = ws ? *ws : w_new;
      void* const pw = out_ptr(&w);
      const size_t nw = static_cast<size_t>(w.numel());
      Py_BEGIN_ALLOW_THREADS
      st = w4_gemm_epilogue(pa, a_code, M, K, pb, wtype, N, ps, s_code, pz, gs, pt, pc, pbias, act,
                            gated, pr, po, o_code, pw, nw, stream, schedule);
      Py_END_ALLOW_THREADS
      if (st != W4_ERR_WORKSPACE || ws || bytes) break;
    }
    check(st, "w4_gemm_epilogue");
    return result(v[10], *out);
  } catch (const Bad&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// gemm_dynamic(a, b_packed, wtype, N, act_code, scales, group_size,
// channel_scales, bias, out, token_scales_out, ws, act, gated, residual)
PyObject* gemm_dynamic(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  try {
    if (nargs != 15) bad(PyExc_TypeError, "gemm_dynamic takes 15 arguments");
    const at::Tensor *a = tensor(v[0], "a"), *b = tensor(v[1], "b_packed");
    if (!a || !b) bad(PyExc_TypeError, "a and b_packed must be tensors");
    const int wtype = static_cast<int>(integer(v[2])), code = static_cast<int>(integer(v[4]));
    const int64_t N = integer(v[3]), gs = integer(v[6]);
    const at::Tensor *scales = tensor(v[5], "scales"), *s_ch = tensor(v[7], "channel_scales");
    const at::Tensor *bias = tensor(v[8], "bias"), *out = tensor(v[9], "out");
    const at::Tensor *s_tok = tensor(v[10], "token_scales_out"), *ws = tensor(v[11], "ws");
    const at::Tensor* residual = tensor(v[14], "residual");
    const int act = static_cast<int>(integer(v[12]));
    const int gated = PyObject_IsTrue(v[13]);
    if (gated < 0) throw Bad();
    Product p{a, b, scales, nullptr, s_tok, s_ch, out, ws, bias, residual, N, gs, at::kHalf, gated};
    p.devices();
    p.sizes();
    if (!is_current(p.dev)) Py_RETURN_NOTIMPLEMENTED;
    const int64_t M = p.M, K = p.K;
    at::Tensor o_new, w_new;
    if (!out) out = &(o_new = empty({M, p.cols}, at::kHalf, p.dev));
    void* const stream = c10::cuda::getCurrentCUDAStream(p.dev.index()).stream();
    const int a_code = code_of(a->scalar_type());
    const int s_code = scales ? code_of(scales->scalar_type()) : W4_S8;
    const void *pa = ptr(a), *pb = ptr(b), *ps = ptr(scales), *pbias = ptr(bias), *pr = ptr(residual);
    const float* pc = static_cast<const float*>(ptr(s_ch));
    float* const pt = static_cast<float*>(out_ptr(s_tok));
    void* const po = out_ptr(out);
    int st;
    for (int64_t bytes = 0;; bytes = static_cast<int64_t>(
                                 w4_gemm_dynamic_workspace_size(M, N, K, code, gs))) {
      if (!ws) w_new = workspace(v[0], p.dev, stream, bytes);
      const at::Tensor& w = ws ? *ws : w_new;
      void* const pw = out_ptr(&w);
      const size_t nw = static_cast<size_t>(w.numel());
      Py_BEGIN_ALLOW_THREADS
      st = w4_gemm_dynamic_epilogue(pa, a_code, M, K, pb, wtype, N, ps, s_code, gs, pc, code, pbias,
                                    act, gated, pr, po, pt, pw, nw, stream);
      Py_END_ALLOW_THREADS
      if (st != W4_ERR_WORKSPACE || ws || bytes) break;
    }
    check(st, "w4_gemm_dynamic_epilogue");
    return result(v[9], *out);
  } catch (const Bad&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// init(ws_cache, workspace, check)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (nargs != 3) {
    PyErr_SetString(PyExc_TypeError, "init takes 3 arguments");
    return nullptr;
  }
  for (int i = 0; i < 3; ++i) Py_INCREF(a[i]);
  ws_cache = a[0];
  make_workspace = a[1];
  raise_status = a[2];
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(init)), METH_FASTCALL, nullptr},
    {"norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm)), METH_FASTCALL, nullptr},
    {"gemm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gemm)), METH_FASTCALL, nullptr},
    {"gemm_dynamic", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gemm_dynamic)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "w4_host", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_w4_host() { return PyModule_Create(&module); }
