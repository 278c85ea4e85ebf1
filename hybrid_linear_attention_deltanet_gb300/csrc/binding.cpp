// The layer operators' calls from Python for the ordinary case: tensors in,
// new tensors out, on the current stream.  A decoding step makes these calls
// for single tokens, where the interpreter's checks and allocations took
// longer than the kernels (8-bit norm of one token: 17.7 us a call through
// ctypes).  Each function checks its arguments, allocates the outputs and
// calls the C ABI; where anything is not as it expects (another type, shape,
// stride or device, a refusal by the library) it returns None and has done
// nothing, and the Python binding takes its own path, which names the error.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/gdn.h"

namespace {

struct Library {
  decltype(&gdn_residual_norm) residual_norm = nullptr;
  decltype(&gdn_residual_norm_fp8) residual_norm_fp8 = nullptr;
  decltype(&gdn_residual_norm_backward) residual_norm_backward = nullptr;
  decltype(&gdn_quantize_fp8) quantize_fp8 = nullptr;
  decltype(&gdn_linear_fp8) linear_fp8 = nullptr;
  decltype(&gdn_gated_ffn) gated_ffn = nullptr;
  decltype(&gdn_gated_ffn_backward) gated_ffn_backward = nullptr;
  bool ready = false;
} lib;

constexpr int64_t kBlock = 128;
constexpr auto kFp8 = at::ScalarType::Float8_e4m3fn;

int64_t blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }

// The device of tensor `o`, which must be the current one; -1 otherwise.
c10::DeviceIndex device_of(PyObject* o) {
  if (!THPVariable_Check(o)) return -1;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda()) return -1;
  const c10::DeviceIndex index = t.device().index();
  return index == c10::cuda::current_device() ? index : -1;
}
// A plain CUDA tensor of this type, contiguous, on the current device; at
// least one element.
const at::Tensor* plain(PyObject* o, at::ScalarType type, c10::DeviceIndex index) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != index ||
      t.scalar_type() != type || t.dim() < 1 || t.numel() < 1 || !t.is_contiguous())
    return nullptr;
  return &t;
}
// bf16 or fp32, the io types of the C ABI; -1 for others
int io_code(PyObject* o) {
  if (!THPVariable_Check(o)) return -1;
  const auto type = THPVariable_Unpack(o).scalar_type();
  return type == at::kBFloat16 ? GDN_BF16 : type == at::kFloat ? GDN_F32 : -1;
}
at::ScalarType io_type(int code) { return code == GDN_BF16 ? at::kBFloat16 : at::kFloat; }

// New tensors on x's device, straight from the CUDA allocator (what at::empty
// comes to behind its dispatch, which costs 0.3 us a tensor).
at::Tensor make(const at::Tensor& x, c10::IntArrayRef shape, at::ScalarType type) {
  return at::detail::empty_cuda(shape, type, x.device(), std::nullopt);
}
at::Tensor like(const at::Tensor& x) { return make(x, x.sizes(), x.scalar_type()); }
// x's shape with its last axis replaced
at::Tensor with_last(const at::Tensor& x, int64_t last, at::ScalarType type) {
  c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
  shape.back() = last;
  return make(x, shape, type);
}
bool leading_and_last(const at::Tensor& t, const at::Tensor& x, int64_t last) {
  return t.dim() == x.dim() && t.size(-1) == last &&
         t.sizes().slice(0, t.dim() - 1) == x.sizes().slice(0, x.dim() - 1);
}
bool is_vector(const at::Tensor& t, int64_t n) { return t.dim() == 1 && t.size(0) == n; }

gdn_stream_t stream_of(c10::DeviceIndex index) {
  return (gdn_stream_t)c10::cuda::getCurrentCUDAStream(index).stream();
}
template <typename F>
bool call(F&& f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc == GDN_OK;
}
PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* none() { Py_RETURN_NONE; }
// a new tuple of new references
PyObject* pack(std::initializer_list<PyObject*> items) {
  PyObject* r = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (!o || !r) {
      Py_XDECREF(o);
      Py_CLEAR(r);
      continue;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// (x, w, residual or None, eps) -> the checked inputs
struct NormIn {
  const at::Tensor *x = nullptr, *w = nullptr, *r = nullptr;
  double eps = 0;
  int io = -1;
  int64_t dim = 0, tokens = 0;
  c10::DeviceIndex index = 0;
};
bool norm_in(PyObject* const* a, Py_ssize_t n, NormIn& v) {
  if (!lib.ready || n != 4) return false;
  v.io = io_code(a[0]);
  if (v.io < 0) return false;
  v.index = device_of(a[0]);
  if (v.index < 0) return false;
  v.x = plain(a[0], io_type(v.io), v.index);
  v.w = plain(a[1], at::kFloat, v.index);
  if (!v.x || !v.w) return false;
  v.dim = v.x->size(-1);
  v.tokens = v.x->numel() / v.dim;
  if (!is_vector(*v.w, v.dim) || v.dim > INT32_MAX) return false;
  if (a[2] != Py_None) {
    v.r = plain(a[2], io_type(v.io), v.index);
    if (!v.r || v.r->sizes() != v.x->sizes()) return false;
  }
  v.eps = PyFloat_AsDouble(a[3]);
  if (v.eps == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}
void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

PyObject* residual_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  NormIn v;
  if (!norm_in(a, n, v)) return none();
  at::Tensor y = like(*v.x);
  at::Tensor s = v.r ? like(*v.x) : at::Tensor();
  const gdn_stream_t st = stream_of(v.index);
  if (!call([&] {
        return lib.residual_norm(ptr(v.x), ptr(v.r), (const float*)ptr(v.w), (float)v.eps,
                                 v.r ? s.data_ptr() : nullptr, y.data_ptr(), v.tokens,
                                 (int32_t)v.dim, v.io, st);
      }))
    return none();
  return pack({wrap(y), v.r ? wrap(s) : Py_NewRef(a[0])});
  END_HANDLE_TH_ERRORS
}

PyObject* residual_norm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  NormIn v;
  if (!norm_in(a, n, v)) return none();
  at::Tensor q = make(*v.x, v.x->sizes(), kFp8);
  at::Tensor scale = with_last(*v.x, blocks(v.dim), at::kFloat);
  at::Tensor s = v.r ? like(*v.x) : at::Tensor();
  const gdn_stream_t st = stream_of(v.index);
  if (!call([&] {
        return lib.residual_norm_fp8(ptr(v.x), ptr(v.r), (const float*)ptr(v.w), (float)v.eps,
                                     v.r ? s.data_ptr() : nullptr, q.data_ptr(),
                                     (float*)scale.data_ptr(), v.tokens, (int32_t)v.dim, v.io, st);
      }))
    return none();
  return pack({wrap(q), wrap(scale), v.r ? wrap(s) : Py_NewRef(a[0])});
  END_HANDLE_TH_ERRORS
}

// (dy, s, w, ds or None, eps) -> (dx, dw)
PyObject* residual_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5) return none();
  PyObject* in[4] = {a[1], a[2], a[3], a[4]};   // s and ds as x and residual
  NormIn v;
  if (!norm_in(in, 4, v)) return none();
  const at::Tensor* dy = plain(a[0], io_type(v.io), v.index);
  if (!dy || dy->sizes() != v.x->sizes()) return none();
  at::Tensor dx = like(*v.x);
  at::Tensor dw = like(*v.w);
  const gdn_stream_t st = stream_of(v.index);
  if (!call([&] {
        return lib.residual_norm_backward(ptr(dy), ptr(v.x), (const float*)ptr(v.w), ptr(v.r),
                                          (float)v.eps, dx.data_ptr(), (float*)dw.data_ptr(),
                                          v.tokens, (int32_t)v.dim, v.io, st);
      }))
    return none();
  return pack({wrap(dx), wrap(dw)});
  END_HANDLE_TH_ERRORS
}

// an int argument, or `other` where it is none
long int_arg(PyObject* o, long other) {
  if (!PyLong_CheckExact(o)) return other;
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return other;
  }
  return v;
}

// (x, block_rows) -> (q, scale)
PyObject* quantize_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!lib.ready || n != 2) return none();
  const int io = io_code(a[0]);
  const long block_rows = int_arg(a[1], 0);
  if (io < 0 || (block_rows != 1 && block_rows != kBlock)) return none();
  const c10::DeviceIndex index = device_of(a[0]);
  if (index < 0) return none();
  const at::Tensor* x = plain(a[0], io_type(io), index);
  if (!x || (block_rows != 1 && x->dim() != 2) || x->size(-1) > INT32_MAX) return none();
  const int64_t cols = x->size(-1), rows = x->numel() / cols;
  at::Tensor q = make(*x, x->sizes(), kFp8);
  at::Tensor scale = block_rows == 1 ? with_last(*x, blocks(cols), at::kFloat)
                                     : make(*x, {blocks(rows), blocks(cols)}, at::kFloat);
  const gdn_stream_t st = stream_of(index);
  if (!call([&] {
        return lib.quantize_fp8(ptr(x), q.data_ptr(), (float*)scale.data_ptr(), rows,
                                (int32_t)cols, (int32_t)block_rows, io, st);
      }))
    return none();
  return pack({wrap(q), wrap(scale)});
  END_HANDLE_TH_ERRORS
}

// (x, x_scale, w, w_scale, io code of the result) -> out
PyObject* linear_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!lib.ready || n != 5) return none();
  const long code = int_arg(a[4], -1);
  if (code != GDN_BF16 && code != GDN_F32) return none();
  const c10::DeviceIndex index = device_of(a[0]);
  if (index < 0) return none();
  const at::Tensor *x = plain(a[0], kFp8, index), *sx = plain(a[1], at::kFloat, index),
                   *w = plain(a[2], kFp8, index), *sw = plain(a[3], at::kFloat, index);
  if (!x || !sx || !w || !sw || w->dim() != 2 || sw->dim() != 2) return none();
  const int64_t k = w->size(1), rows = w->size(0);
  if (x->size(-1) != k || k > INT32_MAX || rows > INT32_MAX ||
      !leading_and_last(*sx, *x, blocks(k)) || sw->size(0) != blocks(rows) ||
      sw->size(1) != blocks(k))
    return none();
  at::Tensor out = with_last(*x, rows, io_type((int)code));
  const gdn_stream_t st = stream_of(index);
  if (!call([&] {
        return lib.linear_fp8(ptr(x), (const float*)ptr(sx), ptr(w), (const float*)ptr(sw),
                              out.data_ptr(), x->numel() / k, (int32_t)k, (int32_t)rows,
                              (int32_t)code, st);
      }))
    return none();
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

struct FfnIn {
  const at::Tensor *x = nullptr, *wg = nullptr, *wu = nullptr;
  int64_t dim = 0, hidden = 0, tokens = 0;
  long act = -1;
  c10::DeviceIndex index = 0;
};
bool ffn_in(PyObject* x, PyObject* wg, PyObject* wu, PyObject* act, FfnIn& v) {
  if (!lib.ready) return false;
  v.act = int_arg(act, -1);
  if (v.act != GDN_GATE_SILU && v.act != GDN_GATE_SIGMOID) return false;
  v.index = device_of(x);
  if (v.index < 0) return false;
  v.x = plain(x, at::kBFloat16, v.index);
  v.wg = plain(wg, at::kBFloat16, v.index);
  v.wu = plain(wu, at::kBFloat16, v.index);
  if (!v.x || !v.wg || !v.wu || v.wg->dim() != 2 || v.wu->sizes() != v.wg->sizes()) return false;
  v.hidden = v.wg->size(0);
  v.dim = v.wg->size(1);
  if (v.x->size(-1) != v.dim || v.dim > INT32_MAX || v.hidden > INT32_MAX) return false;
  v.tokens = v.x->numel() / v.dim;
  return true;
}

// (x, w_gate, w_up, act code) -> h
PyObject* gated_ffn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  FfnIn v;
  if (n != 4 || !ffn_in(a[0], a[1], a[2], a[3], v)) return none();
  at::Tensor h = with_last(*v.x, v.hidden, at::kBFloat16);
  const gdn_stream_t st = stream_of(v.index);
  if (!call([&] {
        return lib.gated_ffn(ptr(v.x), ptr(v.wg), ptr(v.wu), (int32_t)v.act, h.data_ptr(),
                             v.tokens, (int32_t)v.dim, (int32_t)v.hidden, GDN_BF16, st);
      }))
    return none();
  return wrap(h);
  END_HANDLE_TH_ERRORS
}

// (x, w_gate, w_up, dh, act code) -> (dx, dw_gate, dw_up)
PyObject* gated_ffn_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  FfnIn v;
  if (n != 5 || !ffn_in(a[0], a[1], a[2], a[4], v)) return none();
  const at::Tensor* dh = plain(a[3], at::kBFloat16, v.index);
  if (!dh || !leading_and_last(*dh, *v.x, v.hidden)) return none();
  at::Tensor dx = like(*v.x);
  at::Tensor dwg = like(*v.wg);
  at::Tensor dwu = like(*v.wu);
  const gdn_stream_t st = stream_of(v.index);
  if (!call([&] {
        return lib.gated_ffn_backward(ptr(v.x), ptr(v.wg), ptr(v.wu), ptr(dh), (int32_t)v.act,
                                      dx.data_ptr(), dwg.data_ptr(), dwu.data_ptr(), v.tokens,
                                      (int32_t)v.dim, (int32_t)v.hidden, GDN_BF16, st);
      }))
    return none();
  return pack({wrap(dx), wrap(dwg), wrap(dwu)});
  END_HANDLE_TH_ERRORS
}

// bind(path of the library, already loaded): looks its functions up
PyObject* bind(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* h = dlopen(p, RTLD_NOW | RTLD_NOLOAD);
  if (!h) {
    PyErr_Format(PyExc_ImportError, "%s is not loaded", p);
    return nullptr;
  }
  bool ok = true;
  auto find = [&](auto& f, const char* name) {
    f = (std::decay_t<decltype(f)>)dlsym(h, name);
    ok = ok && f;
  };
  find(lib.residual_norm, "gdn_residual_norm");
  find(lib.residual_norm_fp8, "gdn_residual_norm_fp8");
  find(lib.residual_norm_backward, "gdn_residual_norm_backward");
  find(lib.quantize_fp8, "gdn_quantize_fp8");
  find(lib.linear_fp8, "gdn_linear_fp8");
  find(lib.gated_ffn, "gdn_gated_ffn");
  find(lib.gated_ffn_backward, "gdn_gated_ffn_backward");
  lib.ready = ok;
  if (!ok) {
    PyErr_Format(PyExc_ImportError, "%s lacks an entry point", p);
    return nullptr;
  }
  Py_RETURN_NONE;
}

#define GDN_CALL(name) \
  {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", bind, METH_O, nullptr},
    GDN_CALL(residual_norm),
    GDN_CALL(residual_norm_fp8),
    GDN_CALL(residual_norm_backward),
    GDN_CALL(quantize_fp8),
    GDN_CALL(linear_fp8),
    GDN_CALL(gated_ffn),
    GDN_CALL(gated_ffn_backward),
    {nullptr, nullptr, 0, nullptr}};
#undef GDN_CALL
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_calls",
                      "Direct calls of the layer operators (None: take the general path).", -1,
                      methods};

}  // namespace

PyMODINIT_FUNC PyInit__layer_calls(void) { return PyModule_Create(&module); }
