// The 8-bit path's Python calls without ctypes: checks, outputs and the C call in one step. A decode
// step's kernels take 3 to 6 us each; through ctypes a call costs 7 to 10 us of host time, here 3.7 to 4.9
// (2.5 of it the runtime's launch).
//
// Every function here returns None, having done nothing, when an argument is not what the call takes
// (another type, shape, device, stride or a tensor subclass, or a gradient asked for), when another GPU is current, or when the
// library refuses: w8a8.py then goes through its own checks, which say what is wrong. The library's
// entry points (include/paro_w8a8.h) are handed over as addresses by bind().
#include <Python.h>
#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <ATen/core/grad_mode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <limits>

#include "paro_w8a8.h"

namespace {

decltype(&paro_rmsnorm_q8) g_rmsnorm_q8;
decltype(&paro_rmsnorm) g_rmsnorm;
decltype(&paro_quantize_q8) g_quantize;
decltype(&paro_pack_weights_q8) g_pack;
decltype(&paro_dequantize_q8) g_dequantize;
decltype(&paro_w8a8_linear) g_linear;
decltype(&paro_w8a8_gated_linear) g_gated;
decltype(&paro_w8a8_workspace_bytes) g_linear_ws;
decltype(&paro_w8a8_gated_workspace_bytes) g_gated_ws;

using at::ScalarType;
using at::Tensor;

const Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

int dtype_code(ScalarType t) {
  return t == ScalarType::Half ? PARO_F16 : t == ScalarType::BFloat16 ? PARO_BF16 : t == ScalarType::Float ? PARO_F32 : -1;
}

// A contiguous tensor of this type on GPU `device`, with these sizes.
bool fits(const Tensor* t, ScalarType type, int device, int64_t a) {
  return t && t->layout() == at::kStrided && t->scalar_type() == type && t->is_cuda() && t->get_device() == device &&
         t->dim() == 1 && t->size(0) == a && t->is_contiguous();
}
bool fits(const Tensor* t, ScalarType type, int device, int64_t a, int64_t b) {
  return t && t->layout() == at::kStrided && t->scalar_type() == type && t->is_cuda() && t->get_device() == device &&
         t->dim() == 2 && t->size(0) == a && t->size(1) == b && t->is_contiguous();
}
// A 2-d tensor on the current GPU whose sizes are ints.
bool starts(const Tensor* t, int* device, int* rows, int* cols) {
  if (!t || t->layout() != at::kStrided || !t->is_cuda() || t->dim() != 2 || !t->is_contiguous()) return false;
  constexpr int64_t kMax = std::numeric_limits<int>::max();
  if (t->size(0) > kMax || t->size(1) > kMax) return false;
  *device = t->get_device();
  *rows = int(t->size(0));
  *cols = int(t->size(1));
  return c10::hip::current_device() == *device;
}
void* stream(int device) { return c10::hip::getCurrentHIPStream(c10::DeviceIndex(device)).stream(); }
// A new tensor on the current GPU, from the allocator that `like` came from: torch's empty without its
// dispatcher, 0.3 us instead of 0.7. (Memory that torch has not allocated names no allocator.)
Tensor make(const Tensor& like, at::IntArrayRef sizes, ScalarType type) {
  if (c10::Allocator* const a = like.storage().allocator())
    return at::detail::empty_generic(sizes, a, c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt);
  return at::empty(sizes, like.options().dtype(type));
}

// An output argument: None (then `*t` becomes a new tensor) or a tensor that fits.
bool output(PyObject* o, const Tensor& like, int device, ScalarType type, at::IntArrayRef sizes, Tensor* t) {
  if (o == Py_None) {
    *t = make(like, sizes, type);
    return true;
  }
  const Tensor* given = tensor(o);
  if (!(sizes.size() == 1 ? fits(given, type, device, sizes[0]) : fits(given, type, device, sizes[0], sizes[1]))) return false;
  *t = *given;
  return true;
}

// Autograd would lose a gradient without a word: the calls are forward only.
template <class... T>
bool wants_grad(const T*... t) {
  return at::GradMode::is_enabled() && (... || (t && t->requires_grad()));
}
// A tensor of the caller's was written: its version counter says so to autograd.
void wrote(PyObject* o) {
  if (o == Py_None) return;
  const Tensor* const t = tensor(o);
  if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// The type of an output: `o` (a torch.dtype or None), else the output's own, else float16.
bool out_type(PyObject* o, const Tensor* out, ScalarType* type) {
  if (o == Py_None)
    *type = out ? out->scalar_type() : ScalarType::Half;
  else if (THPDtype_Check(o))
    *type = reinterpret_cast<THPDtype*>(o)->scalar_type;
  else
    return false;
  return dtype_code(*type) >= 0;
}

// (gated, x, x_scales, qweight, w_scales, out_dtype, out, ws) -> y
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) Py_RETURN_NONE;
  const bool gated = a[0] == Py_True;
  const Tensor *x = tensor(a[1]), *xs = tensor(a[2]), *w = tensor(a[3]), *wsc = tensor(a[4]);
  const Tensor* out = a[6] == Py_None ? nullptr : tensor(a[6]);
  const Tensor* ws = a[7] == Py_None ? nullptr : tensor(a[7]);
  int device, M, D, wdev, rows, wD;
  ScalarType type;
  if (!starts(x, &device, &M, &D) || !starts(w, &wdev, &rows, &wD) || wdev != device || wD != D || (gated && rows % 2) ||
      x->scalar_type() != ScalarType::Char || w->scalar_type() != ScalarType::Char || !out_type(a[5], out, &type) ||
      !fits(xs, ScalarType::Float, device, M) || !fits(wsc, ScalarType::Float, device, rows))
    Py_RETURN_NONE;
  const int N = gated ? rows / 2 : rows;
  if ((a[6] != Py_None && !fits(out, type, device, M, N)) ||
      (a[7] != Py_None && !(ws && fits(ws, ScalarType::Byte, device, ws->numel()))) || wants_grad(xs, wsc, out))
    Py_RETURN_NONE;
  Tensor y = out ? *out : make(*x, {M, N}, type);
  const auto call = [&](void* work, size_t bytes) {
    return (gated ? g_gated : g_linear)(M, D, N, static_cast<const int8_t*>(x->const_data_ptr()), static_cast<const float*>(xs->const_data_ptr()),
                                        static_cast<const int8_t*>(w->const_data_ptr()), static_cast<const float*>(wsc->const_data_ptr()),
                                        y.mutable_data_ptr(), dtype_code(type), work, bytes, stream(device));
  };
  paro_status st = ws ? call(ws->mutable_data_ptr(), size_t(ws->numel())) : call(nullptr, 0);
  if (st == PARO_EWORKSPACE && !ws) {  // nothing has been enqueued yet
    const size_t bytes = (gated ? g_gated_ws : g_linear_ws)(M, D, N);
    const Tensor work = make(*x, {int64_t(bytes)}, ScalarType::Byte);
    st = call(work.mutable_data_ptr(), bytes);
  }
  if (st != PARO_OK) Py_RETURN_NONE;
  wrote(a[6]);
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// (pack, x, address of the transform's handle or 0, its descriptor or None, q, scales) -> (q, scales)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 6) Py_RETURN_NONE;
  const Tensor* x = tensor(a[1]);
  int device, M, D;
  if (!starts(x, &device, &M, &D) || dtype_code(x->scalar_type()) < 0 || x->scalar_type() == ScalarType::Float) Py_RETURN_NONE;
  const auto* rot = static_cast<const paro_rotation*>(PyLong_AsVoidPtr(a[2]));
  if (!rot && PyErr_Occurred()) return nullptr;
  if (rot) {
    const Tensor* desc = tensor(a[3]);
    if (!desc || !desc->is_cuda() || desc->get_device() != device || rot->dev != desc->const_data_ptr()) Py_RETURN_NONE;
  }
  Tensor q, s;
  if (!output(a[4], *x, device, ScalarType::Char, {M, D}, &q) || !output(a[5], *x, device, ScalarType::Float, {M}, &s) ||
      wants_grad(a[0] == Py_True ? nullptr : x, &s))  // packed weights are constants: W may be a parameter
    Py_RETURN_NONE;
  const paro_status st = (a[0] == Py_True ? g_pack : g_quantize)(rot, M, D, dtype_code(x->scalar_type()), x->const_data_ptr(),
                                                                 static_cast<int8_t*>(q.mutable_data_ptr()),
                                                                 static_cast<float*>(s.mutable_data_ptr()), stream(device));
  if (st != PARO_OK) Py_RETURN_NONE;
  wrote(a[4]);
  wrote(a[5]);
  return Py_BuildValue("(NN)", THPVariable_Wrap(q), THPVariable_Wrap(s));
  END_HANDLE_TH_ERRORS
}

// (q, scales, out_dtype, out) -> x
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) Py_RETURN_NONE;
  const Tensor *q = tensor(a[0]), *s = tensor(a[1]);
  int device, M, D;
  ScalarType type;
  if (!starts(q, &device, &M, &D) || q->scalar_type() != ScalarType::Char || !fits(s, ScalarType::Float, device, M) ||
      !out_type(a[2], a[3] == Py_None ? nullptr : tensor(a[3]), &type))
    Py_RETURN_NONE;
  Tensor x;
  if (!output(a[3], *q, device, type, {M, D}, &x) || wants_grad(s, &x)) Py_RETURN_NONE;
  const paro_status st = g_dequantize(M, D, static_cast<const int8_t*>(q->const_data_ptr()), static_cast<const float*>(s->const_data_ptr()),
                                      x.mutable_data_ptr(), dtype_code(type), stream(device));
  if (st != PARO_OK) Py_RETURN_NONE;
  wrote(a[3]);
  return THPVariable_Wrap(x);
  END_HANDLE_TH_ERRORS
}

// (q8, x, gamma, eps, residual, residual_out, q or y, scales) -> (q, scales, h) or (y, h)
PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) Py_RETURN_NONE;
  const bool q8 = a[0] == Py_True, has = a[4] != Py_None;
  const Tensor *x = tensor(a[1]), *gamma = tensor(a[2]), *res = has ? tensor(a[4]) : nullptr;
  int device, M, D;
  if (!starts(x, &device, &M, &D) || dtype_code(x->scalar_type()) < 0 || x->scalar_type() == ScalarType::Float) Py_RETURN_NONE;
  const ScalarType type = x->scalar_type();
  if (!fits(gamma, type, device, D) || (has ? !fits(res, type, device, M, D) : a[5] != Py_None) || !PyFloat_Check(a[3]))
    Py_RETURN_NONE;
  const float eps = float(PyFloat_AS_DOUBLE(a[3]));
  Tensor h, q, s;
  if (!output(a[6], *x, device, q8 ? ScalarType::Char : type, {M, D}, &q) ||
      (q8 && !output(a[7], *x, device, ScalarType::Float, {M}, &s)) || (has && !output(a[5], *x, device, type, {M, D}, &h)) ||
      wants_grad(x, gamma, res, has ? &h : nullptr, &q, q8 ? &s : nullptr))
    Py_RETURN_NONE;
  void* const hp = has ? h.mutable_data_ptr() : nullptr;
  const void* const rp = has ? res->const_data_ptr() : nullptr;
  PyObject* const none = Py_None;
  if (q8) {
    if (g_rmsnorm_q8(M, D, dtype_code(type), x->const_data_ptr(), rp, gamma->const_data_ptr(), eps, hp,
                     static_cast<int8_t*>(q.mutable_data_ptr()), static_cast<float*>(s.mutable_data_ptr()), stream(device)) != PARO_OK)
      Py_RETURN_NONE;
    wrote(a[5]);
    wrote(a[6]);
    wrote(a[7]);
    if (!has) return Py_BuildValue("(NNO)", THPVariable_Wrap(q), THPVariable_Wrap(s), none);
    return Py_BuildValue("(NNN)", THPVariable_Wrap(q), THPVariable_Wrap(s), THPVariable_Wrap(h));
  }
  if (g_rmsnorm(M, D, dtype_code(type), x->const_data_ptr(), rp, gamma->const_data_ptr(), eps, hp, q.mutable_data_ptr(),
                stream(device)) != PARO_OK)
    Py_RETURN_NONE;
  wrote(a[5]);
  wrote(a[6]);
  if (!has) return Py_BuildValue("(NO)", THPVariable_Wrap(q), none);
  return Py_BuildValue("(NN)", THPVariable_Wrap(q), THPVariable_Wrap(h));
  END_HANDLE_TH_ERRORS
}

// The library's entry points, in this order.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9) {
    PyErr_SetString(PyExc_TypeError, "bind takes nine addresses");
    return nullptr;
  }
  void* p[9];
  for (int i = 0; i < 9; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point's address is zero");
      return nullptr;
    }
  }
  g_rmsnorm_q8 = reinterpret_cast<decltype(g_rmsnorm_q8)>(p[0]);
  g_rmsnorm = reinterpret_cast<decltype(g_rmsnorm)>(p[1]);
  g_quantize = reinterpret_cast<decltype(g_quantize)>(p[2]);
  g_pack = reinterpret_cast<decltype(g_pack)>(p[3]);
  g_dequantize = reinterpret_cast<decltype(g_dequantize)>(p[4]);
  g_linear = reinterpret_cast<decltype(g_linear)>(p[5]);
  g_gated = reinterpret_cast<decltype(g_gated)>(p[6]);
  g_linear_ws = reinterpret_cast<decltype(g_linear_ws)>(p[7]);
  g_gated_ws = reinterpret_cast<decltype(g_gated_ws)>(p[8]);
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear)), METH_FASTCALL, nullptr},
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantize)), METH_FASTCALL, nullptr},
    {"dequantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(dequantize)), METH_FASTCALL, nullptr},
    {"rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rmsnorm)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* const m = PyModule_Create(&kModule);
  // the torch whose headers this was compiled with: another's tensors may be laid out differently
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
