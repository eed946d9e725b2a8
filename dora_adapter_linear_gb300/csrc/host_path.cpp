// The host side of calls whose kernels take a few microseconds: operand checks, output allocation and the
// call of the C ABI in one go.  In Python they take longer than the kernels (norm of one token: 21 us, here 7.3,
// 2.4 on the device).  A function returns None for anything but well-formed operands: the Python
// wrapper then names the fault, or serves what is rare.  A status other than LORA_OK comes back as an int.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/lora_gb300.h"

namespace {

using at::Tensor;

// entry points of the library that the binding has loaded
decltype(&block_norm_fwd) norm_fwd_call = nullptr;
decltype(&block_norm_bwd) norm_bwd_call = nullptr;
decltype(&rotary_fwd) rotary_fwd_call = nullptr;
decltype(&rotary_bwd) rotary_bwd_call = nullptr;

// a tensor argument: absent (None), a tensor, or something else
struct Arg {
  const Tensor* t = nullptr;
  bool ok = true;
  explicit Arg(PyObject* o) {
    if (o == Py_None) return;
    if (THPVariable_Check(o)) t = &THPVariable_Unpack(o);
    else ok = false;
  }
  explicit operator bool() const { return t != nullptr; }
  const Tensor& operator*() const { return *t; }
  void* ptr() const { return t ? t->data_ptr() : nullptr; }
};

int dtype_of(const Tensor& x) {
  return x.scalar_type() == at::kBFloat16 ? LORA_BF16 : x.scalar_type() == at::kFloat ? LORA_F32 : -1;
}
// the calls run on the current device's current stream
bool here(const Tensor& x) { return x.is_cuda() && x.device().index() == c10::cuda::current_device(); }
bool strided(const Tensor& t) { return t.layout() == at::kStrided; }
bool same_kind(const Tensor& t, const Tensor& x) {
  return strided(t) && t.scalar_type() == x.scalar_type() && t.device() == x.device();
}
bool dense(const Tensor& t, const Tensor& x, at::ScalarType type, at::IntArrayRef sizes) {
  return strided(t) && t.scalar_type() == type && t.device() == x.device() && t.sizes() == sizes && t.is_contiguous();
}
// the row stride of a [M, D] operand with consecutive elements in a row, or -1
int64_t row_stride(const Tensor& t, const Tensor& x) {
  if (!same_kind(t, x) || t.sizes() != x.sizes() || t.stride(1) != 1) return -1;
  if (t.size(0) <= 1) return t.size(1);
  return t.stride(0) >= t.size(1) ? t.stride(0) : -1;
}
// a new tensor next to x, without the dispatcher's way to the same function (0.5 us a tensor)
Tensor fresh(const Tensor& x, at::IntArrayRef sizes, at::ScalarType type) {
  return at::detail::empty_cuda(sizes, type, x.device(), std::nullopt);
}
Tensor fresh(const Tensor& x, at::IntArrayRef sizes) { return fresh(x, sizes, x.scalar_type()); }
// Other Python threads run while this one allocates and launches: either may have to wait for the device.
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
// A kernel has written t: autograd notices if it had kept t for a backward.
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void* stream() { return c10::cuda::getCurrentCUDAStream().stream(); }
// the truth of a flag; false: it has none, and the error is set
bool truth(PyObject* o, bool* value) {
  const int v = PyObject_IsTrue(o);
  *value = v == 1;
  return v >= 0;
}
PyObject* not_here() { Py_RETURN_NONE; }
PyObject* wrap(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
template <typename... Ts>
PyObject* tuple_of(const Ts&... ts) {
  PyObject* items[] = {wrap(ts)...};
  PyObject* r = PyTuple_New(sizeof...(Ts));
  for (size_t i = 0; i < sizeof...(Ts); ++i) {
    if (r && items[i]) PyTuple_SET_ITEM(r, i, items[i]);
    else if (items[i]) Py_DECREF(items[i]);
  }
  if (r)
    for (PyObject* o : items)
      if (!o) {
        Py_DECREF(r);
        return nullptr;
      }
  return r;
}

// The shape both norm calls share; false: not for here.
bool norm_shape(lora_norm_shape* sh, const Tensor& x, const Arg& w_pre, const Arg& w_post, const Arg& gate,
                PyObject* rows_per_gate, double alpha, double eps, double off, bool post) {
  if (!here(x) || !strided(x) || x.dim() != 2 || dtype_of(x) < 0) return false;
  const int64_t M = x.size(0), D = x.size(1);
  if (M < 1 || D < 1) return false;
  if (w_pre && !dense(*w_pre, x, x.scalar_type(), {D})) return false;
  if (w_post && (!post || !dense(*w_post, x, x.scalar_type(), {D}))) return false;
  int64_t per = 0;
  if (gate) {
    if ((*gate).dim() != 2) return false;
    const int64_t G = (*gate).size(0);
    if (G < 1 || !dense(*gate, x, x.scalar_type(), {G, D})) return false;
    if (rows_per_gate == Py_None) {
      if (M % G) return false;
      per = M / G;
    } else {
      per = PyLong_AsLongLong(rows_per_gate);
      if (per == -1 && PyErr_Occurred()) PyErr_Clear();
    }
    if (per < 1 || G != (M - 1) / per + 1) return false;
  }
  *sh = lora_norm_shape{M, D, per, D, D, D, D, (float)alpha, (float)eps, (float)off, post ? 1 : 0, dtype_of(x)};
  return true;
}

// (X, Y, w_pre, w_post, gate, rows_per_gate, alpha, eps, w_offset, pre_norm, post_norm)
PyObject* py_norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 11) return not_here();
  const Arg X(a[0]), Y(a[1]), w_pre(a[2]), w_post(a[3]), gate(a[4]);
  const double alpha = PyFloat_AsDouble(a[6]), eps = PyFloat_AsDouble(a[7]), off = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred()) return nullptr;
  bool pre, post;
  if (!truth(a[9], &pre) || !truth(a[10], &post)) return nullptr;
  lora_norm_shape sh;
  if (!X || !Y.ok || !w_pre.ok || !w_post.ok || !gate.ok || (!Y && (gate || post || !pre)) || (w_pre && !pre) ||
      !norm_shape(&sh, *X, w_pre, w_post, gate, a[5], alpha, eps, off, post))
    return not_here();
  if ((sh.ldx = row_stride(*X, *X)) < 0 || (Y && (sh.ldy = row_stride(*Y, *X)) < 0)) return not_here();
  Tensor z, h, r_pre, r_post;
  int e;
  {
    const Unlocked unlocked;
    if (Y) z = fresh(*X, {sh.M, sh.D});
    if (pre) h = fresh(*X, {sh.M, sh.D}), r_pre = fresh(*X, {sh.M}, at::kFloat);
    if (post) r_post = fresh(*X, {sh.M}, at::kFloat);
    const auto p = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    e = norm_fwd_call(&sh, X.ptr(), Y.ptr(), w_pre.ptr(), w_post.ptr(), gate.ptr(), p(z), p(h),
                      static_cast<float*>(p(r_pre)), static_cast<float*>(p(r_post)), stream());
  }
  if (e != LORA_OK) return PyLong_FromLong(e);
  return tuple_of(Y ? z : *X, h, r_pre, r_post);
  END_HANDLE_TH_ERRORS
}

// (Xout, Y, r_pre, r_post, dH, dXout, w_pre, w_post, gate, rows_per_gate, alpha, w_offset, post_norm, need_dx,
//  need_dw, need_dgate, workspace)
PyObject* py_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 17) return not_here();
  const Arg X(a[0]), Y(a[1]), r_pre(a[2]), r_post(a[3]), dH(a[4]), dZ(a[5]), w_pre(a[6]), w_post(a[7]), gate(a[8]),
      ws(a[16]);
  const double alpha = PyFloat_AsDouble(a[10]), off = PyFloat_AsDouble(a[11]);
  if (PyErr_Occurred()) return nullptr;
  bool post, need_dx, need_dw, need_dgate;
  if (!truth(a[12], &post) || !truth(a[13], &need_dx) || !truth(a[14], &need_dw) || !truth(a[15], &need_dgate)) return nullptr;
  for (const Arg* t : {&Y, &r_pre, &r_post, &dH, &dZ, &w_pre, &w_post, &gate})
    if (!t->ok) return not_here();
  lora_norm_shape sh;
  if (!X || !ws || (!dH && !dZ) || (!Y && (gate || post)) || (dH && !r_pre) || (post && !r_post) ||
      !norm_shape(&sh, *X, w_pre, w_post, gate, a[9], alpha, 1.0, off, post))
    return not_here();
  for (const Arg* r : {&r_pre, &r_post})
    if (*r && !dense(**r, *X, at::kFloat, {sh.M})) return not_here();
  if ((sh.ldx = row_stride(*X, *X)) < 0 || (Y && (sh.ldy = row_stride(*Y, *X)) < 0) ||
      (dH && (sh.lddh = row_stride(*dH, *X)) < 0) || (dZ && (sh.lddz = row_stride(*dZ, *X)) < 0))
    return not_here();
  Tensor dX, dY, dw_pre, dw_post, dgate;
  int e;
  {
    const Unlocked unlocked;
    if (need_dx) dX = fresh(*X, {sh.M, sh.D});
    if (Y) dY = fresh(*X, {sh.M, sh.D});
    if (need_dw && w_pre) dw_pre = fresh(*X, {sh.D});
    if (need_dw && w_post) dw_post = fresh(*X, {sh.D});
    if (need_dgate && gate) dgate = fresh(*X, (*gate).sizes());
    const auto p = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    e = norm_bwd_call(&sh, X.ptr(), Y.ptr(), w_pre.ptr(), w_post.ptr(), gate.ptr(),
                      static_cast<const float*>(r_pre.ptr()), static_cast<const float*>(r_post.ptr()), dH.ptr(),
                      dZ.ptr(), p(dX), p(dY), p(dw_pre), p(dw_post), p(dgate), ws.ptr(), (*ws).nbytes(), stream());
  }
  if (e != LORA_OK) return PyLong_FromLong(e);
  return tuple_of(dX, dY, dw_pre, dw_post, dgate);
  END_HANDLE_TH_ERRORS
}

// (inverse, X, pos, freq, rot_dim, scale, layout, out)
PyObject* py_rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) return not_here();
  const Arg X(a[1]), pos(a[2]), freq(a[3]), out(a[7]);
  if (!X || !pos || !freq || !out.ok) return not_here();
  const Tensor &x = *X, &p = *pos;
  const int64_t rot = PyLong_AsLongLong(a[4]);
  const double scale = PyFloat_AsDouble(a[5]);
  const long layout = PyLong_AsLong(a[6]);
  if (PyErr_Occurred()) return nullptr;
  if (!here(x) || !strided(x) || x.dim() != 3 || dtype_of(x) < 0 || x.size(0) < 1 || x.size(1) < 1 || x.stride(2) != 1)
    return not_here();
  const bool wide = p.scalar_type() == at::kLong;
  if (!(wide || p.scalar_type() == at::kInt) || !dense(p, x, p.scalar_type(), {x.size(0)}) || rot > x.size(2) ||
      !dense(*freq, x, at::kLong, {rot / 2}))
    return not_here();
  if (out && (!same_kind(*out, x) || (*out).sizes() != x.sizes() || (*out).stride(2) != 1 ||
              ((*out).requires_grad() && at::GradMode::is_enabled())))
    return not_here();
  bool inverse;
  if (!truth(a[0], &inverse)) return nullptr;
  const auto call = inverse ? rotary_bwd_call : rotary_fwd_call;
  Tensor y;
  int e;
  {
    const Unlocked unlocked;
    y = out ? *out : fresh(x, x.sizes());
    const lora_rotary_shape sh{x.size(0), x.size(1), x.size(2), rot, x.stride(0), x.stride(1), y.stride(0), y.stride(1),
                               (float)scale, (int32_t)layout, wide ? 64 : 32, dtype_of(x)};
    e = call(&sh, x.data_ptr(), p.data_ptr(), static_cast<const uint64_t*>((*freq).data_ptr()), y.data_ptr(), stream());
  }
  if (e != LORA_OK) return PyLong_FromLong(e);
  if (!out) return THPVariable_Wrap(y);
  written(y);
  Py_INCREF(a[7]);
  return a[7];
  END_HANDLE_TH_ERRORS
}

// (gradients, tensors): the gradients' addresses as bytes, 0 for a None, each like its tensor
PyObject* py_pointers(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 2 || !(PyList_Check(a[0]) || PyTuple_Check(a[0])) || !PyList_Check(a[1])) return not_here();
  const Py_ssize_t count = PySequence_Fast_GET_SIZE(a[0]);
  if (count != PyList_GET_SIZE(a[1])) return not_here();
  PyObject* bytes = PyBytes_FromStringAndSize(nullptr, count * (Py_ssize_t)sizeof(uint64_t));
  if (!bytes) return nullptr;
  char* to = PyBytes_AS_STRING(bytes);
  PyObject** grads = PySequence_Fast_ITEMS(a[0]);
  for (Py_ssize_t i = 0; i < count; ++i) {
    const Arg g(grads[i]), p(PyList_GET_ITEM(a[1], i));
    if (!g.ok || !p || (g && !dense(*g, *p, (*p).scalar_type(), (*p).sizes()))) {
      Py_DECREF(bytes);
      return not_here();
    }
    const uint64_t at = reinterpret_cast<uint64_t>(g.ptr());
    memcpy(to + i * sizeof at, &at, sizeof at);
  }
  return bytes;
  END_HANDLE_TH_ERRORS
}

// (tensors, addresses): the tensors whose gradients' addresses, from pointers(), are not 0 have been written
PyObject* py_written(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 2 || !PyList_Check(a[0]) || !PyBytes_Check(a[1])) return not_here();
  const Py_ssize_t count = PyList_GET_SIZE(a[0]);
  if (PyBytes_GET_SIZE(a[1]) != count * (Py_ssize_t)sizeof(uint64_t)) return not_here();
  for (Py_ssize_t i = 0; i < count; ++i) {
    uint64_t at;
    memcpy(&at, PyBytes_AS_STRING(a[1]) + i * sizeof at, sizeof at);
    const Arg t(PyList_GET_ITEM(a[0], i));
    if (at && t) written(*t);
  }
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (tensor): a 0-d fp32 tensor next to it whose storage holds two values, the second behind the one it shows
PyObject* py_pair(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 1) return not_here();
  const Arg like(a[0]);
  if (!like || !(*like).is_cuda()) return not_here();
  Tensor t;
  {
    const Unlocked unlocked;
    t = fresh(*like, {2}, at::kFloat);
  }
  t.unsafeGetTensorImpl()->set_sizes_contiguous({});
  return THPVariable_Wrap(t);
  END_HANDLE_TH_ERRORS
}

// (block_norm_fwd, block_norm_bwd, rotary_fwd, rotary_bwd): addresses in the loaded library
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* at[4];
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "four addresses");
    return nullptr;
  }
  for (int i = 0; i < 4; ++i)
    if (!(at[i] = PyLong_AsVoidPtr(a[i]))) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is zero");
      return nullptr;
    }
  norm_fwd_call = reinterpret_cast<decltype(norm_fwd_call)>(at[0]);
  norm_bwd_call = reinterpret_cast<decltype(norm_bwd_call)>(at[1]);
  rotary_fwd_call = reinterpret_cast<decltype(rotary_fwd_call)>(at[2]);
  rotary_bwd_call = reinterpret_cast<decltype(rotary_bwd_call)>(at[3]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", FAST(py_bind), "take the library's entry points"},
                         {"block_norm_fwd", FAST(py_norm_fwd), "ops.block_norm_fwd"},
                         {"block_norm_bwd", FAST(py_norm_bwd), "ops.block_norm_bwd"},
                         {"rotary", FAST(py_rotary), "ops.rotary_fwd and rotary_bwd"},
                         {"pair", FAST(py_pair), "an optimiser's norm and factor"},
                         {"pointers", FAST(py_pointers), "addresses of an optimiser's gradients"},
                         {"written", FAST(py_written), "an optimiser's tensors after its step"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host", "host side of short calls", -1, methods, nullptr, nullptr, nullptr,
                      nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host() { return PyModule_Create(&module); }
