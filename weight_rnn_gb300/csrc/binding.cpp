// binding.cpp -- the Python calls of the block operators for the common case:
// plain CUDA tensors of the right types and shapes, outputs to be allocated,
// the current stream.  Checking, allocating and calling here takes about a
// third of what the same does in Python, which is what a small call costs.
// Whatever else comes (another stream, given outputs, a wrong argument, tensors on
// a device that is not the current one) gets
// NotImplemented, and block.py takes it from there: its checks say what is
// wrong.  A status other than DELTA_OK comes back as an int.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/delta.h"

namespace {

using at::Tensor;

// a plain CUDA tensor, else nullptr
const Tensor *tensor(PyObject *o) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const Tensor &t = THPVariable_Unpack(o);
  return t.defined() && t.is_cuda() && t.layout() == at::kStrided ? &t : nullptr;
}

// the library launches on the current device
bool here(int dev) { return c10::cuda::current_device() == dev; }

int code(at::ScalarType t) { return t == at::kBFloat16 ? DELTA_BF16 : t == at::kFloat ? DELTA_F32 : -1; }

// of the given type, shape and device, contiguous
bool whole(const Tensor *t, at::ScalarType dt, at::IntArrayRef shape, int dev) {
  return t && t->scalar_type() == dt && t->get_device() == dev && t->sizes() == shape && t->is_contiguous();
}
// the same with contiguous rows and any strides above them
bool rows(const Tensor *t, at::ScalarType dt, at::IntArrayRef shape, int dev) {
  return t && t->scalar_type() == dt && t->get_device() == dev && t->sizes() == shape &&
         (shape.back() <= 1 || t->stride(-1) == 1);
}
// an optional argument: None passes; `t` stays nullptr then
bool optional_whole(PyObject *o, const Tensor *&t, at::ScalarType dt, at::IntArrayRef shape, int dev) {
  if (o == Py_None) return true;
  t = tensor(o);
  return whole(t, dt, shape, dev);
}

Tensor empty(at::IntArrayRef shape, at::ScalarType dt, int dev) {
  return at::detail::empty_cuda(shape, dt, c10::Device(c10::DeviceType::CUDA, (c10::DeviceIndex)dev), std::nullopt);
}
CUstream_st *stream(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }
PyObject *wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }
template <typename... T>
PyObject *tuple(T... t) {
  PyObject *parts[] = {t...};
  constexpr int n = sizeof...(T);
  PyObject *r = PyTuple_New(n);
  for (int i = 0; i < n; ++i) PyTuple_SET_ITEM(r, i, parts[i]);
  return r;
}
bool truth(PyObject *o) { return PyObject_IsTrue(o) == 1; }
PyObject *none() { return Py_NewRef(Py_None); }
PyObject *other() { return Py_NewRef(Py_NotImplemented); }

// C++ exceptions (an allocation that fails) become Python's
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *, PyObject *const *args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (const std::exception &e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

constexpr int kScanBlock = 64;
bool fits(int64_t n) { return n >= 0 && n < (int64_t(1) << 31); }

// x, gate, h0, lengths, save_states, form
PyObject *scan_fwd(PyObject *const *a, Py_ssize_t n) {
  if (n != 6) return other();
  const Tensor *x = tensor(a[0]), *g = tensor(a[1]), *h0 = nullptr, *len = nullptr;
  const int form = (int)PyLong_AsLong(a[5]);
  if (!x || x->dim() != 3 || code(x->scalar_type()) < 0 || (form != 0 && form != 1)) return other();
  const int dev = x->get_device();
  const auto dt = x->scalar_type(), gt = form == DELTA_SCAN_LINEAR ? at::kFloat : dt;
  const int64_t B = x->size(0), T = x->size(1), D = x->size(2);
  if (!here(dev) || !fits(B) || !fits(T) || !fits(D) || !rows(x, dt, x->sizes(), dev) || !rows(g, gt, x->sizes(), dev) ||
      !optional_whole(a[2], h0, at::kFloat, {B, D}, dev) || !optional_whole(a[3], len, at::kInt, {B}, dev))
    return other();
  const bool save = truth(a[4]);
  Tensor out = empty({B, T, D}, dt, dev), hT = empty({B, D}, at::kFloat, dev), states;
  if (save) states = empty({B, (T + kScanBlock - 1) / kScanBlock, D}, at::kFloat, dev);
  const int st = delta_scan_fwd(ptr(x), ptr(g), static_cast<float *>(ptr(h0)), static_cast<int *>(ptr(len)),
                                out.data_ptr(), static_cast<float *>(hT.data_ptr()),
                                save ? static_cast<float *>(states.data_ptr()) : nullptr, (int)B, (int)T, (int)D,
                                x->stride(0), x->stride(1), g->stride(0), g->stride(1),
                                (delta_dtype)code(dt), (delta_scan_form)form, stream(dev));
  if (st != DELTA_OK) return PyLong_FromLong(st);
  return save ? tuple(wrap(out), wrap(hT), wrap(states)) : tuple(wrap(out), wrap(hT));
}

// x, gate, state, form
PyObject *scan_step(PyObject *const *a, Py_ssize_t n) {
  if (n != 4) return other();
  const Tensor *x = tensor(a[0]), *g = tensor(a[1]), *s = tensor(a[2]);
  const int form = (int)PyLong_AsLong(a[3]);
  if (!x || x->dim() != 2 || code(x->scalar_type()) < 0 || (form != 0 && form != 1)) return other();
  const int dev = x->get_device();
  const auto dt = x->scalar_type();
  if (!here(dev) || !fits(x->size(0)) || !fits(x->size(1)) || !rows(x, dt, x->sizes(), dev) ||
      !rows(g, form == DELTA_SCAN_LINEAR ? at::kFloat : dt, x->sizes(), dev) ||
      !whole(s, at::kFloat, x->sizes(), dev))
    return other();
  Tensor out = empty(x->sizes(), dt, dev);
  const int st = delta_scan_step(ptr(x), ptr(g), static_cast<float *>(ptr(s)), out.data_ptr(), (int)x->size(0),
                                 (int)x->size(1), x->stride(0), g->stride(0), (delta_dtype)code(dt),
                                 (delta_scan_form)form, stream(dev));
  return st == DELTA_OK ? wrap(out) : PyLong_FromLong(st);
}

// x, gate, states, dout, dhT, lengths, form
PyObject *scan_bwd(PyObject *const *a, Py_ssize_t n) {
  if (n != 7) return other();
  const Tensor *x = tensor(a[0]), *g = tensor(a[1]), *s = tensor(a[2]), *d = tensor(a[3]), *dh = nullptr,
               *len = nullptr;
  const int form = (int)PyLong_AsLong(a[6]);
  if (!x || x->dim() != 3 || code(x->scalar_type()) < 0 || (form != 0 && form != 1)) return other();
  const int dev = x->get_device();
  const auto dt = x->scalar_type(), gt = form == DELTA_SCAN_LINEAR ? at::kFloat : dt;
  const int64_t B = x->size(0), T = x->size(1), D = x->size(2);
  if (!here(dev) || !fits(B) || !fits(T) || !fits(D) || !rows(x, dt, x->sizes(), dev) || !rows(g, gt, x->sizes(), dev) ||
      !whole(s, at::kFloat, {B, (T + kScanBlock - 1) / kScanBlock, D}, dev) || !whole(d, dt, x->sizes(), dev) ||
      !optional_whole(a[4], dh, at::kFloat, {B, D}, dev) || !optional_whole(a[5], len, at::kInt, {B}, dev))
    return other();
  Tensor dx = empty({B, T, D}, dt, dev), dg = empty({B, T, D}, gt, dev), dh0 = empty({B, D}, at::kFloat, dev);
  const int st = delta_scan_bwd(ptr(x), ptr(g), static_cast<float *>(ptr(s)), static_cast<int *>(ptr(len)), ptr(d),
                                static_cast<float *>(ptr(dh)), dx.data_ptr(), dg.data_ptr(),
                                static_cast<float *>(dh0.data_ptr()), (int)B, (int)T, (int)D, x->stride(0),
                                x->stride(1), g->stride(0), g->stride(1), (delta_dtype)code(dt),
                                (delta_scan_form)form, stream(dev));
  return st == DELTA_OK ? tuple(wrap(dx), wrap(dg), wrap(dh0)) : PyLong_FromLong(st);
}

// [..., D] as rows: contiguous, or two axes with contiguous rows
bool as_rows(const Tensor *t, at::ScalarType dt, at::IntArrayRef shape, int dev, int64_t &ld) {
  if (!t || shape.empty() || t->scalar_type() != dt || t->get_device() != dev || t->sizes() != shape) return false;
  ld = shape.back();
  if (t->is_contiguous()) return true;
  if (t->dim() != 2 || (shape[1] > 1 && t->stride(1) != 1)) return false;
  ld = t->stride(0);
  return true;
}

// x, weight, residual, eps, quant: (y, sum, rstd) or (y, scale, sum)
PyObject *norm_fwd(PyObject *const *a, Py_ssize_t n) {
  if (n != 5) return other();
  const Tensor *x = tensor(a[0]), *w = tensor(a[1]), *r = a[2] == Py_None ? nullptr : tensor(a[2]);
  if (!x || x->dim() < 1 || code(x->scalar_type()) < 0 || !w || code(w->scalar_type()) < 0 || !PyFloat_Check(a[3]))
    return other();
  const int dev = x->get_device();
  const auto dt = x->scalar_type();
  const auto shape = x->sizes();
  const int64_t D = shape.back();
  int64_t ldx = 0, ldr = D;
  if (!here(dev) || !fits(D) || D == 0 || !as_rows(x, dt, shape, dev, ldx) || !whole(w, w->scalar_type(), {D}, dev) ||
      (a[2] != Py_None && !as_rows(r, dt, shape, dev, ldr)))
    return other();
  const int64_t count = x->numel() / D;
  const bool quant = truth(a[4]);
  Tensor y = empty(shape, quant ? at::kFloat8_e4m3fn : dt, dev), per = empty(shape.slice(0, shape.size() - 1), at::kFloat, dev);
  Tensor sum;
  if (r) sum = empty(shape, dt, dev);
  void *s = r ? sum.data_ptr() : nullptr;
  const float eps = (float)PyFloat_AS_DOUBLE(a[3]);
  const auto dc = (delta_dtype)code(dt), wc = (delta_dtype)code(w->scalar_type());
  const int st = quant ? delta_add_rmsnorm_quant(ptr(x), ptr(r), ptr(w), y.data_ptr(), static_cast<float *>(per.data_ptr()),
                                                 s, count, (int)D, ldx, ldr, eps, dc, wc, stream(dev))
                       : delta_add_rmsnorm_fwd(ptr(x), ptr(r), ptr(w), y.data_ptr(), s, static_cast<float *>(per.data_ptr()),
                                               count, (int)D, ldx, ldr, eps, dc, wc, stream(dev));
  if (st != DELTA_OK) return PyLong_FromLong(st);
  PyObject *ps = r ? wrap(sum) : Py_NewRef(a[0]);
  return quant ? tuple(wrap(y), wrap(per), ps) : tuple(wrap(y), ps, wrap(per));
}

// dy, sum, weight, rstd, dsum
PyObject *norm_bwd(PyObject *const *a, Py_ssize_t n) {
  if (n != 5) return other();
  const Tensor *dy = tensor(a[0]), *sum = tensor(a[1]), *w = tensor(a[2]), *r = tensor(a[3]), *ds = nullptr;
  if (!dy || dy->dim() < 1 || code(dy->scalar_type()) < 0 || !w || code(w->scalar_type()) < 0) return other();
  const int dev = dy->get_device();
  const auto dt = dy->scalar_type();
  const auto shape = dy->sizes();
  const int64_t D = shape.back();
  if (!here(dev) || !fits(D) || !whole(dy, dt, shape, dev) || !whole(sum, dt, shape, dev) || !whole(w, w->scalar_type(), {D}, dev) ||
      !whole(r, at::kFloat, shape.slice(0, shape.size() - 1), dev) || !optional_whole(a[4], ds, dt, shape, dev))
    return other();
  Tensor dx = empty(shape, dt, dev), dw = empty({D}, at::kFloat, dev);
  const int st = delta_add_rmsnorm_bwd(ptr(dy), ptr(sum), ptr(w), static_cast<float *>(ptr(r)), ptr(ds), dx.data_ptr(),
                                       static_cast<float *>(dw.data_ptr()), D > 0 ? dy->numel() / D : 0, (int)D,
                                       (delta_dtype)code(dt), (delta_dtype)code(w->scalar_type()), stream(dev));
  return st == DELTA_OK ? tuple(wrap(dx), wrap(dw)) : PyLong_FromLong(st);
}

// The operands that the linear calls share.
struct Linear {
  const Tensor *x = nullptr, *w = nullptr, *bias = nullptr, *res = nullptr;
  int dev = 0;
  int64_t M = 1, N = 0, K = 0, ldx = 0, ldw = 0, ldr = 0;
  c10::SmallVector<int64_t, 6> shape;  // of the result
  delta_dtype bcode = DELTA_F32;

  bool take(PyObject *px, PyObject *pw, at::ScalarType dt) {
    x = tensor(px);
    w = tensor(pw);
    if (!x || !w || x->dim() < 1 || w->dim() != 2 || x->scalar_type() != dt) return false;
    dev = x->get_device();
    N = w->size(0);
    K = w->size(1);
    if (!here(dev) || !fits(N) || !fits(K) || x->size(-1) != K || !rows(w, dt, w->sizes(), dev) ||
        !as_rows(x, dt, x->sizes(), dev, ldx))
      return false;
    ldw = w->stride(0);
    shape.assign(x->sizes().begin(), x->sizes().end());
    shape.back() = N;
    for (size_t i = 0; i + 1 < shape.size(); ++i) M *= shape[i];
    ldr = N;
    return fits(M);
  }
  bool extras(PyObject *pb, PyObject *pr, at::ScalarType odt) {
    if (pb != Py_None) {
      bias = tensor(pb);
      if (!bias || code(bias->scalar_type()) < 0 || !whole(bias, bias->scalar_type(), {N}, dev)) return false;
      bcode = (delta_dtype)code(bias->scalar_type());
    }
    if (pr == Py_None) return true;
    res = tensor(pr);
    return as_rows(res, odt, shape, dev, ldr);
  }
};

// x, w, bias, residual, act, save_pre
PyObject *linear_fwd(PyObject *const *a, Py_ssize_t n) {
  if (n != 6) return other();
  const Tensor *x = tensor(a[0]);
  const int act = (int)PyLong_AsLong(a[4]);
  Linear l;
  if (!x || code(x->scalar_type()) < 0 || act < 0 || !l.take(a[0], a[1], x->scalar_type()) ||
      !l.extras(a[2], a[3], x->scalar_type()))
    return other();
  const auto dt = x->scalar_type();
  const bool save = truth(a[5]);
  Tensor out = empty(l.shape, dt, l.dev), pre;
  if (save) pre = empty(l.shape, dt, l.dev);
  const int st = delta_linear_fwd(ptr(x), ptr(l.w), ptr(l.bias), ptr(l.res), out.data_ptr(),
                                  save ? pre.data_ptr() : nullptr, (int)l.M, (int)l.N, (int)l.K, l.ldx, l.ldw, l.ldr,
                                  (delta_act)act, (delta_dtype)code(dt), l.bcode, stream(l.dev));
  if (st != DELTA_OK) return PyLong_FromLong(st);
  return save ? tuple(wrap(out), wrap(pre)) : wrap(out);
}

// x, x_scale, w, w_scale, bias, residual, act
PyObject *linear_quant(PyObject *const *a, Py_ssize_t n) {
  if (n != 7) return other();
  const Tensor *sx = tensor(a[1]), *sw = tensor(a[3]);
  const int act = (int)PyLong_AsLong(a[6]);
  Linear l;
  if (act < 0 || !l.take(a[0], a[2], at::kFloat8_e4m3fn) || !l.extras(a[4], a[5], at::kBFloat16) ||
      !whole(sx, at::kFloat, l.x->sizes().slice(0, l.x->dim() - 1), l.dev) || !whole(sw, at::kFloat, {l.N}, l.dev))
    return other();
  Tensor out = empty(l.shape, at::kBFloat16, l.dev);
  const int st = delta_linear_quant(ptr(l.x), static_cast<float *>(ptr(sx)), ptr(l.w), static_cast<float *>(ptr(sw)),
                                    ptr(l.bias), ptr(l.res), out.data_ptr(), (int)l.M, (int)l.N, (int)l.K, l.ldx, l.ldw,
                                    l.ldr, (delta_act)act, l.bcode, stream(l.dev));
  return st == DELTA_OK ? wrap(out) : PyLong_FromLong(st);
}

// x, w, dout, pre, act, want_dx, want_dw, want_dbias
PyObject *linear_bwd(PyObject *const *a, Py_ssize_t n) {
  if (n != 8) return other();
  const Tensor *x = tensor(a[0]), *d = tensor(a[2]), *pre = nullptr;
  const int act = (int)PyLong_AsLong(a[4]);
  Linear l;
  if (!x || code(x->scalar_type()) < 0 || act < 0 || !l.take(a[0], a[1], x->scalar_type())) return other();
  const auto dt = x->scalar_type();
  if (!whole(d, dt, l.shape, l.dev) || !optional_whole(a[3], pre, dt, l.shape, l.dev) || (act != 0 && !pre))
    return other();
  Tensor dx, dw, db;
  if (truth(a[5])) dx = empty(x->sizes(), dt, l.dev);
  if (truth(a[6])) dw = empty({l.N, l.K}, dt, l.dev);
  if (truth(a[7])) db = empty({l.N}, at::kFloat, l.dev);
  const auto at_ = [](Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; };
  const int st = delta_linear_bwd(ptr(x), ptr(l.w), ptr(d), ptr(pre), at_(dx), at_(dw), static_cast<float *>(at_(db)),
                                  (int)l.M, (int)l.N, (int)l.K, l.ldx, l.ldw, (delta_act)act, (delta_dtype)code(dt),
                                  stream(l.dev));
  if (st != DELTA_OK) return PyLong_FromLong(st);
  const auto give = [](Tensor &t) { return t.defined() ? wrap(t) : none(); };
  return tuple(give(dx), give(dw), give(db));
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))guarded<name>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(scan_fwd),   FAST(scan_step),    FAST(scan_bwd),   FAST(norm_fwd), FAST(norm_bwd),
                         FAST(linear_fwd), FAST(linear_quant), FAST(linear_bwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", "block operators, the common case", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast(void) { return PyModule_Create(&module); }
