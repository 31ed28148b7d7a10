// Python extension module _tensors: what the helpers on torch tensors do per call, where Python would
// take longer than the GPU. addresses(): a list of tensors, checked (reading five attributes of 200
// tensors from Python takes 45 us, this 3 us). written(): their version counters moved (torch's own call takes
// 8 us for 200, this 1.2). linear() and linear_backward(): the checks, outputs and
// workspace of one call of the layer and the call itself (7.6 and 14.7 us from Python, 3.7 and
// 8.0 here; a small layer takes the GPU 4 us). Host code only; built against torch's headers, resolved
// against the torch that the process has imported; the C entry points come in by bind().
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

// addresses(tensors: list, numel: address of int64[n], out: address of uint64[n], n, device: int) -> -1, or
// the position of the first tensor that is not a contiguous strided tensor of numel[i] elements on GPU
// `device` with the first tensor's type.
PyObject* addresses(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 5 || !PyList_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "addresses(list, numel, out, n, device)");
    return nullptr;
  }
  const int64_t* numel = static_cast<const int64_t*>(PyLong_AsVoidPtr(args[1]));
  uint64_t* out = static_cast<uint64_t*>(PyLong_AsVoidPtr(args[2]));
  const Py_ssize_t n = PyLong_AsSsize_t(args[3]);
  const long device = PyLong_AsLong(args[4]);
  if (PyErr_Occurred()) return nullptr;
  if (PyList_GET_SIZE(args[0]) != n) return PyLong_FromSsize_t(0);
  c10::ScalarType type{};
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = PyList_GET_ITEM(args[0], i);
    if (!THPVariable_Check(o)) return PyLong_FromSsize_t(i);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (i == 0) type = t.scalar_type();
    if (!t.is_cuda() || t.layout() != c10::kStrided || t.get_device() != device || t.scalar_type() != type ||
        t.numel() != numel[i] || !t.is_contiguous())
      return PyLong_FromSsize_t(i);
    out[i] = reinterpret_cast<uint64_t>(t.data_ptr());
  }
  return PyLong_FromSsize_t(-1);
}

// written(tensors: list): tells autograd that the tensors have been written in place.
PyObject* written(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 1 || !PyList_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "written(list)");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < PyList_GET_SIZE(args[0]); ++i) {
    PyObject* o = PyList_GET_ITEM(args[0], i);
    if (!THPVariable_Check(o)) {
      PyErr_SetString(PyExc_TypeError, "written(list of tensors)");
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();  // tensors of inference mode have no counter
  }
  Py_RETURN_NONE;
}

// The entry points as include/xtvxy.h declares them, element pointers untyped; one per element type.
typedef int (*LinearSize)(int64_t, int64_t, int64_t, int, size_t*);
typedef int (*Linear)(int64_t, int64_t, int64_t, const void*, int64_t, const void*, int64_t, const float*, const void*,
                      int64_t, int, void*, int64_t, void*, int64_t, void*, size_t, void*);
typedef int (*BackwardSize)(int64_t, int64_t, int64_t, int, int, size_t*);
typedef int (*Backward)(int64_t, int64_t, int64_t, const void*, int64_t, const void*, int64_t, const void*, int64_t,
                        const void*, int64_t, int, void*, int64_t, void*, int64_t, float*, void*, size_t, void*);
struct Entries {
  LinearSize linear_size;
  Linear linear;
  BackwardSize backward_size;
  Backward backward;
} entries[3];  // f32, bf16, f16
bool bound = false;

// bind(addresses of the 3 x 4 entry points)
PyObject* bind(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 12) {
    PyErr_SetString(PyExc_TypeError, "bind takes 12 addresses");
    return nullptr;
  }
  for (int t = 0; t < 3; ++t) {
    entries[t].linear_size = reinterpret_cast<LinearSize>(PyLong_AsVoidPtr(args[4 * t]));
    entries[t].linear = reinterpret_cast<Linear>(PyLong_AsVoidPtr(args[4 * t + 1]));
    entries[t].backward_size = reinterpret_cast<BackwardSize>(PyLong_AsVoidPtr(args[4 * t + 2]));
    entries[t].backward = reinterpret_cast<Backward>(PyLong_AsVoidPtr(args[4 * t + 3]));
  }
  if (PyErr_Occurred()) return nullptr;
  bound = true;
  Py_RETURN_NONE;
}

// A call whose arguments are anything but right and usual ends with None: the caller's own checks then
// say what is wrong, or make the call.
struct Unusual {};

struct Call {
  c10::ScalarType type;
  int64_t device;
  int element = -1, es = 4;

  explicit Call(const at::Tensor& x, int64_t current) : type(x.scalar_type()), device(current) {
    if (type == at::kFloat) element = 0;
    else if (type == at::kBFloat16) element = 1;
    else if (type == at::kHalf) element = 2;
    if (element < 0 || !bound) throw Unusual{};
    es = element == 0 ? 4 : 2;
  }
  void on_device(const at::Tensor& t, c10::ScalarType of) const {
    if (!t.is_cuda() || t.layout() != c10::kStrided || t.get_device() != device || t.scalar_type() != of) throw Unusual{};
  }
  // The row stride of a rows x cols matrix.
  int64_t pitch(const at::Tensor& t, int64_t rows, int64_t cols) const {
    on_device(t, type);
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || (t.stride(1) != 1 && cols > 1)) throw Unusual{};
    if (rows <= 1) return cols > 0 ? cols : 1;
    const int64_t s = t.stride(0);
    if (s < cols || s < 1) throw Unusual{};
    return s;
  }
  float* vector(const at::Tensor& t, int64_t n) const {
    on_device(t, at::kFloat);
    if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1)) throw Unusual{};
    return static_cast<float*>(t.data_ptr());
  }
  bool aligned(const void* p, int64_t ld) const {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0 && ld * es <= 4 << 20;
  }
};

const at::Tensor* tensor_or_none(PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Unusual{};
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o) {
  const at::Tensor* t = tensor_or_none(o);
  if (!t) throw Unusual{};
  return *t;
}
int64_t number(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Unusual{};
  }
  return v;
}

struct Workspace {
  at::Tensor made;
  void* p = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* given, size_t need, const at::Tensor& like, const Call& c) {
    if (const at::Tensor* t = tensor_or_none(given)) {
      if (!t->is_cuda() || t->get_device() != c.device || !t->is_contiguous()) throw Unusual{};
      p = t->data_ptr();
      bytes = t->nbytes();
    } else if (need > 0) {
      made = at::empty({(int64_t)need}, like.options().dtype(at::kByte));
      p = made.data_ptr();
      bytes = need;
    }
  }
};

PyObject* wrapped(const at::Tensor& t, PyObject* given) {
  if (given == Py_None) return THPVariable_Wrap(t);
  Py_INCREF(given);
  return given;
}

// linear(X, W, bias, residual, activation, save_pre, out, pre, workspace, device, stream) -> out or (out, pre);
// a number: the entry point's error; None: left to the caller.
PyObject* linear(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 11) throw Unusual{};
  const at::Tensor &X = tensor(args[0]), &W = tensor(args[1]);
  const int64_t act = number(args[4]);
  if (X.dim() != 2 || W.dim() != 2 || act < 0) throw Unusual{};
  const Call c(X, number(args[9]));
  void* stream = reinterpret_cast<void*>(number(args[10]));
  const int64_t m = X.size(0), k = X.size(1), n = W.size(0);
  const int64_t ldx = c.pitch(X, m, k), ldw = c.pitch(W, n, k);
  const at::Tensor *bias = tensor_or_none(args[2]), *residual = tensor_or_none(args[3]), *out = tensor_or_none(args[6]),
                   *pre = tensor_or_none(args[7]);
  int64_t ldr = n > 0 ? n : 1, ldo = ldr, ldp = ldr;
  const float* b = bias ? c.vector(*bias, n) : nullptr;
  if (residual) ldr = c.pitch(*residual, m, n);
  if (out) ldo = c.pitch(*out, m, n);
  if (pre) ldp = c.pitch(*pre, m, n);
  const int save = PyObject_IsTrue(args[5]);
  if (save < 0) {
    PyErr_Clear();
    throw Unusual{};
  }
  const void *xp = X.data_ptr(), *wp = W.data_ptr();
  const Entries& e = entries[c.element];
  size_t need = 0;
  int status = e.linear_size(m, k, n, c.aligned(xp, ldx) && c.aligned(wp, ldw), &need);
  if (status) return PyLong_FromLong(status);
  at::Tensor made_out, made_pre;
  if (!out) out = &(made_out = at::empty({m, n}, X.options()));
  if (!pre && save) pre = &(made_pre = at::empty({m, n}, X.options()));
  const Workspace ws(args[8], need, X, c);
  void *op = out->data_ptr(), *pp = pre ? pre->data_ptr() : nullptr, *rp = residual ? residual->data_ptr() : nullptr;
  Py_BEGIN_ALLOW_THREADS
  status = e.linear(m, k, n, xp, ldx, wp, ldw, b, rp, ldr, (int)act, op, ldo, pp, ldp, ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  if (status) return PyLong_FromLong(status);
  PyObject* o = wrapped(made_out, args[6]);
  if (!pre || !o) return o;
  PyObject* p = wrapped(made_pre, args[7]);
  PyObject* both = p ? PyTuple_Pack(2, o, p) : nullptr;
  Py_DECREF(o);
  Py_XDECREF(p);
  return both;
}

// linear_backward(G, X, W, pre, activation, need_dX, need_dW, need_db, dX, dW, db, workspace, device, stream) -> (dX,
// dW, db); a number or None as above.
PyObject* linear_backward(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 14) throw Unusual{};
  const at::Tensor &G = tensor(args[0]), &X = tensor(args[1]), &W = tensor(args[2]);
  const at::Tensor* pre = tensor_or_none(args[3]);
  const int64_t act = number(args[4]);
  if (X.dim() != 2 || W.dim() != 2 || act < 0 || (act > 0 && !pre)) throw Unusual{};
  const Call c(X, number(args[12]));
  void* stream = reinterpret_cast<void*>(number(args[13]));
  const int64_t m = X.size(0), k = X.size(1), n = W.size(0);
  const int64_t ldx = c.pitch(X, m, k), ldw = c.pitch(W, n, k), ldg = c.pitch(G, m, n);
  const int64_t ldp = act > 0 ? c.pitch(*pre, m, n) : (n > 0 ? n : 1);
  int need_out[3];
  const at::Tensor* out[3];
  for (int i = 0; i < 3; ++i) {
    need_out[i] = PyObject_IsTrue(args[5 + i]);
    if (need_out[i] < 0) {
      PyErr_Clear();
      throw Unusual{};
    }
    out[i] = need_out[i] ? tensor_or_none(args[8 + i]) : nullptr;
  }
  int64_t ld[2] = {k > 0 ? k : 1, k > 0 ? k : 1};
  if (out[0]) ld[0] = c.pitch(*out[0], m, k);
  if (out[1]) ld[1] = c.pitch(*out[1], n, k);
  if (out[2]) c.vector(*out[2], n);
  const void *gp = G.data_ptr(), *xp = X.data_ptr(), *wp = W.data_ptr(), *zp = act > 0 ? pre->data_ptr() : nullptr;
  const Entries& e = entries[c.element];
  size_t need = 0;
  const bool aligned = c.aligned(gp, ldg) && c.aligned(xp, ldx) && c.aligned(wp, ldw);
  int status = e.backward_size(m, k, n, (int)act, aligned, &need);
  if (status) return PyLong_FromLong(status);
  at::Tensor made[3];
  if (need_out[0] && !out[0]) out[0] = &(made[0] = at::empty({m, k}, X.options()));
  if (need_out[1] && !out[1]) out[1] = &(made[1] = at::empty({n, k}, X.options()));
  if (need_out[2] && !out[2]) out[2] = &(made[2] = at::empty({n}, X.options().dtype(at::kFloat)));
  const Workspace ws(args[11], need, X, c);
  void *p0 = out[0] ? out[0]->data_ptr() : nullptr, *p1 = out[1] ? out[1]->data_ptr() : nullptr;
  float* p2 = out[2] ? static_cast<float*>(out[2]->data_ptr()) : nullptr;
  Py_BEGIN_ALLOW_THREADS
  status = e.backward(m, k, n, gp, ldg, xp, ldx, wp, ldw, zp, ldp, (int)act, p0, ld[0], p1, ld[1], p2, ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  if (status) return PyLong_FromLong(status);
  PyObject* r = PyTuple_New(3);
  for (int i = 0; r && i < 3; ++i) {
    PyObject* o = Py_None;
    if (need_out[i]) o = wrapped(made[i], args[8 + i]);
    else Py_INCREF(o);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

// C++ exceptions (of torch's accessors and allocations) become Python ones here.
template <PyObject* (*fn)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  try {
    return fn(args, nargs);
  } catch (const Unusual&) {
    Py_RETURN_NONE;
  } catch (const c10::OutOfMemoryError&) {  // the caller's own allocation raises torch's error
    Py_RETURN_NONE;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <PyObject* (*fn)(PyObject* const*, Py_ssize_t)>
PyCFunction method() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(guarded<fn>));
}

PyMethodDef methods[] = {
    {"addresses", method<addresses>(), METH_FASTCALL,
     "addresses(tensors, numel, out, n, device): checks the tensors and writes their addresses"},
    {"written", method<written>(), METH_FASTCALL, "written(tensors): moves their version counters"},
    {"bind", method<bind>(), METH_FASTCALL, "bind(12 addresses): the layer's entry points by element type"},
    {"linear", method<linear>(), METH_FASTCALL, "one call of the layer; None if its arguments need the caller's checks"},
    {"linear_backward", method<linear_backward>(), METH_FASTCALL,
     "one call of the layer's gradient; None if its arguments need the caller's checks"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
