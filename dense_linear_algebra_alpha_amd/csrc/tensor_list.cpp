// Python extension module _tensors: what the helpers on torch tensors do per call, where Python would
// take longer than the GPU. addresses(): a list of tensors, checked (reading five attributes of 200
// tensors from Python takes 45 us, this 3 us). written(): their version counters moved (torch's own call takes
// 8 us for 200, this 1.2). linear() and linear_backward(): the checks, outputs and
// workspace of one call of the layer and the call itself (7.6 and 14.7 us from Python, 3.7 and
// 8.0 here; a small layer takes the GPU 4 us); the functions after them the same of layer norm, embedding and the
// losses (one row's layer norm 8.6 us a call from Python, 5.0 here, a token's embedding 8.0 and 4.9). Host code only; built
// against torch's headers, resolved against the torch that the process has imported; the C entry points come in by bind().
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>

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
typedef int (*Norm)(int64_t, int64_t, const void*, int64_t, const float*, const float*, float, void*, int64_t, float*, float*,
                    void*);
typedef int (*NormSize)(int64_t, int64_t, size_t*);
typedef int (*NormBackward)(int64_t, int64_t, const void*, int64_t, const void*, int64_t, const float*, const float*,
                            const float*, void*, int64_t, float*, float*, void*, size_t, void*);
typedef int (*Embedding)(int64_t, int64_t, int64_t, const void*, int, const void*, int64_t, float, void*, int64_t, void*);
typedef int (*EmbeddingSize)(int64_t, int64_t, int64_t, size_t*);
typedef int (*EmbeddingBackward)(int64_t, int64_t, int64_t, const void*, int64_t, const void*, int, float, int, void*, int64_t,
                                 void*, size_t, void*);
typedef int (*EntropySize)(int64_t, int64_t, int64_t, int, size_t*);
typedef int (*Entropy)(int64_t, int64_t, int64_t, const void*, int64_t, const void*, int64_t, const float*, const void*, int,
                       float*, float*, void*, size_t, void*);
typedef int (*EntropyBackward)(int64_t, int64_t, int64_t, const float*, const void*, int64_t, const void*, int64_t, const float*,
                               const void*, int, const float*, void*, int64_t, void*, int64_t, float*, void*, size_t, void*);
typedef int (*DistillationSize)(int64_t, int64_t, int64_t, int64_t, int, size_t*);
typedef int (*Distillation)(int64_t, int64_t, int64_t, const void*, int64_t, const void*, int64_t, const float*, int64_t,
                            const void*, int64_t, int, const void*, int64_t, int, float, float*, float*, float*, void*, size_t,
                            void*);
typedef int (*DistillationBackward)(int64_t, int64_t, int64_t, const float*, const void*, int64_t, const void*, int64_t,
                                    const float*, int64_t, const void*, int64_t, int, const float*, float, const float*, void*,
                                    int64_t, void*, int64_t, float*, void*, size_t, void*);
struct Entries {
  LinearSize linear_size;
  Linear linear;
  BackwardSize backward_size;
  Backward backward;
  Norm norm;
  NormSize norm_size;
  NormBackward norm_backward;
  Embedding embedding;
  EmbeddingSize embedding_size;
  EmbeddingBackward embedding_backward;
  EntropySize entropy_size;
  Entropy entropy;
  EntropySize entropy_backward_size;
  EntropyBackward entropy_backward;
  DistillationSize distillation_size;
  Distillation distillation;
  DistillationSize distillation_backward_size;
  DistillationBackward distillation_backward;
} entries[3];  // f32, bf16, f16
constexpr int kEntries = sizeof(Entries) / sizeof(void*);
bool bound = false;

// bind(addresses of the 3 x kEntries entry points, in the order of the structure)
PyObject* bind(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 3 * kEntries) {
    PyErr_Format(PyExc_TypeError, "bind takes %d addresses", 3 * kEntries);
    return nullptr;
  }
  for (int i = 0; i < 3 * kEntries; ++i) reinterpret_cast<void**>(entries)[i] = PyLong_AsVoidPtr(args[i]);
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

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Unusual{};
  }
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    throw Unusual{};
  }
  return v != 0;
}
// Address of an optional float32 vector.
const float* vector_or_none(const Call& c, PyObject* o, int64_t n) {
  const at::Tensor* t = tensor_or_none(o);
  return t ? c.vector(*t, n) : nullptr;
}
// Bits of a contiguous index tensor's elements.
int index_bits(const Call& c, const at::Tensor& t) {
  const int bits = t.scalar_type() == at::kLong ? 64 : t.scalar_type() == at::kInt ? 32 : 0;
  if (!bits || !t.is_cuda() || t.layout() != c10::kStrided || t.get_device() != c.device || !t.is_contiguous()) throw Unusual{};
  return bits;
}

// An output: the caller's tensor, or one made here, or none.
struct Output {
  at::Tensor made;
  PyObject* given = Py_None;
  void* p = nullptr;
  int64_t ld = 1;
  bool wanted = true;
  void matrix(const Call& c, PyObject* o, int64_t rows, int64_t cols, const at::Tensor& like) {
    if (const at::Tensor* t = tensor_or_none(given = o)) {
      ld = c.pitch(*t, rows, cols);
      p = t->data_ptr();
    } else {
      made = at::empty({rows, cols}, like.options());
      ld = cols > 0 ? cols : 1;
      p = made.data_ptr();
    }
  }
  // float32, of one or two dimensions (cols < 0: one), contiguous
  void floats(const Call& c, PyObject* o, int64_t rows, int64_t cols, const at::Tensor& like) {
    if (const at::Tensor* t = tensor_or_none(given = o)) {
      if (cols < 0) {
        p = c.vector(*t, rows);
        return;
      }
      c.on_device(*t, at::kFloat);
      if (t->dim() != 2 || t->size(0) != rows || t->size(1) != cols || !t->is_contiguous()) throw Unusual{};
      p = t->data_ptr();
    } else {
      made = cols < 0 ? at::empty({rows}, like.options().dtype(at::kFloat)) : at::empty({rows, cols}, like.options().dtype(at::kFloat));
      p = made.data_ptr();
    }
  }
  float* f() const { return static_cast<float*>(p); }
};

// The outputs as Python has them: one, or a tuple.
PyObject* results(std::initializer_list<const Output*> outputs) {
  if (outputs.size() == 1) return wrapped((*outputs.begin())->made, (*outputs.begin())->given);
  PyObject* r = PyTuple_New((Py_ssize_t)outputs.size());
  Py_ssize_t i = 0;
  for (const Output* o : outputs) {
    if (!r) break;
    PyObject* v = Py_None;
    if (o->wanted) v = wrapped(o->made, o->given);
    else Py_INCREF(v);
    if (!v) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, v);
  }
  return r;
}

void* stream_of(PyObject* o) { return reinterpret_cast<void*>(number(o)); }

// Each of the following: the result; a number: the entry point's error; None: left to the caller. They end with the
// workspace (where there is one), the current device and the stream.

// layer_norm(X, weight, bias, eps, save_stats, out, mean, rstd, device, stream)
PyObject* layer_norm(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 10) throw Unusual{};
  const at::Tensor& X = tensor(args[0]);
  const Call c(X, number(args[8]));
  if (X.dim() != 2) throw Unusual{};
  const int64_t m = X.size(0), n = X.size(1), ldx = c.pitch(X, m, n);
  const float *weight = vector_or_none(c, args[1], n), *bias = vector_or_none(c, args[2], n);
  const float eps = (float)real(args[3]);
  const bool stats = truth(args[4]) || args[6] != Py_None || args[7] != Py_None;
  void* stream = stream_of(args[9]);
  Output out, mean, rstd;
  out.matrix(c, args[5], m, n, X);
  if (stats) {
    mean.floats(c, args[6], m, -1, X);
    rstd.floats(c, args[7], m, -1, X);
  }
  const void* x = X.data_ptr();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = entries[c.element].norm(m, n, x, ldx, weight, bias, eps, out.p, out.ld, mean.f(), rstd.f(), stream);
  Py_END_ALLOW_THREADS
  if (status) return PyLong_FromLong(status);
  return stats ? results({&out, &mean, &rstd}) : results({&out});
}

// layer_norm_backward(G, X, mean, rstd, weight, need_dX, need_dweight, need_dbias, dX, dweight, dbias, workspace, device,
// stream)
PyObject* layer_norm_backward(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 14) throw Unusual{};
  const at::Tensor &G = tensor(args[0]), &X = tensor(args[1]);
  const Call c(X, number(args[12]));
  if (X.dim() != 2) throw Unusual{};
  const int64_t m = X.size(0), n = X.size(1), ldx = c.pitch(X, m, n), ldg = c.pitch(G, m, n);
  const float *mean = c.vector(tensor(args[2]), m), *rstd = c.vector(tensor(args[3]), m), *weight = vector_or_none(c, args[4], n);
  void* stream = stream_of(args[13]);
  Output out[3];
  for (int i = 0; i < 3; ++i) {
    out[i].wanted = truth(args[5 + i]);
    if (!out[i].wanted) continue;
    if (i == 0) out[i].matrix(c, args[8], m, n, X);
    else out[i].floats(c, args[8 + i], n, -1, X);
  }
  const Entries& e = entries[c.element];
  size_t need = 0;
  int status = 0;
  if (out[1].wanted || out[2].wanted) status = e.norm_size(m, n, &need);
  if (status) return PyLong_FromLong(status);
  const Workspace ws(args[11], need, X, c);
  const void *g = G.data_ptr(), *x = X.data_ptr();
  Py_BEGIN_ALLOW_THREADS
  status = e.norm_backward(m, n, g, ldg, x, ldx, mean, rstd, weight, out[0].p, out[0].ld < n ? (n > 0 ? n : 1) : out[0].ld,
                           out[1].f(), out[2].f(), ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  if (status) return PyLong_FromLong(status);
  return results({&out[0], &out[1], &out[2]});
}

// embedding(ids, table, scale, out, device, stream)
PyObject* embedding(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 6) throw Unusual{};
  const at::Tensor &ids = tensor(args[0]), &table = tensor(args[1]);
  const Call c(table, number(args[4]));
  if (table.dim() != 2 || ids.dim() != 1) throw Unusual{};
  const int64_t rows = table.size(0), k = table.size(1), count = ids.size(0), ldt = c.pitch(table, rows, k);
  const int bits = index_bits(c, ids);
  const float scale = (float)real(args[2]);
  void* stream = stream_of(args[5]);
  Output out;
  out.matrix(c, args[3], count, k, table);
  const void *i = ids.data_ptr(), *t = table.data_ptr();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = entries[c.element].embedding(count, k, rows, i, bits, t, ldt, scale, out.p, out.ld, stream);
  Py_END_ALLOW_THREADS
  return status ? PyLong_FromLong(status) : results({&out});
}

// embedding_backward(G, ids, rows, scale, dtable, accumulate, workspace, device, stream)
PyObject* embedding_backward(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 9) throw Unusual{};
  const at::Tensor &G = tensor(args[0]), &ids = tensor(args[1]);
  const Call c(G, number(args[7]));
  if (G.dim() != 2 || ids.dim() != 1) throw Unusual{};
  const int64_t count = G.size(0), k = G.size(1), rows = number(args[2]), ldg = c.pitch(G, count, k);
  if (ids.size(0) != count || rows < 0) throw Unusual{};
  const int bits = index_bits(c, ids);
  const float scale = (float)real(args[3]);
  const bool accumulate = truth(args[5]);
  if (accumulate && args[4] == Py_None) throw Unusual{};
  void* stream = stream_of(args[8]);
  const Entries& e = entries[c.element];
  size_t need = 0;
  int status = e.embedding_size(count, k, rows, &need);
  if (status) return PyLong_FromLong(status);
  Output out;
  out.matrix(c, args[4], rows, k, G);
  const Workspace ws(args[6], need, G, c);
  const void *g = G.data_ptr(), *i = ids.data_ptr();
  Py_BEGIN_ALLOW_THREADS
  status = e.embedding_backward(count, k, rows, g, ldg, i, bits, scale, accumulate, out.p, out.ld, ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return status ? PyLong_FromLong(status) : results({&out});
}

// The output layer of a loss.
struct OutputLayer {
  const Call c;
  int64_t m, k, n, ldx, ldw;
  const void *x, *w;
  const float* bias;
  bool aligned;
  OutputLayer(const at::Tensor& X, const at::Tensor& W, PyObject* b, PyObject* device) : c(X, number(device)) {
    if (X.dim() != 2 || W.dim() != 2) throw Unusual{};
    m = X.size(0);
    k = X.size(1);
    n = W.size(0);
    ldx = c.pitch(X, m, k);
    ldw = c.pitch(W, n, k);
    x = X.data_ptr();
    w = W.data_ptr();
    bias = vector_or_none(c, b, n);
    aligned = c.aligned(x, ldx) && c.aligned(w, ldw);
  }
};

// The gradients (dX, dW, db) of a loss, from args: need_dX, need_dW, need_db, dX, dW, db.
struct LossGradients {
  Output out[3];
  LossGradients(const OutputLayer& l, PyObject* const* args, const at::Tensor& X) {
    for (int i = 0; i < 3; ++i) {
      out[i].wanted = truth(args[i]);
      if (i < 2) out[i].ld = l.k > 0 ? l.k : 1;
      if (!out[i].wanted) continue;
      if (i == 2) out[i].floats(l.c, args[5], l.n, -1, X);
      else out[i].matrix(l.c, args[3 + i], i == 0 ? l.m : l.n, l.k, X);
    }
  }
  PyObject* tuple() const { return results({&out[0], &out[1], &out[2]}); }
};

// cross_entropy(X, W, labels, bias, loss, lse, workspace, device, stream)
PyObject* cross_entropy(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 9) throw Unusual{};
  const at::Tensor &X = tensor(args[0]), &labels = tensor(args[2]);
  const OutputLayer l(X, tensor(args[1]), args[3], args[7]);
  if (labels.dim() != 1 || labels.size(0) != l.m) throw Unusual{};
  const int bits = index_bits(l.c, labels);
  void* stream = stream_of(args[8]);
  Output loss, lse;
  loss.floats(l.c, args[4], l.m, -1, X);
  lse.floats(l.c, args[5], l.m, -1, X);
  const Entries& e = entries[l.c.element];
  size_t need = 0;
  int status = e.entropy_size(l.m, l.k, l.n, l.aligned, &need);
  if (status) return PyLong_FromLong(status);
  const Workspace ws(args[6], need, X, l.c);
  const void* y = labels.data_ptr();
  Py_BEGIN_ALLOW_THREADS
  status = e.entropy(l.m, l.k, l.n, l.x, l.ldx, l.w, l.ldw, l.bias, y, bits, loss.f(), lse.f(), ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return status ? PyLong_FromLong(status) : results({&loss, &lse});
}

// cross_entropy_backward(grad, X, W, labels, lse, bias, need_dX, need_dW, need_db, dX, dW, db, workspace, device, stream)
PyObject* cross_entropy_backward(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 15) throw Unusual{};
  const at::Tensor &X = tensor(args[1]), &labels = tensor(args[3]);
  const OutputLayer l(X, tensor(args[2]), args[5], args[13]);
  if (labels.dim() != 1 || labels.size(0) != l.m) throw Unusual{};
  const int bits = index_bits(l.c, labels);
  const float *grad = l.c.vector(tensor(args[0]), l.m), *lse = l.c.vector(tensor(args[4]), l.m);
  void* stream = stream_of(args[14]);
  const LossGradients g(l, args + 6, X);
  const Entries& e = entries[l.c.element];
  size_t need = 0;
  int status = e.entropy_backward_size(l.m, l.k, l.n, l.aligned, &need);
  if (status) return PyLong_FromLong(status);
  const Workspace ws(args[12], need, X, l.c);
  const void* y = labels.data_ptr();
  Py_BEGIN_ALLOW_THREADS
  status = e.entropy_backward(l.m, l.k, l.n, grad, l.x, l.ldx, l.w, l.ldw, l.bias, y, bits, lse, g.out[0].p, g.out[0].ld, g.out[1].p,
                              g.out[1].ld, g.out[2].f(), ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return status ? PyLong_FromLong(status) : g.tuple();
}

// distillation(X, W, classes, teacher, bias, temperature, loss, lse, weights, workspace, device, stream)
PyObject* distillation(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 12) throw Unusual{};
  const at::Tensor &X = tensor(args[0]), &classes = tensor(args[2]), &teacher = tensor(args[3]);
  const OutputLayer l(X, tensor(args[1]), args[4], args[10]);
  if (classes.dim() != 2 || classes.size(0) != l.m) throw Unusual{};
  const int64_t s = classes.size(1);
  const int bits = index_bits(l.c, classes);
  const Call of_teacher(teacher, l.c.device);
  const int64_t ldt = of_teacher.pitch(teacher, l.m, s);
  const float temperature = (float)real(args[5]);
  void* stream = stream_of(args[11]);
  Output loss, lse, weights;
  loss.floats(l.c, args[6], l.m, -1, X);
  lse.floats(l.c, args[7], l.m, -1, X);
  weights.floats(l.c, args[8], l.m, s, X);
  const Entries& e = entries[l.c.element];
  size_t need = 0;
  int status = e.distillation_size(l.m, l.k, l.n, s, l.aligned, &need);
  if (status) return PyLong_FromLong(status);
  const Workspace ws(args[9], need, X, l.c);
  const void *cp = classes.data_ptr(), *tp = teacher.data_ptr();
  Py_BEGIN_ALLOW_THREADS
  status = e.distillation(l.m, l.k, l.n, l.x, l.ldx, l.w, l.ldw, l.bias, s, cp, s > 0 ? s : 1, bits, tp, ldt, of_teacher.element + 1,
                          temperature, loss.f(), lse.f(), weights.f(), ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return status ? PyLong_FromLong(status) : results({&loss, &lse, &weights});
}

// distillation_backward(grad, X, W, classes, weights, lse, bias, temperature, need_dX, need_dW, need_db, dX, dW, db,
// workspace, device, stream)
PyObject* distillation_backward(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 17) throw Unusual{};
  const at::Tensor &X = tensor(args[1]), &classes = tensor(args[3]), &weights = tensor(args[4]);
  const OutputLayer l(X, tensor(args[2]), args[6], args[15]);
  if (classes.dim() != 2 || classes.size(0) != l.m) throw Unusual{};
  const int64_t s = classes.size(1);
  const int bits = index_bits(l.c, classes);
  l.c.on_device(weights, at::kFloat);
  if (weights.dim() != 2 || weights.size(0) != l.m || weights.size(1) != s || !weights.is_contiguous()) throw Unusual{};
  const float *grad = l.c.vector(tensor(args[0]), l.m), *lse = l.c.vector(tensor(args[5]), l.m);
  const float temperature = (float)real(args[7]);
  void* stream = stream_of(args[16]);
  const LossGradients g(l, args + 8, X);
  const Entries& e = entries[l.c.element];
  size_t need = 0;
  int status = e.distillation_backward_size(l.m, l.k, l.n, s, l.aligned, &need);
  if (status) return PyLong_FromLong(status);
  const Workspace ws(args[14], need, X, l.c);
  const void* cp = classes.data_ptr();
  const float* wp = static_cast<const float*>(weights.data_ptr());
  Py_BEGIN_ALLOW_THREADS
  status = e.distillation_backward(l.m, l.k, l.n, grad, l.x, l.ldx, l.w, l.ldw, l.bias, s, cp, s > 0 ? s : 1, bits, wp, temperature,
                                   lse, g.out[0].p, g.out[0].ld, g.out[1].p, g.out[1].ld, g.out[2].f(), ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return status ? PyLong_FromLong(status) : g.tuple();
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
    {"bind", method<bind>(), METH_FASTCALL, "bind(addresses): the entry points by element type"},
    {"linear", method<linear>(), METH_FASTCALL, "one call of the layer; None if its arguments need the caller's checks"},
    {"linear_backward", method<linear_backward>(), METH_FASTCALL,
     "one call of the layer's gradient; None if its arguments need the caller's checks"},
    {"layer_norm", method<layer_norm>(), METH_FASTCALL, "one call of layer norm, as linear"},
    {"layer_norm_backward", method<layer_norm_backward>(), METH_FASTCALL, "one call of layer norm's gradient, as linear"},
    {"embedding", method<embedding>(), METH_FASTCALL, "one call of the embedding lookup, as linear"},
    {"embedding_backward", method<embedding_backward>(), METH_FASTCALL, "one call of its gradient, as linear"},
    {"cross_entropy", method<cross_entropy>(), METH_FASTCALL, "one call of the cross entropy, as linear"},
    {"cross_entropy_backward", method<cross_entropy_backward>(), METH_FASTCALL, "one call of its gradient, as linear"},
    {"distillation", method<distillation>(), METH_FASTCALL, "one call of the distillation, as linear"},
    {"distillation_backward", method<distillation_backward>(), METH_FASTCALL, "one call of its gradient, as linear"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
