// Python extension module _tensors: the addresses of a list of torch tensors, checked, for calls that
// take hundreds of tensors each step (reading five attributes of 200 tensors from Python takes 45 us,
// this 3 us). Host code only; built against torch's headers and resolved against the torch that the
// process has imported.
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

// addresses(tensors: list, numel: address of int64[n], out: address of uint64[n], n, device: int) -> -1, or the position of the first tensor that is not a contiguous strided tensor
// of numel[i] elements on GPU `device` with the first tensor's type.
PyObject* addresses(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
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

// C++ exceptions (of torch's accessors) become Python ones here.
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  try {
    return addresses(self, args, nargs);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {
    {"addresses", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(guarded)), METH_FASTCALL,
     "addresses(tensors, numel, out, n, device): checks the tensors and writes their addresses"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
