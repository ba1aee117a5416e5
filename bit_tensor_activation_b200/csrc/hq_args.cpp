// hq_args.cpp -- the binding's argument checks as a Python module: one call looks a tensor over and
// returns its address, in about a tenth of the time that the same questions take one by one in Python.
// A kernel of the library for a single token runs for a few microseconds, as long as the checks of its
// ten arguments took.  Nothing is raised here: what does not pass returns None, and the binding then
// finds out in Python what to say.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// The tensor of `o` if its type is in `mask`, it lies on CUDA device `dev` (any, if negative) and has the
// sizes in the tuple `shape`; else null.
const at::Tensor* match(PyObject* o, long dev, unsigned long long mask, PyObject* shape) {
  if (!THPVariable_Check(o) || !PyTuple_Check(shape)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || !((mask >> static_cast<int>(t.scalar_type())) & 1)) return nullptr;
  if (dev >= 0 && t.get_device() != dev) return nullptr;
  const auto sizes = t.sizes();
  if (static_cast<Py_ssize_t>(sizes.size()) != PyTuple_GET_SIZE(shape)) return nullptr;
  for (size_t i = 0; i < sizes.size(); ++i) {
    const long long n = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
    if (n == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      return nullptr;
    }
    if (n != sizes[i]) return nullptr;
  }
  return &t;
}

bool numbers(PyObject* const* args, long* dev, unsigned long long* mask) {
  *dev = PyLong_AsLong(args[1]);
  *mask = PyLong_AsUnsignedLongLong(args[2]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

// dense(tensor, device, mask, shape) -> address of a contiguous tensor (0 if it is empty), or None
PyObject* dense(PyObject*, PyObject* const* args, Py_ssize_t n) {
  long dev = 0;
  unsigned long long mask = 0;
  if (n == 4 && numbers(args, &dev, &mask)) {
    const at::Tensor* t = match(args[0], dev, mask, args[3]);
    if (t && t->is_contiguous()) return PyLong_FromVoidPtr(t->numel() ? t->data_ptr() : nullptr);
  }
  Py_RETURN_NONE;
}

// mask(dtypes) -> the set of the tuple's types for the calls above
PyObject* mask_of(PyObject*, PyObject* dtypes) {
  unsigned long long m = 0;
  if (!PyTuple_Check(dtypes)) {
    PyErr_SetString(PyExc_TypeError, "a tuple of dtypes");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(dtypes); ++i) {
    PyObject* d = PyTuple_GET_ITEM(dtypes, i);
    if (!THPDtype_Check(d)) {
      PyErr_SetString(PyExc_TypeError, "a tuple of dtypes");
      return nullptr;
    }
    m |= 1ull << static_cast<int>(reinterpret_cast<THPDtype*>(d)->scalar_type);
  }
  return PyLong_FromUnsignedLongLong(m);
}

PyMethodDef methods[] = {
    {"dense", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(dense)), METH_FASTCALL, nullptr},
    {"mask", mask_of, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hqargs", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__hqargs() { return PyModule_Create(&module); }
