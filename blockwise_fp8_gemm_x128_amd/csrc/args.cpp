// Argument checks of the Python binding in one native call: a dozen tensors of an operator against
// their expected types, shapes, contiguity and device, and their addresses, in a microsecond
// instead of the five that the same questions take through the interpreter.
//
//   ptrs(spec, device, d0, d1, d2, *tensors) -> tuple of addresses, or the index of the first
//                                               tensor that is not as the specification says
//
// spec: four bytes per tensor: its type (b bf16, f fp32, q uint8), ! or ? (may be None, address 0),
// and the indices of its one or two sizes among d0, d1, d2 and the number 1 (3), - for none.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

namespace {

bool as_specified(const at::Tensor& t, const char* spec, int64_t device, const int64_t* dims) {
  const at::ScalarType type = spec[0] == 'b'   ? at::kBFloat16
                              : spec[0] == 'f' ? at::kFloat
                                               : at::kByte;
  const int64_t rank = spec[3] == '-' ? 1 : 2;
  if (t.scalar_type() != type || t.dim() != rank) return false;
  for (int64_t i = 0; i < rank; ++i)
    if (t.size(i) != dims[spec[2 + i] - '0']) return false;
  return t.is_contiguous() && t.is_cuda() && t.get_device() == device;
}

PyObject* ptrs(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr Py_ssize_t kFirst = 5;
  if (n < kFirst || !PyBytes_Check(args[0]) || PyBytes_GET_SIZE(args[0]) != 4 * (n - kFirst)) {
    PyErr_SetString(PyExc_TypeError, "ptrs(spec, device, d0, d1, d2, *tensors)");
    return nullptr;
  }
  const char* spec = PyBytes_AS_STRING(args[0]);
  int64_t v[4];
  for (int i = 0; i < 4; ++i) v[i] = PyLong_AsLongLong(args[1 + i]);
  if (PyErr_Occurred()) return nullptr;
  const int64_t dims[4] = {v[1], v[2], v[3], 1};
  PyObject* out = PyTuple_New(n - kFirst);
  if (out == nullptr) return nullptr;
  for (Py_ssize_t i = 0; i < n - kFirst; ++i, spec += 4) {
    PyObject* o = args[kFirst + i];
    uint64_t address = 0;
    bool ok = o == Py_None ? spec[1] == '?' : false;
    if (!ok && THPVariable_Check(o)) {
      try {
        const at::Tensor& t = THPVariable_Unpack(o);
        ok = as_specified(t, spec, v[0], dims);
        if (ok) address = reinterpret_cast<uint64_t>(t.const_data_ptr());
      } catch (const std::exception&) {  // a layout without strides or storage (sparse, nested)
        ok = false;
      }
    }
    PyObject* item = ok ? PyLong_FromUnsignedLongLong(address) : nullptr;
    if (item == nullptr) {
      Py_DECREF(out);
      return PyErr_Occurred() ? nullptr : PyLong_FromSsize_t(i);
    }
    PyTuple_SET_ITEM(out, i, item);
  }
  return out;
}

PyMethodDef kMethods[] = {
    {"ptrs", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(ptrs)), METH_FASTCALL,
     "Checked addresses of an operator's tensors."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_args", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__args(void) { return PyModule_Create(&kModule); }
