// Argument checks of the calls around the experts, for the Python binding.
//
// In a decode step those calls take a few microseconds each, launch included,
// and asking a tensor for its dtype, shape, device and layout from Python costs
// about 0.3 us per tensor; here it is one call of 0.05 us (moe_add_rmsnorm of one
// row of 7168 with a residual: 8.5 -> 6.3 us a call).  These functions only
// answer; what is wrong is said by the binding.  A tensor that has no plain
// memory (sparse, nested, fake) throws when asked for it: that is a no as well,
// and no exception leaves an entry.
#include <Python.h>

#include <exception>

#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// head(t) -> (device index, rows, columns) of a two-dimensional tensor on the
// current GPU, else None.
PyObject* head(PyObject*, PyObject* obj) {
  if (!THPVariable_Check(obj)) Py_RETURN_NONE;
  const at::Tensor& t = THPVariable_Unpack(obj);
  try {
    if (!t.is_cuda() || t.dim() != 2) Py_RETURN_NONE;
    const long idx = t.get_device();
    const c10::impl::VirtualGuardImpl gpu(c10::DeviceType::CUDA);
    if (gpu.getDevice().index() != idx) Py_RETURN_NONE;
    return Py_BuildValue("(lLL)", idx, (long long)t.size(0), (long long)t.size(1));
  } catch (const std::exception&) {
    Py_RETURN_NONE;
  }
}

// plain(t, dtype, rows, columns, device index) -> the address of a contiguous
// GPU tensor of just that dtype, shape (columns -1: one-dimensional) and
// device, else -1.
PyObject* plain(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5 || !THPDtype_Check(a[1])) {
    PyErr_SetString(PyExc_TypeError, "plain(tensor, dtype, rows, columns, device index)");
    return nullptr;
  }
  const long long rows = PyLong_AsLongLong(a[2]), cols = PyLong_AsLongLong(a[3]);
  const long idx = PyLong_AsLong(a[4]);
  if (PyErr_Occurred()) return nullptr;
  if (!THPVariable_Check(a[0])) return PyLong_FromLong(-1);
  const at::Tensor& t = THPVariable_Unpack(a[0]);
  try {
    const bool ok = t.scalar_type() == reinterpret_cast<THPDtype*>(a[1])->scalar_type &&
                    t.is_cuda() && t.get_device() == idx && t.dim() == (cols < 0 ? 1 : 2) &&
                    t.size(0) == rows && (cols < 0 || t.size(1) == cols) && t.is_contiguous();
    return ok ? PyLong_FromVoidPtr(t.data_ptr()) : PyLong_FromLong(-1);
  } catch (const std::exception&) {
    return PyLong_FromLong(-1);
  }
}

PyMethodDef methods[] = {
    {"head", head, METH_O, "(device index, rows, columns) of a 2-D tensor on the current GPU"},
    {"plain", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(plain)), METH_FASTCALL,
     "address of a contiguous tensor of this dtype, shape and device, or -1"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args() { return PyModule_Create(&module); }
