// tensors.cpp — what the binding asks of torch tensors, many at a time: a Python extension of its own beside the library, which
// knows nothing of torch.  Looked over from Python a tensor takes 0.3 us (type, shape, device, contiguity, address, each a
// call), here 0.01 us in a list and 0.06 us alone: the norm and clip of 200 small tensors out of place, 161 -> 22 us, a call
// with nine of them 8.6 -> 6.8 us.  (Without it a clip of 1000 small tensors would take longer than elementary operations on
// one tensor that holds them all.)
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

constexpr int kF32 = 0, kBF16 = 1;   // lmoe_dtype

// bf16_at(tensor, shape, device) -> address of a contiguous bf16 tensor of that shape on that CUDA device; -1 if it is not one
PyObject* bf16_at(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 3 || !PyTuple_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "bf16_at(tensor, shape, device)");
    return nullptr;
  }
  const long device = PyLong_AsLong(args[2]);
  if (device == -1 && PyErr_Occurred()) return nullptr;
  if (!THPVariable_Check(args[0])) return PyLong_FromLong(-1);
  try {
    const at::Tensor& t = THPVariable_Unpack(args[0]);
    if (!t.defined() || t.scalar_type() != at::kBFloat16 || !t.is_cuda() || t.get_device() != device || !t.is_contiguous() ||
        t.dim() != PyTuple_GET_SIZE(args[1]))
      return PyLong_FromLong(-1);
    for (Py_ssize_t i = 0; i < t.dim(); ++i) {
      const long long d = PyLong_AsLongLong(PyTuple_GET_ITEM(args[1], i));
      if (d == -1 && PyErr_Occurred()) return nullptr;
      if (t.size(i) != d) return PyLong_FromLong(-1);
    }
    return PyLong_FromVoidPtr(t.data_ptr());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// gradients(iterable, name, device) -> (addresses, sizes, dtypes) of its tensors as packed uint64, int64 and int32, and their number
PyObject* gradients(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "gradients(iterable, name, device)");
    return nullptr;
  }
  const char* name = PyUnicode_AsUTF8(args[1]);
  const long device = PyLong_AsLong(args[2]);
  if (name == nullptr || (device == -1 && PyErr_Occurred())) return nullptr;
  PyObject* seq = PySequence_Tuple(args[0]);   // (of its own: another thread may change the caller's list)
  if (seq == nullptr) return nullptr;
  const Py_ssize_t count = PyTuple_GET_SIZE(seq);
  PyObject* at = PyBytes_FromStringAndSize(nullptr, count * 8);
  PyObject* sizes = PyBytes_FromStringAndSize(nullptr, count * 8);
  PyObject* kinds = PyBytes_FromStringAndSize(nullptr, count * 4);
  PyObject* result = nullptr;
  if (at != nullptr && sizes != nullptr && kinds != nullptr) {
    auto* p = reinterpret_cast<uint64_t*>(PyBytes_AS_STRING(at));
    auto* s = reinterpret_cast<int64_t*>(PyBytes_AS_STRING(sizes));
    auto* k = reinterpret_cast<int32_t*>(PyBytes_AS_STRING(kinds));
    bool ok = true;
    try {
      for (Py_ssize_t i = 0; ok && i < count; ++i) {
        PyObject* item = PyTuple_GET_ITEM(seq, i);
        ok = THPVariable_Check(item);
        if (!ok) {
          PyErr_Format(PyExc_ValueError, "%s: element %zd is not a tensor", name, i);
          break;
        }
        const at::Tensor& t = THPVariable_Unpack(item);
        const auto type = t.scalar_type();
        if (!t.is_cuda() || t.get_device() != device) {
          PyErr_Format(PyExc_ValueError, "%s: all tensors must be on cuda:%ld", name, device);
          ok = false;
        } else if (t.layout() != at::kStrided || !t.is_contiguous()) {
          PyErr_Format(PyExc_ValueError, "%s: tensors must be contiguous", name);
          ok = false;
        } else if (type != at::kFloat && type != at::kBFloat16) {
          PyErr_Format(PyExc_ValueError, "%s: tensors must be float32 or bfloat16", name);
          ok = false;
        } else {
          p[i] = reinterpret_cast<uint64_t>(t.data_ptr());
          s[i] = t.numel();
          k[i] = type == at::kFloat ? kF32 : kBF16;
        }
      }
    } catch (const std::exception& e) {
      PyErr_SetString(PyExc_RuntimeError, e.what());
      ok = false;
    }
    if (ok) result = Py_BuildValue("(OOOn)", at, sizes, kinds, count);
  }
  Py_XDECREF(at);
  Py_XDECREF(sizes);
  Py_XDECREF(kinds);
  Py_DECREF(seq);
  return result;
}

PyMethodDef methods[] = {
    {"bf16_at", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bf16_at)), METH_FASTCALL, nullptr},
    {"gradients", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gradients)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: of the headers, whose layout of torch's objects is compiled in
PyMODINIT_FUNC PyInit__tensors(void) {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", LMOE_TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
