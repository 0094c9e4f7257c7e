// tensor_list.cpp -- the addresses, sizes and types of a list of torch tensors as an
// array of mxfp4_grad_item_t, for the calls on all gradients of a model.  Hundreds of
// tensors cost a few microseconds here; asked one by one from Python they cost more than
// the kernels (448 gradients, in and out: 160 us of calls for 78 us of kernels).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <exception>

#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mxfp4.h"

namespace {

// The i-th tensor, checked; NULL with a Python error set.
const at::Tensor *tensor_at(PyObject *list, Py_ssize_t i, const char *what) {
  PyObject *o = PySequence_Fast_GET_ITEM(list, i);
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s is a list of tensors, got %s", what, Py_TYPE(o)->tp_name);
    return nullptr;
  }
  const at::Tensor &t = THPVariable_Unpack(o);
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat) {
    PyErr_Format(PyExc_ValueError, "%s must be bfloat16 or float32 tensors, got %s", what, c10::toString(t.scalar_type()));
    return nullptr;
  }
  if (t.layout() != at::kStrided || !t.is_contiguous()) {
    PyErr_SetString(PyExc_ValueError, "tensors must be contiguous");
    return nullptr;
  }
  return &t;
}

bool on_device(const at::Tensor &t, long device) {
  if (t.is_cuda() && t.get_device() == device) return true;
  PyErr_SetString(PyExc_ValueError, t.is_cuda() ? "tensors must live on the current GPU"
                                                : "tensors must live on the GPU (no CPU path)");
  return false;
}

// pack(grads, outs or None, device, write) -> (items as bytes, elements); without outs and
// with write, the gradients are the outputs.
PyObject *pack(PyObject *, PyObject *args) {
  PyObject *grads, *outs;
  long device;
  int write;
  if (!PyArg_ParseTuple(args, "OOlp", &grads, &outs, &device, &write)) return nullptr;
  PyObject *g = PySequence_Fast(grads, "grads is a list of tensors");
  if (!g) return nullptr;
  PyObject *o = nullptr;
  if (outs != Py_None && !(o = PySequence_Fast(outs, "outs is a list of tensors"))) {
    Py_DECREF(g);
    return nullptr;
  }
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(g);
  PyObject *bytes = nullptr, *result = nullptr;
  try {
    int64_t elements = 0;
    bool good = true;
    if (o && PySequence_Fast_GET_SIZE(o) != n) {
      PyErr_SetString(PyExc_ValueError, "outs must have the types and sizes of grads");
      good = false;
    }
    bytes = good ? PyBytes_FromStringAndSize(nullptr, n * (Py_ssize_t)sizeof(mxfp4_grad_item_t)) : nullptr;
    good = bytes != nullptr;
    mxfp4_grad_item_t *item = good ? reinterpret_cast<mxfp4_grad_item_t *>(PyBytes_AS_STRING(bytes)) : nullptr;
    for (Py_ssize_t i = 0; good && i < n; ++i) {
      const at::Tensor *t = tensor_at(g, i, "grads");
      const at::Tensor *u = t && o ? tensor_at(o, i, "outs") : t;
      if (!t || !u) {
        good = false;
      } else if (u->scalar_type() != t->scalar_type() || u->numel() != t->numel()) {
        PyErr_SetString(PyExc_ValueError, "outs must have the types and sizes of grads");
        good = false;
      } else if (!on_device(*t, device) || (o && !on_device(*u, device))) {
        good = false;
      } else {
        item[i] = {t->const_data_ptr(), write ? u->mutable_data_ptr() : nullptr, t->numel(),
                   t->scalar_type() == at::kFloat ? MXFP4_F32 : MXFP4_BF16, 0};
        elements += t->numel();
      }
    }
    if (good) result = Py_BuildValue("(OL)", bytes, (long long)elements);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    result = nullptr;
  }
  Py_XDECREF(bytes);
  Py_XDECREF(o);
  Py_DECREF(g);
  return result;
}

PyMethodDef methods[] = {{"pack", pack, METH_VARARGS, "pack(grads, outs or None, device, write) -> (items, elements)"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_list", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_list() { return PyModule_Create(&module); }
