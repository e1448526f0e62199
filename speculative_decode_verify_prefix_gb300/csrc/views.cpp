// The tensor views of a call, for the Python binding (cache_ops.py): what
// include/verify_splitkv.h wants to know of every tensor, packed into one buffer.
// (In Python the attributes of 14 tensors take 10.5 us, more than all the rest of a
// short call; so 0.5.)
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <exception>

#include <torch/csrc/autograd/python_variable.h>

#include "../../include/verify_splitkv.h"

namespace {

int code_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return VSK_DTYPE_BF16;
    case at::kFloat8_e4m3fn: return VSK_DTYPE_FP8E4M3;
    case at::kInt: return VSK_DTYPE_I32;
    case at::kLong: return VSK_DTYPE_I64;
    case at::kByte:
    case at::kBool: return VSK_DTYPE_U8;
    case at::kFloat: return VSK_DTYPE_F32;
    default: return -1;
  }
}

// views(names, tensors): (device index, the views' buffer, each view's address or
// None).  ValueError where a tensor is not on a CUDA device, or not on the first
// one's, or has no memory to point at.
PyObject* views(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 2 || !PyTuple_Check(args[0]) || !PyTuple_Check(args[1]) || PyTuple_GET_SIZE(args[0]) < PyTuple_GET_SIZE(args[1])) {
    PyErr_SetString(PyExc_TypeError, "views(names, tensors)");
    return nullptr;
  }
  const Py_ssize_t n = PyTuple_GET_SIZE(args[1]);
  PyObject* buf = PyBytes_FromStringAndSize(nullptr, n * static_cast<Py_ssize_t>(sizeof(vsk_tensor)));
  PyObject* list = PyList_New(n);
  if (!buf || !list) {
    Py_XDECREF(buf);
    Py_XDECREF(list);
    return nullptr;
  }
  vsk_tensor* v = reinterpret_cast<vsk_tensor*>(PyBytes_AS_STRING(buf));
  long device = -1;
  bool bad = false;
  for (Py_ssize_t i = 0; i < n && !bad; ++i, ++v) {
    PyObject* o = PyTuple_GET_ITEM(args[1], i);
    PyObject* entry;
    if (o == Py_None) {
      Py_INCREF(o);
      entry = o;
    } else {
      PyObject* name = PyTuple_GET_ITEM(args[0], i);
      const long dev = THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda() ? THPVariable_Unpack(o).get_device() : -1;
      if (dev < 0 || (device >= 0 && dev != device)) {
        if (dev < 0)
          PyErr_Format(PyExc_ValueError, "%U must be a CUDA tensor", name);
        else
          PyErr_Format(PyExc_ValueError, "%U is on cuda:%ld, the call's other tensors on cuda:%ld", name, dev, device);
        bad = true;
        break;
      }
      device = dev;
      try {
        const at::Tensor& t = THPVariable_Unpack(o);
        v->data = t.data_ptr();
        v->dtype = code_of(t.scalar_type());
        v->ndim = static_cast<int32_t>(t.dim());
        for (int d = 0; d < 3; ++d) {
          v->shape[d] = d < v->ndim ? t.size(d) : 0;
          v->stride[d] = d < v->ndim ? t.stride(d) : 0;
        }
      } catch (const std::exception&) {  // a layout without memory or strides
        PyErr_Format(PyExc_ValueError, "%U must be a strided CUDA tensor", name);
        bad = true;
        break;
      }
      entry = PyLong_FromVoidPtr(v);
      if (!entry) {
        bad = true;
        break;
      }
    }
    PyList_SET_ITEM(list, i, entry);
  }
  if (!bad && device < 0) {
    PyErr_Format(PyExc_ValueError, "%U must be a CUDA tensor", PyTuple_GET_ITEM(args[0], 0));
    bad = true;
  }
  PyObject* out = bad ? nullptr : Py_BuildValue("(lNN)", device, buf, list);
  if (!out) {
    if (bad) {
      Py_DECREF(buf);
      Py_DECREF(list);
    }
    return nullptr;
  }
  return out;
}

PyMethodDef kMethods[] = {{"views", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(views)), METH_FASTCALL,
                           "views(names, tensors): the packed views of a call's tensors"},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "vsk_views", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_vsk_views() { return PyModule_Create(&kModule); }
