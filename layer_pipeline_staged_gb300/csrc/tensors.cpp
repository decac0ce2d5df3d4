// Tensors' facts, new tensors and version counters through torch's C++ interface, for
// the marshalling of the torch wrappers (tensors.h). A Python extension of its own, so
// that the rest needs no particular torch.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <torch/version.h>

#include "tensors.h"

namespace {

int kind_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return LPS_T_BF16;
    case at::kHalf: return LPS_T_FP16;
    case at::kFloat: return LPS_T_FP32;
    case at::kDouble: return LPS_T_FP64;
    case at::kInt: return LPS_T_INT32;
    default: return LPS_T_OTHER;
  }
}

int facts(PyObject* obj, tensor_facts* f) {
  if (!THPVariable_CheckExact(obj)) return 1;
  try {
    const at::Tensor& t = THPVariable_Unpack(obj);
    if (t.layout() != at::kStrided || t.dim() > LPS_TENSORS_DIM) return 1;
    f->dim = static_cast<int>(t.dim());
    const auto shape = t.sizes(), stride = t.strides();
    for (int i = 0; i < f->dim; ++i) f->shape[i] = shape[i], f->stride[i] = stride[i];
    f->dtype = kind_of(t.scalar_type());
    f->device = static_cast<int>(t.get_device());
    f->grad = t.requires_grad();
    f->neg = t.is_neg();
    f->ptr = t.data_ptr();
    return 0;
  } catch (...) {
    return 1;
  }
}

PyObject* empty(const int64_t* shape, int dim, int dtype, int device) {
  static const at::ScalarType types[] = {at::kByte, at::kBFloat16, at::kHalf, at::kFloat, at::kDouble, at::kInt};
  if (dtype <= LPS_T_OTHER || dtype > LPS_T_INT32) return nullptr;
  try {
    PyObject* x = THPVariable_Wrap(at::empty(at::IntArrayRef(shape, dim), at::TensorOptions().dtype(types[dtype]).device(at::kCUDA, static_cast<c10::DeviceIndex>(device))));
    if (!x) PyErr_Clear();
    return x;
  } catch (...) {
    return nullptr;
  }
}

int written(PyObject* obj) {
  if (!THPVariable_CheckExact(obj)) return 1;
  try {
    THPVariable_Unpack(obj).unsafeGetTensorImpl()->bump_version();
    return 0;
  } catch (...) {
    return 1;
  }
}

tensor_api api = {facts, empty, written};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, nullptr, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() {
  PyObject* m = PyModule_Create(&module);
  PyObject* capsule = m ? PyCapsule_New(&api, "layer_pipeline_staged_gb300.tensor_api", nullptr) : nullptr;
  if (!capsule || PyModule_AddObject(m, "api", capsule) || PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION)) {
    Py_XDECREF(m);
    return nullptr;
  }
  return m;
}
