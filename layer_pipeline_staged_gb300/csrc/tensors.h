/* What the marshalling (marshal.c) asks of torch's C++ side (tensors.cpp), which is
 * built against one version of torch and loaded for that one only: the same facts
 * through a tensor's Python attributes take half a microsecond a tensor instead of a
 * few hundredths. Every function returns nonzero (or NULL) where it has no answer,
 * with no Python error set; the Python way then has it, or its error. */
#ifndef LPS_TENSORS_H
#define LPS_TENSORS_H

#include <Python.h>
#include <stdint.h>

#define LPS_TENSORS_DIM 5

enum { LPS_T_OTHER, LPS_T_BF16, LPS_T_FP16, LPS_T_FP32, LPS_T_FP64, LPS_T_INT32 };

typedef struct {
  int64_t shape[LPS_TENSORS_DIM], stride[LPS_TENSORS_DIM];
  void *ptr;
  int dim, dtype, device, grad, neg;
} tensor_facts;

typedef struct {
  int (*facts)(PyObject *obj, tensor_facts *f);  /* of a torch.Tensor itself or a Parameter */
  PyObject *(*empty)(const int64_t *shape, int dim, int dtype, int device); /* a new dense CUDA tensor */
  int (*written)(PyObject *obj);                 /* its version counter moves on */
} tensor_api;

#endif
