/* layer_tensor.h -- what layer_py.c reads of a torch tensor and of torch's state,
 * from torch's C++ side (layer_tensor.cpp).  Errors set a Python exception. */
#pragma once
#include <Python.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Types by bigemm_dtype (F32, F16, BF16, MXF8 for float8_e4m3fn), and those of scales. */
enum { TYPE_SCALE_U8 = 4, TYPE_SCALE_E8M0 = 5, TYPE_OTHER = -1 };

typedef struct {
    int dims, type, contiguous;
    long device;                     /* -1: not a CUDA tensor */
    long long size[2], stride[2];    /* of the first two axes */
    long long numel;
    void *ptr;
} LayerTensor;

int layer_tensor(PyObject *t, const char *name, LayerTensor *out);

/* The current device, and its current stream of `device`. */
int layer_current(long device, long *current, void **stream);

#ifdef __cplusplus
}
#endif
