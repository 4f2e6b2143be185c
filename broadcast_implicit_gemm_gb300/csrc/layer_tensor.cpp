// layer_tensor.cpp -- torch tensors as layer_py.c reads them.  Through Python a tensor's
// shape, strides, type, device and address are five calls, 0.4 us; here they are a few
// loads (8 x 256 rmsnorm_backward, five tensors: 7.6 us of host time with the calls, 4.8
// so; rmsnorm 3.5 and 2.4, matmul_gated_backward 10.5 and 5.8).
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "layer_tensor.h"

namespace {

int type_of(at::ScalarType t)
{
    switch (t) {
    case at::ScalarType::Float: return 0;
    case at::ScalarType::Half: return 1;
    case at::ScalarType::BFloat16: return 2;
    case at::ScalarType::Float8_e4m3fn: return 3;
    case at::ScalarType::Byte: return TYPE_SCALE_U8;
    case at::ScalarType::Float8_e8m0fnu: return TYPE_SCALE_E8M0;
    default: return TYPE_OTHER;
    }
}

}  // namespace

int layer_tensor(PyObject *o, const char *name, LayerTensor *out)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
        return -1;
    }
    // (a tensor without memory of its own, a fake one for instance, throws)
    try {
        const at::Tensor &t = THPVariable_Unpack(o);
        if (t.is_neg()) {
            PyErr_Format(PyExc_ValueError, "%s: its values are still to be negated (resolve_neg does it)", name);
            return -1;
        }
        out->dims = (int)t.dim();
        const at::IntArrayRef size = t.sizes(), stride = t.strides();
        for (int i = 0; i < 2; ++i) {
            out->size[i] = i < out->dims ? size[i] : 0;
            out->stride[i] = i < out->dims ? stride[i] : 0;
        }
        out->numel = t.numel();
        out->contiguous = t.is_contiguous();
        out->type = type_of(t.scalar_type());
        out->device = t.is_cuda() ? (long)t.get_device() : -1;
        out->ptr = t.data_ptr();
        return 0;
    } catch (const std::exception &e) {
        PyErr_Format(PyExc_RuntimeError, "%s: %s", name, e.what());
    } catch (...) {
        PyErr_Format(PyExc_RuntimeError, "%s: not readable", name);
    }
    return -1;
}

int layer_current(long device, long *current, void **stream)
{
    try {
        *current = (long)c10::cuda::current_device();
        *stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
        return 0;
    } catch (const std::exception &e) {
        PyErr_Format(PyExc_RuntimeError, "current stream: %s", e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "current stream: not readable");
    }
    return -1;
}
