// art_marshal.cpp -- argument marshalling of the binding's cache operators: a
// CPython module that turns torch tensors into the art_tensor_t descriptors of
// a parameter structure and calls the library's entry point on the right
// device and stream.  Filling the same structures from Python took 16 of the
// 20 us a small art_rope_append call took on the host; here it is under one.
//
//   call(entry, name, stream, tensors, others, tail) -> status
//     entry    address of art_status_t fn(const void *params, art_stream_t)
//     stream   None for the tensors' device's current stream, or a handle
//     tensors  the structure's leading descriptors, None for an absent one
//     others   further tensors of the call (None allowed), checked for their device
//     tail     bytes of the structure after the descriptors
//   query(entry, tensors, tail) -> int   int64_t fn(const void *params)
//   empty(like, type, sizes...) -> tensor   contiguous, uninitialised, on like's device; type
//                                           an art_dtype_t, or -1 for bytes
//   empty_as(like, type, drop) -> tensor  the same with like's sizes but its last `drop` ones; type
//                                         -2: like's own
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <exception>

#include "../../include/art.h"

namespace {

constexpr Py_ssize_t kMostTensors = 16;
constexpr Py_ssize_t kMostTail = 256;

// What an empty tensor's descriptor points at: NULL data means an absent
// argument, and one that was passed has to meet the shape checks instead (no
// tensor that passes them is empty, but for an append of no tokens, which
// launches nothing: it is never read).
alignas(256) unsigned char no_elements[256];

struct Params {
    alignas(16) unsigned char bytes[kMostTensors * sizeof(art_tensor_t) + kMostTail];
    int device = -1;
};

// the tensor's device joins the call's; false with a Python error set
bool join_device(const at::Tensor &t, Params *p, const char *name)
{
    if (!t.is_cuda()) {
        PyErr_SetString(PyExc_ValueError, "libart runs on the GPU only: every tensor must be on a CUDA device");
        return false;
    }
    const int d = t.get_device();
    if (p->device >= 0 && d != p->device) {
        PyErr_Format(PyExc_ValueError, "%s: the tensors are on different devices", name);
        return false;
    }
    p->device = d;
    return true;
}

const at::Tensor *tensor_of(PyObject *o)
{
    if (!THPVariable_Check(o)) {
        PyErr_SetString(PyExc_TypeError, "expected a torch.Tensor or None");
        return nullptr;
    }
    return &THPVariable_Unpack(o);
}

bool fill(PyObject *tensors, PyObject *others, PyObject *tail, const char *name, Params *p)
{
    if (!PyTuple_Check(tensors) || PyTuple_GET_SIZE(tensors) > kMostTensors || !PyBytes_Check(tail) ||
        PyBytes_GET_SIZE(tail) > kMostTail || (others && !PyTuple_Check(others))) {
        PyErr_SetString(PyExc_TypeError, "bad argument block");
        return false;
    }
    const Py_ssize_t n = PyTuple_GET_SIZE(tensors);
    for (Py_ssize_t i = 0; i < n; ++i) {
        art_tensor_t d;
        std::memset(&d, 0, sizeof d);
        PyObject *o = PyTuple_GET_ITEM(tensors, i);
        if (o != Py_None) {
            const at::Tensor *t = tensor_of(o);
            if (!t || !join_device(*t, p, name))
                return false;
            const auto type = t->scalar_type();
            d.data = t->numel() ? t->data_ptr() : no_elements;
            d.dtype = type == at::kFloat ? ART_F32 : type == at::kBFloat16 ? ART_BF16 : type == at::kInt ? ART_I32 : -1;
            d.ndim = (int32_t)t->dim();
            for (int64_t k = 0; k < t->dim() && k < 4; ++k) {
                d.shape[k] = t->size(k);
                d.stride[k] = t->stride(k);
            }
        }
        std::memcpy(p->bytes + i * sizeof d, &d, sizeof d);
    }
    std::memcpy(p->bytes + n * sizeof(art_tensor_t), PyBytes_AS_STRING(tail), (size_t)PyBytes_GET_SIZE(tail));
    for (Py_ssize_t i = 0; others && i < PyTuple_GET_SIZE(others); ++i) {
        PyObject *o = PyTuple_GET_ITEM(others, i);
        if (o == Py_None)
            continue;
        const at::Tensor *t = tensor_of(o);
        if (!t || !join_device(*t, p, name))
            return false;
    }
    if (p->device < 0) {
        PyErr_SetString(PyExc_TypeError, "no tensor given");
        return false;
    }
    return true;
}

PyObject *raised(const std::exception &e)
{
    if (!PyErr_Occurred())
        PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
}

PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (nargs != 6) {
        PyErr_SetString(PyExc_TypeError, "call(entry, name, stream, tensors, others, tail)");
        return nullptr;
    }
    using Entry = art_status_t (*)(const void *, art_stream_t);
    const Entry entry = reinterpret_cast<Entry>(PyLong_AsVoidPtr(args[0]));
    const char *name = entry ? PyUnicode_AsUTF8(args[1]) : nullptr;
    if (!name) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_TypeError, "no entry point");
        return nullptr;
    }
    try {
        Params p;
        if (!fill(args[3], args[4], args[5], name, &p))
            return nullptr;
        art_stream_t stream;
        if (args[2] == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)p.device).stream();
        } else {
            stream = static_cast<art_stream_t>(PyLong_AsVoidPtr(args[2]));
            if (PyErr_Occurred())
                return nullptr;
        }
        art_status_t status;
        {
            const c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.device);
            Py_BEGIN_ALLOW_THREADS
            status = entry(p.bytes, stream);
            Py_END_ALLOW_THREADS
        }
        return PyLong_FromLong((long)status);
    } catch (const std::exception &e) {
        return raised(e);
    }
}

PyObject *query(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (nargs != 3) {
        PyErr_SetString(PyExc_TypeError, "query(entry, tensors, tail)");
        return nullptr;
    }
    using Entry = int64_t (*)(const void *);
    const Entry entry = reinterpret_cast<Entry>(PyLong_AsVoidPtr(args[0]));
    if (!entry) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_TypeError, "no entry point");
        return nullptr;
    }
    try {
        Params p;
        if (!fill(args[1], nullptr, args[2], "query", &p))
            return nullptr;
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.device);
        return PyLong_FromLongLong((long long)entry(p.bytes));
    } catch (const std::exception &e) {
        return raised(e);
    }
}

PyObject *new_tensor(const at::Tensor &like, long type, at::IntArrayRef sizes)
{
    const auto kind = type == -2 ? like.scalar_type() : type == ART_F32 ? at::kFloat : type == ART_BF16 ? at::kBFloat16
                      : type == ART_I32 ? at::kInt : at::kByte;
    return THPVariable_Wrap(at::empty(sizes, at::TensorOptions().dtype(kind).device(like.device())));
}

PyObject *empty(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (nargs < 3 || nargs > 6) {
        PyErr_SetString(PyExc_TypeError, "empty(like, type, sizes...)");
        return nullptr;
    }
    try {
        const at::Tensor *like = tensor_of(args[0]);
        if (!like)
            return nullptr;
        const long type = PyLong_AsLong(args[1]);
        int64_t sizes[4];
        for (Py_ssize_t i = 2; i < nargs; ++i) {
            sizes[i - 2] = PyLong_AsLongLong(args[i]);
            if (sizes[i - 2] < 0 && !PyErr_Occurred())
                PyErr_SetString(PyExc_ValueError, "negative size");
        }
        if (PyErr_Occurred())
            return nullptr;
        return new_tensor(*like, type, at::IntArrayRef(sizes, (size_t)(nargs - 2)));
    } catch (const std::exception &e) {
        return raised(e);
    }
}

PyObject *empty_as(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    if (nargs != 3) {
        PyErr_SetString(PyExc_TypeError, "empty_as(like, type, drop)");
        return nullptr;
    }
    try {
        const at::Tensor *like = tensor_of(args[0]);
        if (!like)
            return nullptr;
        const long type = PyLong_AsLong(args[1]), drop = PyLong_AsLong(args[2]);
        if (PyErr_Occurred())
            return nullptr;
        const auto sizes = like->sizes();
        if (drop < 0 || (size_t)drop > sizes.size()) {
            PyErr_SetString(PyExc_ValueError, "too few dimensions");
            return nullptr;
        }
        return new_tensor(*like, type, sizes.slice(0, sizes.size() - (size_t)drop));
    } catch (const std::exception &e) {
        return raised(e);
    }
}

PyMethodDef methods[] = {
    {"empty", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(empty)), METH_FASTCALL, nullptr},
    {"empty_as", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(empty_as)), METH_FASTCALL, nullptr},
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL, nullptr},
    {"query", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(query)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "argument marshalling of the cache operators", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
