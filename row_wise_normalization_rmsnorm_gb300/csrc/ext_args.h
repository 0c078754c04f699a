// ext_args.h -- what the Python binding's calls share: errors, argument
// checks, the stream a call launches on and the memory its results lie in.
#pragma once

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <optional>
#include <string>
#include <vector>

#include "../../include/rmsnorm.h"

namespace ext {

// A Python exception to raise; thrown inside, set at the entry points.
struct Bad {
    PyObject *type;
    std::string what;
};
// A Python exception that is already set.
struct AlreadySet {};

[[noreturn]] inline void value_error(std::string s) { throw Bad{PyExc_ValueError, std::move(s)}; }
[[noreturn]] inline void type_error(std::string s) { throw Bad{PyExc_TypeError, std::move(s)}; }

inline std::string str(int64_t v) { return std::to_string(v); }
inline std::string shape_of(const at::Tensor &t) {
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + str(t.size(i));
    return s + "]";
}

inline const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

// RMSNORM_* code of a tensor's type.
inline int dtype_code(const at::Tensor &t) {
    switch (t.scalar_type()) {
    case at::kFloat: return RMSNORM_F32;
    case at::kBFloat16: return RMSNORM_BF16;
    case at::kHalf: return RMSNORM_F16;
    default: type_error("unsupported dtype; use torch.float32, torch.bfloat16 or torch.float16");
    }
}

// A vector or table beside the rows.
inline void beside(const at::Tensor &t, const char *name, at::ScalarType a, at::ScalarType b, const at::Tensor &like,
            bool contiguous = true) {
    if (t.device() != like.device()) value_error(std::string(name) + " must be on the input's device");
    if (t.scalar_type() != a && t.scalar_type() != b)
        value_error(std::string(name) + " must be " + c10::toString(a) + (a == b ? "" : std::string(" or ") + c10::toString(b)) +
                    ", is " + c10::toString(t.scalar_type()));
    if (contiguous && !t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
}

inline void *ptr(const at::Tensor &t) { return t.data_ptr(); }

// The stream that a call launches on: the device's current one (None), a
// handle, or an object with one.
struct LaunchStream {
    rmsnorm_stream_t handle;
    std::optional<c10::cuda::CUDAStream> named;  // where the caller named one
    LaunchStream(PyObject *stream, const at::Tensor &like) {
        const c10::DeviceIndex device = like.device().index();
        if (stream == Py_None) {
            handle = reinterpret_cast<rmsnorm_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
            return;
        }
        PyObject *h = PyLong_Check(stream) ? Py_NewRef(stream) : PyObject_GetAttrString(stream, "cuda_stream");
        if (!h) throw AlreadySet{};
        void *p = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!p && PyErr_Occurred()) throw AlreadySet{};
        if (p == static_cast<void *>(cudaStreamLegacy)) p = nullptr;  // the same stream; PyTorch knows it as 0
        handle = static_cast<rmsnorm_stream_t>(p);
        named = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), device);
    }
};

// A contiguous tensor on `like`'s device, from PyTorch's allocator (its CUDA
// entry itself: the dispatched at::empty takes 0.9 us a tensor longer). For a
// named stream the memory is that stream's own: the current stream's may still
// be in use by what was queued there before its last owner dropped it, and the
// named stream waits for none of that. Its first reader is likely to be the
// current stream, so the memory is not given out again, once dropped, before
// that one is done with it either.
inline at::Tensor new_tensor(at::IntArrayRef size, at::ScalarType type, const at::Tensor &like, const LaunchStream &s) {
    if (!s.named) return at::Tensor(at::detail::empty_cuda(size, type, like.device(), std::nullopt));
    const c10::cuda::CUDAStream reader = c10::cuda::getCurrentCUDAStream(like.device().index());
    at::Tensor t;
    {
        c10::cuda::CUDAStreamGuard on(*s.named);
        t = at::Tensor(at::detail::empty_cuda(size, type, like.device(), std::nullopt));
    }
    if (t.numel() > 0) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), reader);
    return t;
}

inline int32_t size32(int64_t v, const char *name) {
    if (v < 0 || v > 0x7fffffff) value_error(std::string(name) + " is out of range");
    return (int32_t)v;
}

inline int32_t int_arg(PyObject *o, const char *name) {
    PyObject *n = PyNumber_Index(o);
    if (!n) {
        PyErr_Clear();
        type_error(std::string(name) + " must be an integer");
    }
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(n, &overflow);
    Py_DECREF(n);
    if (overflow) value_error(std::string(name) + " is out of range");
    return size32(v, name);
}

inline float float_arg(PyObject *o, const char *name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(std::string(name) + " must be a number");
    }
    return (float)v;
}

// The tensors' device made current for the call, where it is not.
struct OnDevice {
    std::optional<c10::cuda::CUDAGuard> guard;
    explicit OnDevice(const at::Tensor &t) {
        if (t.device().index() != c10::cuda::current_device()) guard.emplace(t.device());
    }
};

// _binding._raise(status, what): the library's error as RMSNormError
inline void check(rmsnorm_status_t st, const char *what) {
    if (st == RMSNORM_SUCCESS) return;
    PyObject *m = PyImport_ImportModule("row_wise_normalization_rmsnorm_gb300._binding");
    PyObject *r = m ? PyObject_CallMethod(m, "_raise", "is", (int)st, what) : nullptr;
    Py_XDECREF(m);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, what);
    throw AlreadySet{};
}

// A new reference that is dropped unless taken.
struct Ref {
    PyObject *o = nullptr;
    ~Ref() { Py_XDECREF(o); }
    PyObject *take() {
        PyObject *r = o;
        o = nullptr;
        return r;
    }
};

template <class F> PyObject *guarded(F &&f) {
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Bad &b) {
        PyErr_SetString(b.type, b.what.c_str());
    } catch (const AlreadySet &) {
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

inline bool count(Py_ssize_t have, Py_ssize_t want) {
    if (have == want) return true;
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return false;
}

}  // namespace ext
