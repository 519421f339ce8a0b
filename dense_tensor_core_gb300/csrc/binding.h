// binding.h -- what the files of the Python binding share: the checks of arguments, the stream of a call, and
// errors (see ffn_binding.cpp).
#pragma once

#include <Python.h>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <exception>
#include <sstream>
#include <string>

#include <initializer_list>

#include "dtc_ffn.h"

namespace dtc_py {

inline PyObject* g_gemm_error = nullptr;  // GemmError(status, message)

struct Refusal {
    PyObject* type;
    std::string what;
};
[[noreturn]] inline void refuse(PyObject* type, const std::string& what) { throw Refusal{type, what}; }
struct LibraryError {
    int status;
};
struct PythonError {};  // an exception is set already

inline std::string shape_of(at::IntArrayRef s) {
    std::ostringstream o;
    o << "(";
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << (s.size() == 1 ? ",)" : ")");
    return o.str();
}

inline int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}
// A number of a C int, and a wait's limit.
inline int small(PyObject* o, const char* name) {
    const int64_t v = integer(o);
    if (v != (int)v) refuse(PyExc_ValueError, std::string(name) + " is out of range: " + std::to_string(v));
    return (int)v;
}
inline uint64_t timeout(PyObject* o) {
    const int64_t v = integer(o);
    if (v < 0) refuse(PyExc_ValueError, "timeout_ns must not be negative");
    return (uint64_t)v;
}
inline double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return v;
}
inline const at::Tensor* maybe(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}
inline const at::Tensor& tensor(PyObject* o, const char* name) {
    const at::Tensor* t = maybe(o, name);
    if (!t) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    return *t;
}

// The operands' device, which every tensor of a call must be on. (The type is looked at first.)
inline c10::Device device_of(const at::Tensor& t, at::ScalarType dt, const char* name) {
    if (t.scalar_type() != dt)
        refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(dt) + ", got " +
                                    c10::toString(t.scalar_type()));
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
    return t.device();
}
inline void base(const at::Tensor& t, at::ScalarType dt, const char* name, c10::Device dev) {
    if (t.scalar_type() != dt)
        refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(dt) + ", got " +
                                    c10::toString(t.scalar_type()));
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
    if (t.device() != dev)
        refuse(PyExc_ValueError, "all tensors must be on one CUDA device, got " + std::string(name) +
                                     " on " + t.device().str() + " and others on " + dev.str());
}
inline void dense(const at::Tensor& t, at::ScalarType dt, const char* name, c10::Device dev) {
    base(t, dt, name, dev);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be dense row-major");
}
// A 2-D operand that may be rows of a larger row-major array; its leading dimension (0: dense).
inline int64_t matrix(const at::Tensor& t, at::ScalarType dt, const char* name, c10::Device dev) {
    base(t, dt, name, dev);
    if (t.dim() != 2) refuse(PyExc_ValueError, std::string(name) + " must be 2-D");
    if (t.is_contiguous()) return 0;
    if (t.stride(1) == 1 && t.stride(0) >= t.size(1)) return t.size(0) > 1 ? t.stride(0) : 0;
    refuse(PyExc_ValueError, std::string(name) + " must be dense row-major or rows of a larger row-major array");
}
inline void shape(const at::Tensor& t, at::IntArrayRef want, const char* name) {
    if (t.sizes() != want)
        refuse(PyExc_ValueError, std::string(name) + " must be " + shape_of(want) + ", got " + shape_of(t.sizes()));
}
inline void* address(const at::Tensor* t) { return t && t->numel() > 0 ? t->data_ptr() : nullptr; }
inline void* address(const at::Tensor& t) { return address(&t); }

inline at::Tensor empty(at::IntArrayRef sizes, at::ScalarType dt, c10::Device dev) {
    return at::empty(sizes, at::TensorOptions().dtype(dt).device(dev));
}

inline at::ScalarType type16(int64_t kind) { return kind == 0 ? at::kBFloat16 : at::kHalf; }
inline int float_code(const at::Tensor& t, const char* name) {
    switch (t.scalar_type()) {
        case at::kBFloat16: return 0;
        case at::kHalf: return 1;
        case at::kFloat: return 2;
        default:
            refuse(PyExc_TypeError, std::string(name) + " must be bf16, fp16 or fp32, got " +
                                        c10::toString(t.scalar_type()));
    }
}
inline bool gated(int64_t act) { return act >= GEMM_ACT_SWIGLU; }

// Makes `dev` current, and with it the given stream (an integer handle; None: the current one), for as
// long as it lives. Set up before anything is allocated: the allocator hands memory that is freed on a
// stream to that stream's next request, so buffers that die when the call returns must have come from
// the stream their kernels run on, and so must outputs, whose memory earlier work of another stream may
// still be using.
class OnStream {
public:
    OnStream(c10::Device dev, PyObject* stream) {
        device_.set_device(dev);
        if (stream != Py_None)
            stream_.reset_stream(c10::cuda::getStreamFromExternal(
                (cudaStream_t)(uintptr_t)integer(stream), dev.index()));
        handle_ = (dtc_stream_t)c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    }
    // Calls the library, without the interpreter lock (a launch may wait for room in the queue).
    template <typename F>
    void call(F f) const {
        int status;
        Py_BEGIN_ALLOW_THREADS;
        status = f(handle_);
        Py_END_ALLOW_THREADS;
        if (status) throw LibraryError{status};
    }

private:
    c10::cuda::OptionalCUDAGuard device_;
    c10::cuda::OptionalCUDAStreamGuard stream_;
    dtc_stream_t handle_ = nullptr;
};

inline PyObject* wrap(const at::Tensor& t) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) throw PythonError{};
    return o;
}
// A tuple of tensors (None for undefined ones).
inline PyObject* tuple(std::initializer_list<at::Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) throw PythonError{};
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) {
        PyObject* o = t.defined() ? THPVariable_Wrap(t) : (Py_INCREF(Py_None), Py_None);
        if (!o) {
            Py_DECREF(r);
            throw PythonError{};
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// Every entry: the argument count, and no C++ exception past it.
template <typename F>
inline PyObject* entry(Py_ssize_t got, Py_ssize_t want, F f) {
    try {
        if (got != want) refuse(PyExc_TypeError, "expected " + std::to_string(want) + " arguments");
        // outputs and views are made without torch's gradient bookkeeping (a microsecond or two each)
        const at::AutoDispatchBelowADInplaceOrView guard;
        return f();
    } catch (const Refusal& r) {
        PyErr_SetString(r.type, r.what.c_str());
    } catch (const LibraryError& e) {
        const char* msg = gemm_last_error();
        PyObject* v = PyObject_CallFunction(g_gemm_error, "iN", e.status,
                                            PyUnicode_DecodeUTF8(msg, (Py_ssize_t)strlen(msg), "replace"));
        if (v) {
            PyErr_SetObject(g_gemm_error, v);
            Py_DECREF(v);
        }
    } catch (const PythonError&) {
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

#define DTC_FN(name) {#name, (PyCFunction)(void*)py_##name, METH_FASTCALL, nullptr}

// The methods of fp4_binding.cpp, ended by an empty one.
extern PyMethodDef kFp4Methods[];

}  // namespace dtc_py
