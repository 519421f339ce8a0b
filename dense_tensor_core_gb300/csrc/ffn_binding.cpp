// ffn_binding.cpp -- the Python binding of the feed-forward operators (include/dtc_ffn.h) as a
// CPython module: argument checks, output allocation and the call, no arithmetic.
//
// Native because the smallest calls are bound by the host: a call of gemm_act on 256 x 256 x 512
// operands, whose kernel takes a few microseconds, spent 10 of its 14 us in checks and marshalling
// written in Python. The functions take their arguments by position, as _ffn.py passes them, which
// also documents them. Refusals are TypeError (a type), ValueError (anything else about an argument)
// and GemmError (what the library answers).
#include <Python.h>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <sstream>
#include <string>

#include "dtc_ffn.h"

namespace {

PyObject* g_gemm_error = nullptr;  // GemmError(status, message)

struct Refusal {
    PyObject* type;
    std::string what;
};
[[noreturn]] void refuse(PyObject* type, const std::string& what) { throw Refusal{type, what}; }
struct LibraryError {
    int status;
};
struct PythonError {};  // an exception is set already

std::string shape_of(at::IntArrayRef s) {
    std::ostringstream o;
    o << "(";
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << (s.size() == 1 ? ",)" : ")");
    return o.str();
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}
// A number of a C int, and a wait's limit.
int small(PyObject* o, const char* name) {
    const int64_t v = integer(o);
    if (v != (int)v) refuse(PyExc_ValueError, std::string(name) + " is out of range: " + std::to_string(v));
    return (int)v;
}
uint64_t timeout(PyObject* o) {
    const int64_t v = integer(o);
    if (v < 0) refuse(PyExc_ValueError, "timeout_ns must not be negative");
    return (uint64_t)v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return v;
}
const at::Tensor* maybe(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name) {
    const at::Tensor* t = maybe(o, name);
    if (!t) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    return *t;
}

// The operands' device, which every tensor of a call must be on. (The type is looked at first.)
c10::Device device_of(const at::Tensor& t, at::ScalarType dt, const char* name) {
    if (t.scalar_type() != dt)
        refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(dt) + ", got " +
                                    c10::toString(t.scalar_type()));
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
    return t.device();
}
void base(const at::Tensor& t, at::ScalarType dt, const char* name, c10::Device dev) {
    if (t.scalar_type() != dt)
        refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(dt) + ", got " +
                                    c10::toString(t.scalar_type()));
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
    if (t.device() != dev)
        refuse(PyExc_ValueError, "all tensors must be on one CUDA device, got " + std::string(name) +
                                     " on " + t.device().str() + " and others on " + dev.str());
}
void dense(const at::Tensor& t, at::ScalarType dt, const char* name, c10::Device dev) {
    base(t, dt, name, dev);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be dense row-major");
}
// A 2-D operand that may be rows of a larger row-major array; its leading dimension (0: dense).
int64_t matrix(const at::Tensor& t, at::ScalarType dt, const char* name, c10::Device dev) {
    base(t, dt, name, dev);
    if (t.dim() != 2) refuse(PyExc_ValueError, std::string(name) + " must be 2-D");
    if (t.is_contiguous()) return 0;
    if (t.stride(1) == 1 && t.stride(0) >= t.size(1)) return t.size(0) > 1 ? t.stride(0) : 0;
    refuse(PyExc_ValueError, std::string(name) + " must be dense row-major or rows of a larger row-major array");
}
void shape(const at::Tensor& t, at::IntArrayRef want, const char* name) {
    if (t.sizes() != want)
        refuse(PyExc_ValueError, std::string(name) + " must be " + shape_of(want) + ", got " + shape_of(t.sizes()));
}
void* address(const at::Tensor* t) { return t && t->numel() > 0 ? t->data_ptr() : nullptr; }
void* address(const at::Tensor& t) { return address(&t); }

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType dt, c10::Device dev) {
    return at::empty(sizes, at::TensorOptions().dtype(dt).device(dev));
}

at::ScalarType type16(int64_t kind) { return kind == 0 ? at::kBFloat16 : at::kHalf; }
int float_code(const at::Tensor& t, const char* name) {
    switch (t.scalar_type()) {
        case at::kBFloat16: return 0;
        case at::kHalf: return 1;
        case at::kFloat: return 2;
        default:
            refuse(PyExc_TypeError, std::string(name) + " must be bf16, fp16 or fp32, got " +
                                        c10::toString(t.scalar_type()));
    }
}
bool gated(int64_t act) { return act >= GEMM_ACT_SWIGLU; }

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

PyObject* wrap(const at::Tensor& t) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) throw PythonError{};
    return o;
}
// A tuple of tensors (None for undefined ones).
PyObject* tuple(std::initializer_list<at::Tensor> ts) {
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
PyObject* entry(Py_ssize_t got, Py_ssize_t want, F f) {
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

struct ActShape {
    int64_t M, N, K, Nb;
};
ActShape act_shape(const at::Tensor& A, const at::Tensor& B, int64_t layout, int64_t act) {
    if (A.dim() != 2 || B.dim() != 2) refuse(PyExc_ValueError, "A and B must be 2-D");
    const bool a_t = layout >= GEMM_LAYOUT_TN, b_t = layout == GEMM_LAYOUT_NT || layout == GEMM_LAYOUT_TT;
    ActShape s;
    s.M = A.size(a_t ? 1 : 0);
    s.K = A.size(a_t ? 0 : 1);
    s.Nb = B.size(b_t ? 0 : 1);
    if (B.size(b_t ? 1 : 0) != s.K)
        refuse(PyExc_ValueError, "inner sizes differ: A is " + shape_of(A.sizes()) + ", B is " + shape_of(B.sizes()));
    if (gated(act) && s.Nb % 2)
        refuse(PyExc_ValueError, "a gated activation needs an even number of columns, got " + std::to_string(s.Nb));
    s.N = gated(act) ? s.Nb / 2 : s.Nb;
    return s;
}
void set_workspace(gemm_act_options* o, const at::Tensor* ws, c10::Device dev) {
    if (!ws) return;
    if (ws->device() != dev || !ws->is_contiguous())
        refuse(PyExc_ValueError, "workspace must be a contiguous CUDA tensor of the operands' device");
    o->workspace = ws->data_ptr();
    o->workspace_bytes = (uint64_t)ws->nbytes();
}

// (kind, activation, layout, A, B, C, bias, residual, preact, workspace, timeout_ns, fault, stream)
PyObject* py_gemm_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 13, [&]() -> PyObject* {
        const int64_t kind = integer(a[0]), act = integer(a[1]), layout = integer(a[2]);
        const at::ScalarType dt = type16(kind);
        const at::Tensor &A = tensor(a[3], "A"), &B = tensor(a[4], "B");
        const at::Tensor *Cin = maybe(a[5], "C"), *bias = maybe(a[6], "bias"),
                         *res = maybe(a[7], "residual"), *pre = maybe(a[8], "preact");
        const c10::Device dev = device_of(A, dt, "A");
        const OnStream on(dev, a[12]);
        gemm_act_options o = {};
        o.activation = (int)act;
        o.lda = matrix(A, dt, "A", dev);
        o.ldb = matrix(B, dt, "B", dev);
        const ActShape s = act_shape(A, B, layout, act);
        if (bias) {
            dense(*bias, dt, "bias", dev);
            shape(*bias, {s.Nb}, "bias");
            o.bias = address(bias);
        }
        if (res) {
            o.ld_residual = matrix(*res, dt, "residual", dev);
            shape(*res, {s.M, s.N}, "residual");
            o.residual = address(res);
        }
        if (pre) {
            o.ld_preact = matrix(*pre, dt, "preact", dev);
            shape(*pre, {s.M, s.Nb}, "preact");
            o.preact = address(pre);
        }
        set_workspace(&o, maybe(a[9], "workspace"), dev);
        o.timeout_ns = timeout(a[10]);
        o.fault_inject = small(a[11], "fault_inject");
        at::Tensor C;
        if (Cin) {
            o.ldc = matrix(*Cin, dt, "C", dev);
            shape(*Cin, {s.M, s.N}, "C");
            C = *Cin;
        } else {
            C = empty({s.M, s.N}, dt, dev);
        }
        on.call([&](dtc_stream_t st) {
            return gemm_act((int)kind, address(A), address(B), address(C), s.M, s.N, s.K, (int)layout, &o, st);
        });
        return wrap(C);
    });
}

// (kind, activation, layout, dC, A, B, preact, need_a, need_b, need_bias, workspace, timeout_ns, stream)
PyObject* py_gemm_act_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 13, [&]() -> PyObject* {
        const int64_t kind = integer(a[0]), act = integer(a[1]), layout = integer(a[2]);
        const at::ScalarType dt = type16(kind);
        const at::Tensor &dC = tensor(a[3], "dC"), &A = tensor(a[4], "A"), &B = tensor(a[5], "B");
        const at::Tensor* pre = maybe(a[6], "preact");
        const c10::Device dev = device_of(dC, dt, "dC");
        const OnStream on(dev, a[12]);
        gemm_act_options o = {};
        o.activation = (int)act;
        o.ldc = matrix(dC, dt, "dC", dev);
        o.lda = matrix(A, dt, "A", dev);
        o.ldb = matrix(B, dt, "B", dev);
        const ActShape s = act_shape(A, B, layout, act);
        shape(dC, {s.M, s.N}, "dC");
        if (act != GEMM_ACT_NONE) {
            if (!pre) refuse(PyExc_ValueError, "the gradient of an activation needs preact");
            o.ld_preact = matrix(*pre, dt, "preact", dev);
            shape(*pre, {s.M, s.Nb}, "preact");
            o.preact = address(pre);
        }
        set_workspace(&o, maybe(a[10], "workspace"), dev);
        o.timeout_ns = timeout(a[11]);
        at::Tensor dA, dB, db;
        if (a[7] == Py_True) dA = empty(A.sizes(), dt, dev);
        if (a[8] == Py_True) dB = empty(B.sizes(), dt, dev);
        if (a[9] == Py_True) db = empty({s.Nb}, at::kFloat, dev);
        auto out = [](const at::Tensor& t) { return t.defined() ? address(t) : nullptr; };
        on.call([&](dtc_stream_t st) {
            return gemm_act_backward((int)kind, address(dC), address(A), address(B), out(dA), out(dB),
                                     static_cast<float*>(out(db)), s.M, s.N, s.K, (int)layout, &o, st);
        });
        return tuple({dA, dB, db});
    });
}

moe_route_options route_options(PyObject* k, PyObject* scoring, PyObject* groups, PyObject* top,
                                PyObject* renorm, PyObject* scale) {
    moe_route_options o;
    o.top_k = small(k, "top_k");
    o.scoring = small(scoring, "scoring");
    o.groups = small(groups, "groups");
    o.top_groups = small(top, "top_groups");
    o.renormalize = PyObject_IsTrue(renorm) == 1;
    o.scale = (float)real(scale);
    return o;
}

// (logits, top_k, bias, scoring, groups, top_groups, renormalize, scale, weights, indices, stream)
PyObject* py_moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 11, [&]() -> PyObject* {
        const at::Tensor& z = tensor(a[0], "logits");
        const at::Tensor *bias = maybe(a[2], "bias"), *win = maybe(a[8], "weights"), *iin = maybe(a[9], "indices");
        const int code = float_code(z, "logits");
        const c10::Device dev = device_of(z, z.scalar_type(), "logits");
        const OnStream on(dev, a[10]);
        const int64_t ld = matrix(z, z.scalar_type(), "logits", dev);
        const moe_route_options o = route_options(a[1], a[3], a[4], a[5], a[6], a[7]);
        const int64_t T = z.size(0), E = z.size(1), k = o.top_k;
        if (bias) {
            dense(*bias, at::kFloat, "bias", dev);
            shape(*bias, {E}, "bias");
        }
        if (win) {
            dense(*win, at::kFloat, "weights", dev);
            shape(*win, {T, k}, "weights");
        }
        if (iin) {
            dense(*iin, at::kInt, "indices", dev);
            shape(*iin, {T, k}, "indices");
        }
        if (k < 0) refuse(PyExc_ValueError, "top_k must not be negative");
        const at::Tensor w = win ? *win : empty({T, k}, at::kFloat, dev);
        const at::Tensor i = iin ? *iin : empty({T, k}, at::kInt, dev);
        on.call([&](dtc_stream_t st) {
            return moe_route(code, address(z), ld, static_cast<const float*>(address(bias)), T, E, &o,
                             static_cast<float*>(address(w)), static_cast<int*>(address(i)), st);
        });
        return tuple({w, i});
    });
}

// (dweights, logits, indices, scoring, renormalize, scale, stream)
PyObject* py_moe_route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 7, [&]() -> PyObject* {
        const at::Tensor &dw = tensor(a[0], "dweights"), &z = tensor(a[1], "logits"), &idx = tensor(a[2], "indices");
        const int code = float_code(z, "logits");
        const c10::Device dev = device_of(z, z.scalar_type(), "logits");
        const OnStream on(dev, a[6]);
        const int64_t ld = matrix(z, z.scalar_type(), "logits", dev);
        dense(idx, at::kInt, "indices", dev);
        dense(dw, at::kFloat, "dweights", dev);
        if (idx.dim() != 2) refuse(PyExc_ValueError, "indices must be [T, k]");
        const int64_t T = z.size(0), E = z.size(1), k = idx.size(1);
        shape(idx, {T, k}, "indices");
        shape(dw, {T, k}, "dweights");
        moe_route_options o = {(int)k, small(a[3], "scoring"), 1, 1, PyObject_IsTrue(a[4]) == 1, (float)real(a[5])};
        const at::Tensor out = empty({T, E}, z.scalar_type(), dev);
        on.call([&](dtc_stream_t st) {
            return moe_route_backward(code, static_cast<const float*>(address(dw)), address(z), ld,
                                      static_cast<const int*>(address(idx)), T, E, &o, address(out), st);
        });
        return wrap(out);
    });
}

// (indices, experts, words of the plan, its first words of offsets, counts, slots and rows, rows,
// stream) to (plan, offsets, counts, slots, rows). The views are made before the launch: tensor
// bookkeeping right behind a launch costs several microseconds here, before it a fraction of one.
PyObject* py_moe_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 9, [&]() -> PyObject* {
        const at::Tensor& idx = tensor(a[0], "indices");
        const c10::Device dev = device_of(idx, at::kInt, "indices");
        const OnStream on(dev, a[8]);
        dense(idx, at::kInt, "indices", dev);
        if (idx.dim() != 2) refuse(PyExc_ValueError, "indices must be [T, k]");
        const int64_t E = integer(a[1]), T = idx.size(0), k = idx.size(1);
        const at::Tensor data = empty({integer(a[2])}, at::kInt, dev);
        PyObject* const r = tuple({data, data.as_strided({E + 1}, {1}, integer(a[3])),
                                   data.as_strided({E}, {1}, integer(a[4])),
                                   data.as_strided({T, k}, {k, 1}, integer(a[5])),
                                   data.as_strided({integer(a[7])}, {1}, integer(a[6]))});
        try {
            on.call([&](dtc_stream_t st) {
                return moe_plan(static_cast<const int*>(address(idx)), T, (int)k, E, data.data_ptr(), st);
            });
        } catch (...) {
            Py_DECREF(r);
            throw;
        }
        return r;
    });
}

struct ExpertsArgs {
    int64_t kind, T, k, E, H, F;
    at::ScalarType dt;
    const at::Tensor *x, *w_in, *w_out, *w, *plan;
    c10::Device dev{c10::kCPU};
    moe_experts_options o = {};
};
// (kind, activation, x or dy, w_in, w_out, weights, plan, the plan's tokens, top_k and experts, ...)
ExpertsArgs experts_args(PyObject* const* a, const char* name) {
    ExpertsArgs e;
    e.kind = integer(a[0]);
    e.dt = type16(e.kind);
    const int64_t act = integer(a[1]);
    e.x = &tensor(a[2], name);
    e.w_in = &tensor(a[3], "w_in");
    e.w_out = &tensor(a[4], "w_out");
    e.w = &tensor(a[5], "weights");
    e.plan = &tensor(a[6], "plan");
    e.dev = device_of(*e.x, e.dt, name);
    dense(*e.x, e.dt, name, e.dev);
    dense(*e.w_in, e.dt, "w_in", e.dev);
    dense(*e.w_out, e.dt, "w_out", e.dev);
    if (e.x->dim() != 2 || e.w_in->dim() != 3 || e.w_out->dim() != 3)
        refuse(PyExc_ValueError, std::string(name) + " must be [T, H], w_in [E, F, H] (gated [E, 2F, H]), w_out [E, H, F]");
    e.T = e.x->size(0);
    e.H = e.x->size(1);
    e.E = e.w_out->size(0);
    e.F = e.w_out->size(2);
    shape(*e.w_out, {e.E, e.H, e.F}, "w_out");
    shape(*e.w_in, {e.E, gated(act) ? 2 * e.F : e.F, e.H}, "w_in");
    e.k = integer(a[8]);
    if (integer(a[7]) != e.T || integer(a[9]) != e.E)
        refuse(PyExc_ValueError, "the plan is for " + std::to_string(integer(a[7])) + " tokens and " +
                                     std::to_string(integer(a[9])) + " experts, not " + std::to_string(e.T) +
                                     " and " + std::to_string(e.E));
    // (the kernels read the plan where its layout for these sizes says)
    moe_plan_info layout;
    const int status = moe_plan_layout(e.T, (int)e.k, e.E, &layout);
    if (status) throw LibraryError{status};
    dense(*e.plan, at::kInt, "the plan", e.dev);
    if (e.plan->numel() != layout.words)
        refuse(PyExc_ValueError, "the plan holds " + std::to_string(e.plan->numel()) + " words, not the " +
                                     std::to_string(layout.words) + " of a plan for these sizes");
    e.o.activation = (int)act;
    e.o.weights_dtype = float_code(*e.w, "weights");
    dense(*e.w, e.w->scalar_type(), "weights", e.dev);
    shape(*e.w, {e.T, e.k}, "weights");
    return e;
}

// (... as experts_args, residual, out, save, bytes of the buffer, timeout_ns, fault, stream)
PyObject* py_moe_experts(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 17, [&]() -> PyObject* {
        ExpertsArgs e = experts_args(a, "x");
        const OnStream on(e.dev, a[16]);
        const at::Tensor *res = maybe(a[10], "residual"), *oin = maybe(a[11], "out");
        if (res) {
            dense(*res, e.dt, "residual", e.dev);
            shape(*res, {e.T, e.H}, "residual");
            e.o.residual = address(res);
        }
        if (oin) {
            dense(*oin, e.dt, "out", e.dev);
            shape(*oin, {e.T, e.H}, "out");
        }
        const bool save = a[12] == Py_True;
        e.o.timeout_ns = timeout(a[14]);
        e.o.fault_inject = small(a[15], "fault_inject");
        const at::Tensor out = oin ? *oin : empty({e.T, e.H}, e.dt, e.dev);
        const at::Tensor buffer = empty({integer(a[13])}, at::kByte, e.dev);
        on.call([&](dtc_stream_t st) {
            return moe_experts((int)e.kind, address(e.x), address(e.w_in), address(e.w_out), address(e.w),
                               e.plan->data_ptr(), address(out), e.T, (int)e.k, e.E, e.H, e.F, &e.o, save,
                               address(buffer), st);
        });
        return save ? tuple({out, buffer}) : wrap(out);
    });
}

// (... as experts_args, saved, bytes of it, bytes of scratch, need_x, need_weights, timeout_ns, stream)
PyObject* py_moe_experts_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 17, [&]() -> PyObject* {
        ExpertsArgs e = experts_args(a, "dy");
        const OnStream on(e.dev, a[16]);
        const at::Tensor& saved = tensor(a[10], "saved");
        if (saved.scalar_type() != at::kByte || saved.numel() != integer(a[11]) || saved.device() != e.dev ||
            !saved.is_contiguous())
            refuse(PyExc_ValueError, "saved is not what moe_experts returned for these sizes with save=True");
        e.o.timeout_ns = timeout(a[15]);
        at::Tensor dx, dwi, dwo;
        if (a[13] == Py_True) dx = empty({e.T, e.H}, e.dt, e.dev);
        if (a[14] == Py_True) {
            dwi = empty(e.w_in->sizes(), e.dt, e.dev);
            dwo = empty(e.w_out->sizes(), e.dt, e.dev);
        }
        const at::Tensor dw = empty(e.w->sizes(), e.w->scalar_type(), e.dev);
        const int64_t bytes = integer(a[12]);
        const at::Tensor ws = empty({bytes}, at::kByte, e.dev);
        auto out = [](const at::Tensor& t) { return t.defined() ? address(t) : nullptr; };
        on.call([&](dtc_stream_t st) {
            return moe_experts_backward((int)e.kind, address(e.x), address(e.w_in), address(e.w_out), address(e.w),
                                        e.plan->data_ptr(), address(saved), out(dx), out(dwi), out(dwo), address(dw),
                                        e.T, (int)e.k, e.E, e.H, e.F, &e.o, address(ws), (uint64_t)bytes, st);
        });
        return tuple({dx, dwi, dwo, dw});
    });
}

PyObject* py_set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XSETREF(g_gemm_error, type);
    Py_RETURN_NONE;
}

#define DTC_FN(name) {#name, (PyCFunction)(void*)py_##name, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {DTC_FN(gemm_act),      DTC_FN(gemm_act_backward),
                          DTC_FN(moe_route),     DTC_FN(moe_route_backward),
                          DTC_FN(moe_plan),      DTC_FN(moe_experts),
                          DTC_FN(moe_experts_backward),
                          {"set_error", py_set_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_ffn_native", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__ffn_native() { return PyModule_Create(&kModule); }
