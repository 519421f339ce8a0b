// fp4_binding.cpp -- the Python binding of the 4-bit operators (include/dtc_fp4.h), part of the module of
// ffn_binding.cpp. A matrix in 4 bits comes as the tuple that _fp4.Fp4 keeps.
#include "dtc_fp4.h"

#include <vector>

#include "binding.h"

namespace {

using namespace dtc_py;

// (codes, scales, row_scale or None, format, gated, matrices, rows, K). With scales None the first tensor
// holds all three, as buffers_of says: one allocation, and no views of it where nobody looks at them.
struct Held {
    fp4_matrix m = {};
    const at::Tensor *codes, *scales, *factors;
};
fp4_info layout_of(const fp4_matrix& m) {
    fp4_info l;
    const int status = fp4_layout(&m, &l);
    if (status) throw LibraryError{status};
    return l;
}
struct Buffers {
    int64_t scales, factors, bytes;  // byte offsets behind the codes
};
Buffers buffers_of(const fp4_matrix& m, const fp4_info& l) {
    auto up = [](uint64_t v) { return (int64_t)((v + 255) & ~(uint64_t)255); };
    Buffers b;
    b.scales = up(l.code_bytes);
    b.factors = b.scales + up(l.scale_bytes);
    b.bytes = b.factors + (m.format == FP4_NVFP4 ? m.matrices * m.rows * 4 : 0);
    return b;
}
void point_at(fp4_matrix* m, const at::Tensor& data, const Buffers& b) {
    if (data.numel() == 0) return;
    char* const p = static_cast<char*>(data.data_ptr());
    m->codes = p;
    m->scales = p + b.scales;
    m->row_scale = m->format == FP4_NVFP4 ? reinterpret_cast<float*>(p + b.factors) : nullptr;
}
Held held(PyObject* o, const char* name) {
    const std::string n(name);
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 8) refuse(PyExc_TypeError, n + " must be an Fp4");
    auto at = [&](int i) { return PyTuple_GET_ITEM(o, i); };
    Held h;
    h.codes = &tensor(at(0), name);
    h.scales = maybe(at(1), name);
    h.factors = maybe(at(2), name);
    h.m.format = small(at(3), "format");
    h.m.gated = small(at(4), "gated");
    h.m.matrices = integer(at(5));
    h.m.rows = integer(at(6));
    h.m.K = integer(at(7));
    const c10::Device dev = device_of(*h.codes, at::kByte, name);
    const fp4_info l = layout_of(h.m);
    dense(*h.codes, at::kByte, name, dev);
    if (!h.scales) {
        const Buffers b = buffers_of(h.m, l);
        if (h.codes->numel() != b.bytes) refuse(PyExc_ValueError, n + " is not what quantize_fp4 made");
        point_at(&h.m, *h.codes, b);
        return h;
    }
    dense(*h.scales, at::kByte, (n + ".scales").c_str(), dev);
    if ((uint64_t)h.codes->numel() != l.code_bytes || (uint64_t)h.scales->numel() != l.scale_bytes)
        refuse(PyExc_ValueError, n + ": codes and scales hold " + std::to_string(h.codes->numel()) + " and " +
                                     std::to_string(h.scales->numel()) + " bytes, not " + std::to_string(l.code_bytes) +
                                     " and " + std::to_string(l.scale_bytes));
    if (h.factors) {
        dense(*h.factors, at::kFloat, (n + ".row_scale").c_str(), dev);
        if (h.factors->numel() != h.m.matrices * h.m.rows)
            refuse(PyExc_ValueError, n + ".row_scale must hold one factor per row");
    }
    h.m.codes = address(h.codes);
    h.m.scales = address(h.scales);
    h.m.row_scale = static_cast<float*>(address(h.factors));
    return h;
}
void on_device(const Held& h, const char* name, c10::Device dev) {
    base(*h.codes, at::kByte, name, dev);
}

// Matrices, rows and K of a tensor [rows, K] or [matrices, rows, K]; its leading dimension.
int64_t stack(const at::Tensor& x, at::ScalarType dt, const char* name, c10::Device dev, fp4_matrix* m) {
    int64_t ld = 0;
    if (x.dim() == 3)
        dense(x, dt, name, dev);
    else if (x.dim() == 2)
        ld = matrix(x, dt, name, dev);
    else
        refuse(PyExc_ValueError, std::string(name) + " must be [rows, K] or [matrices, rows, K]");
    m->matrices = x.dim() == 3 ? x.size(0) : 1;
    m->rows = x.size(-2);
    m->K = x.size(-1);
    return ld;
}

// (x, format, gated, out or None, stream) to (the tensor of codes, scales and factors, matrices, rows, K)
PyObject* py_quantize_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 5, [&]() -> PyObject* {
        const at::Tensor& x = tensor(a[0], "x");
        const int code = float_code(x, "x");
        if (code == 2) refuse(PyExc_TypeError, "x must be bf16 or fp16");
        const c10::Device dev = device_of(x, x.scalar_type(), "x");
        const OnStream on(dev, a[4]);
        fp4_matrix m = {};
        const int64_t ld = stack(x, x.scalar_type(), "x", dev, &m);
        m.format = small(a[1], "format");
        m.gated = small(a[2], "gated");
        at::Tensor data;
        if (a[3] != Py_None) {
            const Held h = held(a[3], "out");
            on_device(h, "out", dev);
            if (h.m.format != m.format || h.m.gated != m.gated || h.m.matrices != m.matrices || h.m.rows != m.rows ||
                h.m.K != m.K)
                refuse(PyExc_ValueError, "out is of another shape, format or order");
            if (h.scales && (h.factors != nullptr) != (m.format == FP4_NVFP4))
                refuse(PyExc_ValueError, "out must have row factors in NVFP4 and only there");
            m = h.m;
            data = *h.codes;
        } else {
            const Buffers b = buffers_of(m, layout_of(m));
            data = empty({b.bytes}, at::kByte, dev);
            point_at(&m, data, b);
        }
        on.call([&](dtc_stream_t st) { return fp4_quantize(code, address(x), ld, &m, st); });
        PyObject* const t = wrap(data);
        PyObject* const r = Py_BuildValue("NLLL", t, (long long)m.matrices, (long long)m.rows, (long long)m.K);
        if (!r) throw PythonError{};
        return r;
    });
}

// (data, format, gated, matrices, rows, K) to the codes, scales and factors in it: views
PyObject* py_fp4_views(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 7, [&]() -> PyObject* {
        const at::Tensor& data = tensor(a[0], "data");
        fp4_matrix m = {};
        m.format = small(a[1], "format");
        m.gated = small(a[2], "gated");
        m.matrices = integer(a[3]);
        m.rows = integer(a[4]);
        m.K = integer(a[5]);
        const fp4_info l = layout_of(m);
        const Buffers b = buffers_of(m, l);
        const bool three = a[6] == Py_True;
        const std::vector<int64_t> rows = three ? std::vector<int64_t>{m.matrices, m.rows} : std::vector<int64_t>{m.rows};
        std::vector<int64_t> codes = rows;
        codes.push_back(m.K / 2);
        at::Tensor f;
        if (m.format == FP4_NVFP4) f = data.narrow(0, b.factors, b.bytes - b.factors).view(at::kFloat).view(rows);
        return tuple({data.narrow(0, 0, (int64_t)l.code_bytes).view(codes),
                      data.narrow(0, b.scales, (int64_t)l.scale_bytes), f});
    });
}

// (q, dtype code, out or None, 3-D, stream)
PyObject* py_dequantize_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 5, [&]() -> PyObject* {
        const Held h = held(a[0], "q");
        const c10::Device dev = h.codes->device();
        const OnStream on(dev, a[4]);
        const int code = small(a[1], "dtype");
        const at::ScalarType dt = code == 0 ? at::kBFloat16 : code == 1 ? at::kHalf : at::kFloat;
        const std::vector<int64_t> size = a[3] == Py_True ? std::vector<int64_t>{h.m.matrices, h.m.rows, h.m.K}
                                                          : std::vector<int64_t>{h.m.rows, h.m.K};
        const at::Tensor* oin = maybe(a[2], "out");
        if (oin) {
            dense(*oin, dt, "out", dev);
            shape(*oin, size, "out");
        }
        const at::Tensor out = oin ? *oin : empty(size, dt, dev);
        on.call([&](dtc_stream_t st) { return fp4_dequantize(code, &h.m, address(out), st); });
        return wrap(out);
    });
}

// (scales, matrices, rows, K, format, gated, stream) to the scales in the tensor cores' order
PyObject* py_pack_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 7, [&]() -> PyObject* {
        const at::Tensor& s = tensor(a[0], "scales");
        const c10::Device dev = device_of(s, at::kByte, "scales");
        const OnStream on(dev, a[6]);
        dense(s, at::kByte, "scales", dev);
        fp4_matrix m = {};
        m.matrices = integer(a[1]);
        m.rows = integer(a[2]);
        m.K = integer(a[3]);
        m.format = small(a[4], "format");
        m.gated = small(a[5], "gated");
        const fp4_info l = layout_of(m);
        if (s.numel() != m.matrices * m.rows * (m.K / (m.format == FP4_NVFP4 ? 16 : 32)))
            refuse(PyExc_ValueError, "scales must hold one byte per block");
        const at::Tensor out = empty({(int64_t)l.scale_bytes}, at::kByte, dev);
        m.scales = address(out);
        on.call([&](dtc_stream_t st) { return fp4_pack_scales(address(s), &m, st); });
        return wrap(out);
    });
}

// (kind, activation, A, B, C, bias, residual, workspace, tile_rows, split_k, timeout_ns, fault, stream)
PyObject* py_gemm_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 13, [&]() -> PyObject* {
        const int64_t kind = integer(a[0]), act = integer(a[1]);
        const at::ScalarType dt = type16(kind);
        const Held A = held(a[2], "A"), B = held(a[3], "B");
        const c10::Device dev = A.codes->device();
        on_device(B, "B", dev);
        const OnStream on(dev, a[12]);
        if (A.m.matrices != 1 || B.m.matrices != 1) refuse(PyExc_ValueError, "A and B must be one matrix each");
        if (A.m.K != B.m.K)
            refuse(PyExc_ValueError, "inner sizes differ: " + std::to_string(A.m.K) + " and " + std::to_string(B.m.K));
        const int64_t M = A.m.rows, Nb = B.m.rows, N = gated(act) ? Nb / 2 : Nb;
        const at::Tensor *Cin = maybe(a[4], "C"), *bias = maybe(a[5], "bias"), *res = maybe(a[6], "residual"),
                         *ws = maybe(a[7], "workspace");
        gemm_fp4_options o = {};
        o.activation = (int)act;
        if (bias) {
            dense(*bias, dt, "bias", dev);
            shape(*bias, {Nb}, "bias");
            o.bias = address(bias);
        }
        if (res) {
            o.ld_residual = matrix(*res, dt, "residual", dev);
            shape(*res, {M, N}, "residual");
            o.residual = address(res);
        }
        if (ws) {
            if (ws->device() != dev || !ws->is_contiguous())
                refuse(PyExc_ValueError, "workspace must be a contiguous CUDA tensor of the operands' device");
            o.workspace = ws->data_ptr();
            o.workspace_bytes = (uint64_t)ws->nbytes();
        }
        o.tile_rows = small(a[8], "tile_rows");
        o.split_k = small(a[9], "split_k");
        o.timeout_ns = timeout(a[10]);
        o.fault_inject = small(a[11], "fault_inject");
        at::Tensor C;
        if (Cin) {
            o.ldc = matrix(*Cin, dt, "C", dev);
            shape(*Cin, {M, N}, "C");
            C = *Cin;
        } else {
            C = empty({M, N}, dt, dev);
        }
        on.call([&](dtc_stream_t st) { return gemm_fp4((int)kind, &A.m, &B.m, address(C), &o, st); });
        return wrap(C);
    });
}

// (kind, activation, x, w_in, w_out, weights, plan, the plan's tokens, top_k and experts, residual, out, bytes
// of the buffer, timeout_ns, fault, stream)
PyObject* py_moe_experts_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return entry(n, 16, [&]() -> PyObject* {
        const int64_t kind = integer(a[0]), act = integer(a[1]);
        const at::ScalarType dt = type16(kind);
        const at::Tensor& x = tensor(a[2], "x");
        const c10::Device dev = device_of(x, dt, "x");
        const Held wi = held(a[3], "w_in"), wo = held(a[4], "w_out");
        on_device(wi, "w_in", dev);
        on_device(wo, "w_out", dev);
        const at::Tensor &w = tensor(a[5], "weights"), &plan = tensor(a[6], "plan");
        const OnStream on(dev, a[15]);
        dense(x, dt, "x", dev);
        if (x.dim() != 2) refuse(PyExc_ValueError, "x must be [T, H]");
        const int64_t T = x.size(0), H = x.size(1), E = wo.m.matrices, F = wo.m.K, k = integer(a[8]);
        if (wi.m.matrices != E || wi.m.K != H || wo.m.rows != H || wi.m.rows != (gated(act) ? 2 * F : F))
            refuse(PyExc_ValueError, "w_in must be [E, F, H] (gated [E, 2F, H]) and w_out [E, H, F] for x [T, H]");
        if (integer(a[7]) != T || integer(a[9]) != E)
            refuse(PyExc_ValueError, "the plan is for " + std::to_string(integer(a[7])) + " tokens and " +
                                         std::to_string(integer(a[9])) + " experts, not " + std::to_string(T) +
                                         " and " + std::to_string(E));
        // (the kernels read the plan where its layout for these sizes says)
        moe_plan_info layout;
        const int status = moe_plan_layout(T, (int)k, E, &layout);
        if (status) throw LibraryError{status};
        dense(plan, at::kInt, "the plan", dev);
        if (plan.numel() != layout.words)
            refuse(PyExc_ValueError, "the plan holds " + std::to_string(plan.numel()) + " words, not the " +
                                         std::to_string(layout.words) + " of a plan for these sizes");
        moe_experts_options o = {};
        o.activation = (int)act;
        o.weights_dtype = float_code(w, "weights");
        dense(w, w.scalar_type(), "weights", dev);
        shape(w, {T, k}, "weights");
        const at::Tensor *res = maybe(a[10], "residual"), *oin = maybe(a[11], "out");
        if (res) {
            dense(*res, dt, "residual", dev);
            shape(*res, {T, H}, "residual");
            o.residual = address(res);
        }
        if (oin) {
            dense(*oin, dt, "out", dev);
            shape(*oin, {T, H}, "out");
        }
        o.timeout_ns = timeout(a[13]);
        o.fault_inject = small(a[14], "fault_inject");
        const int64_t bytes = integer(a[12]);
        const at::Tensor out = oin ? *oin : empty({T, H}, dt, dev);
        const at::Tensor buffer = empty({bytes}, at::kByte, dev);
        on.call([&](dtc_stream_t st) {
            return moe_experts_fp4((int)kind, address(x), &wi.m, &wo.m, address(w), plan.data_ptr(), address(out), T,
                                   (int)k, &o, address(buffer), (uint64_t)bytes, st);
        });
        return wrap(out);
    });
}

}  // namespace

namespace dtc_py {
PyMethodDef kFp4Methods[] = {DTC_FN(quantize_fp4), DTC_FN(fp4_views), DTC_FN(dequantize_fp4), DTC_FN(pack_fp4),
                             DTC_FN(gemm_fp4),     DTC_FN(moe_experts_fp4), {nullptr, nullptr, 0, nullptr}};
}  // namespace dtc_py
