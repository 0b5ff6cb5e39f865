// Calls of the FP8 product and of the norm and rotation of q and k for arguments that are
// in order, as kv_call.cpp has them for the KV cache: the checks of fp8.py and qk.py, the
// allocation of results and the call, in a few microseconds less than Python takes.
// Anything out of order returns None, and the Python side then says what is wrong.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <math.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "../../include/if4_fp8.h"
#include "../../include/if4_qk.h"

namespace {

decltype(&if4_fp8_quantize) fp8_quantize;
decltype(&if4_fp8_quantize_t) fp8_quantize_t;
decltype(&if4_fp8_gemm) fp8_gemm;
decltype(&if4_fp8_gemm_workspace) fp8_gemm_workspace;
decltype(&if4_norm_rotate) qk_norm_rotate;
decltype(&if4_norm_rotate_backward) qk_backward;
decltype(&if4_norm_rotate_backward_workspace) qk_backward_workspace;

bool tensor(PyObject* o, at::Tensor& t) {
    if (!THPVariable_Check(o)) return false;
    t = THPVariable_Unpack(o);
    return t.is_cuda() && t.layout() == at::kStrided;
}

bool plain(PyObject* o, at::Tensor& t, at::ScalarType type, int64_t device, at::IntArrayRef shape) {
    return tensor(o, t) && t.scalar_type() == type && t.device().index() == device &&
           t.sizes() == shape && t.is_contiguous();
}

bool value_type(at::ScalarType s, int& dtype) {
    dtype = s == at::kFloat ? IF4_F32 : IF4_BF16;
    return s == at::kFloat || s == at::kBFloat16;
}

void* stream_of(int64_t device) {
    return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
}

// The tensors' device is the current one for the time of a call: its default stream is a
// null handle, which HIP takes as the default stream of the current device.
struct On {
    std::optional<c10::hip::HIPGuard> guard;
    explicit On(int64_t device) {
        static const bool one = c10::hip::device_count() == 1;
        if (!one && c10::hip::current_device() != device) guard.emplace((c10::DeviceIndex)device);
    }
};

int64_t blocks(int64_t n) { return (n + IF4_FP8_BLOCK - 1) / IF4_FP8_BLOCK; }

// What a call gives: the result, the status that the binding raises, or None.
template <typename F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (...) {
        // (a C++ exception, out of memory say: the Python way meets and raises it again)
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(a));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(b));
    return r;
}

// quantize(x, square, transposed) -> (codes, scales) | status | None
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        at::Tensor x;
        int dtype;
        if (n != 3 || !tensor(a[0], x) || x.dim() != 2 || x.stride(1) != 1 ||
            (x.size(0) > 1 && x.stride(0) < x.size(1)) || !value_type(x.scalar_type(), dtype) ||
            !PyBool_Check(a[1]) || !PyBool_Check(a[2]))
            Py_RETURN_NONE;
        const bool square = a[1] == Py_True, t = a[2] == Py_True;
        const int64_t rows = x.size(t), k = x.size(!t);
        const auto bytes = x.options().dtype(at::kByte);
        const at::Tensor codes = at::empty({rows, k}, bytes);
        const at::Tensor scales = at::empty({square ? blocks(rows) : rows, blocks(k)}, bytes);
        // (one row is none apart from another: its stride has any value)
        const int64_t ld = x.size(0) > 1 ? x.stride(0) : x.size(1);
        const On on(x.device().index());
        const int st = (t ? fp8_quantize_t : fp8_quantize)(
            x.data_ptr(), dtype, x.size(0), x.size(1), ld, square, (uint8_t*)codes.data_ptr(),
            (uint8_t*)scales.data_ptr(), stream_of(x.device().index()));
        if (st != IF4_OK) return PyLong_FromLong(st);
        return pair(codes, scales);
    });
}

// gemm(a_codes, a_scales, w_codes, w_scales, bf16) -> C | status | None
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        at::Tensor ac, as, wc, ws;
        if (n != 5 || !tensor(a[0], ac) || ac.dim() != 2 || !tensor(a[2], wc) || wc.dim() != 2 ||
            !tensor(a[3], ws) || ws.dim() != 2 || !PyBool_Check(a[4]))
            Py_RETURN_NONE;
        const int64_t m = ac.size(0), k = ac.size(1), rows = wc.size(0), device = ac.device().index();
        const bool square = ws.size(0) != rows, bf16 = a[4] == Py_True;
        if (!plain(a[0], ac, at::kByte, device, {m, k}) || !plain(a[1], as, at::kByte, device, {m, blocks(k)}) ||
            !plain(a[2], wc, at::kByte, device, {rows, k}) ||
            !plain(a[3], ws, at::kByte, device, {square ? blocks(rows) : rows, blocks(k)}))
            Py_RETURN_NONE;
        const int64_t need = fp8_gemm_workspace(m, rows, k);
        if (need < 0) return PyLong_FromLong(-need);
        const at::Tensor c = at::empty({m, rows}, ac.options().dtype(bf16 ? at::kBFloat16 : at::kFloat));
        at::Tensor work;
        if (need > 0) work = at::empty({need}, ac.options());
        const On on(device);
        const int st = fp8_gemm((const uint8_t*)ac.data_ptr(), (const uint8_t*)as.data_ptr(),
                                (const uint8_t*)wc.data_ptr(), (const uint8_t*)ws.data_ptr(), square, m, rows, k,
                                c.data_ptr(), bf16 ? IF4_BF16 : IF4_F32, rows, need > 0 ? work.data_ptr() : nullptr,
                                need, stream_of(device));
        if (st != IF4_OK) return PyLong_FromLong(st);
        return THPVariable_Wrap(c);
    });
}

bool vectors(PyObject* o, if4_qk_part& p, at::Tensor& x, at::ScalarType type, int64_t device, int64_t tokens,
             int64_t dim) {
    if (!tensor(o, x) || x.dim() != 3 || x.scalar_type() != type || x.device().index() != device ||
        x.size(0) != tokens || x.size(2) != dim || x.stride(2) != 1)
        return false;
    p.x = x.data_ptr();
    p.x_stride_token = tokens > 1 ? x.stride(0) : 0;
    p.x_stride_head = x.size(1) > 1 ? x.stride(1) : 0;
    p.heads = x.size(1);
    return true;
}

// What the forward and the backward pass are both given, and the tensors that hold it.
struct Rotation {
    if4_qk_args p = {};
    at::Tensor q, k, qw, kw, table, positions;
    int64_t device;

    // a: q, k, q_weight, k_weight, table, positions, eps, interleaved
    bool from(PyObject* const* a) {
        int dtype;
        if (!tensor(a[0], q) || q.dim() != 3 || !value_type(q.scalar_type(), dtype) || !tensor(a[4], table) ||
            table.dim() != 2 || !PyFloat_Check(a[6]) || !PyBool_Check(a[7]))
            return false;
        const int64_t tokens = q.size(0), dim = q.size(2);
        device = q.device().index();
        const double eps = PyFloat_AS_DOUBLE(a[6]);
        if (!vectors(a[0], p.q, q, q.scalar_type(), device, tokens, dim) ||
            !vectors(a[1], p.k, k, q.scalar_type(), device, tokens, dim) ||
            !plain(a[2], qw, at::kFloat, device, {dim}) || !plain(a[3], kw, at::kFloat, device, {dim}) ||
            !plain(a[4], table, at::kFloat, device, table.sizes()) ||
            !plain(a[5], positions, at::kLong, device, {tokens}) || !(eps >= 0.0 && eps < 3e38))
            return false;
        p.q.weight = (const float*)qw.data_ptr();
        p.k.weight = (const float*)kw.data_ptr();
        p.table = (const float*)table.data_ptr();
        p.positions = (const int64_t*)positions.data_ptr();
        p.tokens = tokens;
        p.head_dim = dim;
        p.rotary = table.size(1);
        p.table_rows = table.size(0);
        p.eps = (float)eps;
        p.interleaved = a[7] == Py_True;
        p.dtype = dtype;
        return true;
    }
    // results of q's and k's shapes
    void into(if4_qk_part& part, const at::Tensor& y) {
        part.y = y.data_ptr();
        part.y_stride_token = part.heads * p.head_dim;
        part.y_stride_head = p.head_dim;
    }
};

// norm_rotate(q, k, q_weight, k_weight, table, positions, eps, interleaved, bf16) -> (q, k) | status | None
PyObject* norm_rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Rotation r;
        if (n != 9 || !PyBool_Check(a[8]) || !r.from(a)) Py_RETURN_NONE;
        const bool bf16 = a[8] == Py_True;
        const auto like = r.q.options().dtype(bf16 ? at::kBFloat16 : at::kFloat);
        const at::Tensor qo = at::empty(r.q.sizes(), like), ko = at::empty(r.k.sizes(), like);
        r.into(r.p.q, qo);
        r.into(r.p.k, ko);
        r.p.out_dtype = bf16 ? IF4_BF16 : IF4_F32;
        const On on(r.device);
        const int st = qk_norm_rotate(&r.p, stream_of(r.device));
        if (st != IF4_OK) return PyLong_FromLong(st);
        return pair(qo, ko);
    });
}

// norm_rotate_backward(dq, dk, q, k, q_weight, k_weight, table, positions, eps, interleaved)
//     -> (q's, k's, q_weight's, k_weight's gradients) | status | None
PyObject* norm_rotate_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Rotation r;
        at::Tensor g[2];
        if (n != 10 || !r.from(a + 2) || !tensor(a[0], g[0]) || g[0].dim() != 3 ||
            !value_type(g[0].scalar_type(), r.p.out_dtype) || r.p.q.heads == 0 || r.p.k.heads == 0)
            Py_RETURN_NONE;
        if4_qk_part* const parts[2] = {&r.p.q, &r.p.k};
        for (int i = 0; i < 2; i++) {
            if4_qk_part like = {};
            if (!vectors(a[i], like, g[i], g[0].scalar_type(), r.device, r.p.tokens, r.p.head_dim) ||
                like.heads != parts[i]->heads)
                Py_RETURN_NONE;
            parts[i]->g = like.x;
            parts[i]->g_stride_token = like.x_stride_token;
            parts[i]->g_stride_head = like.x_stride_head;
        }
        const at::Tensor dq = at::empty(r.q.sizes(), r.q.options()), dk = at::empty(r.k.sizes(), r.k.options());
        const auto floats = r.q.options().dtype(at::kFloat);
        const at::Tensor dqw = at::empty({r.p.head_dim}, floats), dkw = at::empty({r.p.head_dim}, floats);
        r.into(r.p.q, dq);
        r.into(r.p.k, dk);
        r.p.q.d_weight = (float*)dqw.data_ptr();
        r.p.k.d_weight = (float*)dkw.data_ptr();
        const int64_t need = qk_backward_workspace(&r.p);
        if (need < 0) return PyLong_FromLong(-need);
        const at::Tensor work = at::empty({need}, r.q.options().dtype(at::kByte));
        const On on(r.device);
        const int st = qk_backward(&r.p, work.data_ptr(), need, stream_of(r.device));
        if (st != IF4_OK) return PyLong_FromLong(st);
        PyObject* t = PyTuple_New(4);
        if (!t) return nullptr;
        const at::Tensor* const results[4] = {&dq, &dk, &dqw, &dkw};
        for (int i = 0; i < 4; i++) PyTuple_SET_ITEM(t, i, THPVariable_Wrap(*results[i]));
        return t;
    });
}

// The library's entry points, as addresses.
bool addresses(PyObject* const* a, Py_ssize_t n, void** f, Py_ssize_t want) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of addresses");
        return false;
    }
    for (Py_ssize_t i = 0; i < n; i++) {
        f[i] = PyLong_AsVoidPtr(a[i]);
        if (!f[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return false;
        }
    }
    return true;
}

// bind_fp8(quantize, quantize_t, gemm, gemm_workspace)
PyObject* bind_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* f[4];
    if (!addresses(a, n, f, 4)) return nullptr;
    fp8_quantize = (decltype(fp8_quantize))f[0];
    fp8_quantize_t = (decltype(fp8_quantize_t))f[1];
    fp8_gemm = (decltype(fp8_gemm))f[2];
    fp8_gemm_workspace = (decltype(fp8_gemm_workspace))f[3];
    Py_RETURN_NONE;
}

// bind_qk(norm_rotate, norm_rotate_backward, its workspace)
PyObject* bind_qk(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* f[3];
    if (!addresses(a, n, f, 3)) return nullptr;
    qk_norm_rotate = (decltype(qk_norm_rotate))f[0];
    qk_backward = (decltype(qk_backward))f[1];
    qk_backward_workspace = (decltype(qk_backward_workspace))f[2];
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"quantize", (PyCFunction)(void*)quantize, METH_FASTCALL, nullptr},
    {"gemm", (PyCFunction)(void*)gemm, METH_FASTCALL, nullptr},
    {"norm_rotate", (PyCFunction)(void*)norm_rotate, METH_FASTCALL, nullptr},
    {"norm_rotate_backward", (PyCFunction)(void*)norm_rotate_backward, METH_FASTCALL, nullptr},
    {"bind_fp8", (PyCFunction)(void*)bind_fp8, METH_FASTCALL, nullptr},
    {"bind_qk", (PyCFunction)(void*)bind_qk, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_op_call", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__op_call(void) { return PyModule_Create(&module); }
