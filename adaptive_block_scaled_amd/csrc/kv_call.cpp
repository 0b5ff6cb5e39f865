// Calls of the KV cache's entry points for arguments that are in order: the
// checks of kv_cache.py, the allocation of results and the call, in a few
// microseconds less than Python takes (a decode step's calls are shorter than
// that).  Anything out of order returns None, and kv_cache.py then says what is
// wrong.  The entry points are those of the library that the binding loaded.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPStream.h>
#include <math.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/if4_kv.h"

namespace {

decltype(&if4_kv_append) kv_append;
decltype(&if4_kv_read) kv_read;
decltype(&if4_kv_attention) kv_attention;
decltype(&if4_kv_attention_workspace) kv_attention_workspace;

bool tensor(PyObject* o, at::Tensor& t) {
    if (!THPVariable_Check(o)) return false;
    t = THPVariable_Unpack(o);
    return t.is_cuda() && t.layout() == at::kStrided;
}

bool plain(PyObject* o, at::Tensor& t, at::ScalarType type, int64_t device, at::IntArrayRef shape) {
    return tensor(o, t) && t.scalar_type() == type && t.device().index() == device &&
           t.sizes() == shape && t.is_contiguous();
}

bool vectors(PyObject* o, at::Tensor& t, at::ScalarType type, int64_t device,
             at::IntArrayRef shape) {
    return tensor(o, t) && t.scalar_type() == type && t.device().index() == device &&
           t.sizes() == shape && t.stride(2) == 1;
}

bool integer(PyObject* o, int64_t& v) {
    if (!PyLong_Check(o)) return false;
    int overflow = 0;
    v = PyLong_AsLongLongAndOverflow(o, &overflow);
    return !overflow;
}

bool exponent(PyObject* o, int32_t& v) {
    int64_t x;
    if (!integer(o, x) || x < -64 || x > 64) return false;
    v = (int32_t)x;
    return true;
}

struct Cache {
    if4_kv_cache c;
    int64_t device;
    at::Tensor t[4];

    bool from(PyObject* o, PyObject* k_exp, PyObject* v_exp) {
        if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) return false;
        if (!exponent(k_exp, c.k_exp) || !exponent(v_exp, c.v_exp)) return false;
        if (!tensor(PyTuple_GET_ITEM(o, 0), t[0]) || t[0].dim() != 4) return false;
        device = t[0].device().index();
        c.pages = t[0].size(0);
        c.kv_heads = t[0].size(1);
        c.page_size = t[0].size(2);
        const int64_t d = c.head_dim = 2 * t[0].size(3);
        if ((d != 64 && d != 128 && d != 256) || c.page_size <= 0 || c.page_size % 16 ||
            c.kv_heads <= 0)
            return false;
        const int64_t tiles = c.page_size / 16;
        if (t[0].scalar_type() != at::kByte || !t[0].is_contiguous() ||
            !plain(PyTuple_GET_ITEM(o, 1), t[1], at::kByte, device,
                   {c.pages, c.kv_heads, c.page_size, d / 16}) ||
            !plain(PyTuple_GET_ITEM(o, 2), t[2], at::kByte, device,
                   {c.pages, c.kv_heads, tiles, 16, 16, d / 32}) ||
            !plain(PyTuple_GET_ITEM(o, 3), t[3], at::kByte, device,
                   {c.pages, c.kv_heads, tiles, d / 16, 16}))
            return false;
        c.k_codes = (uint8_t*)t[0].data_ptr();
        c.k_scales = (uint8_t*)t[1].data_ptr();
        c.v_codes = (uint8_t*)t[2].data_ptr();
        c.v_scales = (uint8_t*)t[3].data_ptr();
        return true;
    }
    void* stream() const {
        return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
    }
};

bool value_type(at::ScalarType s, int& dtype) {
    dtype = s == at::kFloat ? IF4_F32 : IF4_BF16;
    return s == at::kFloat || s == at::kBFloat16;
}

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

// append(cache, k, v, slots, k_exp, v_exp, mode) -> status | None
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Cache c;
        at::Tensor k, v, slots;
        int64_t mode;
        int dtype;
        if (n != 7 || !c.from(a[0], a[4], a[5]) || !tensor(a[1], k) || k.dim() != 3 ||
            !value_type(k.scalar_type(), dtype) || !integer(a[6], mode) || mode < 0 || mode > 2)
            Py_RETURN_NONE;
        const int64_t shape[3] = {k.size(0), c.c.kv_heads, c.c.head_dim};
        if (!vectors(a[1], k, k.scalar_type(), c.device, shape) ||
            !vectors(a[2], v, k.scalar_type(), c.device, shape) ||
            !plain(a[3], slots, at::kLong, c.device, {shape[0]}))
            Py_RETURN_NONE;
        return PyLong_FromLong(kv_append(&c.c, k.data_ptr(), v.data_ptr(), dtype, shape[0],
                                         k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                                         (const int64_t*)slots.data_ptr(), (int)mode, c.stream()));
    });
}

// read(cache, slots, k_exp, v_exp, bf16) -> (k, v) | status | None
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Cache c;
        at::Tensor slots;
        if (n != 5 || !c.from(a[0], a[2], a[3]) || !tensor(a[1], slots) || slots.dim() != 1 ||
            !plain(a[1], slots, at::kLong, c.device, slots.sizes()))
            Py_RETURN_NONE;
        const bool bf16 = a[4] == Py_True;
        const at::Tensor k = at::empty({slots.size(0), c.c.kv_heads, c.c.head_dim},
                                       slots.options().dtype(bf16 ? at::kBFloat16 : at::kFloat));
        const at::Tensor v = at::empty(k.sizes(), k.options());
        const int st = kv_read(&c.c, (const int64_t*)slots.data_ptr(), slots.size(0), k.data_ptr(),
                               v.data_ptr(), bf16 ? IF4_BF16 : IF4_F32, c.stream());
        if (st != IF4_OK) return PyLong_FromLong(st);
        PyObject* r = PyTuple_New(2);
        if (!r) return nullptr;
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(k));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(v));
        return r;
    });
}

// attention(q, cache, page_table, seq_lens, q_starts, max_q, max_len | None, scale | None, k_exp,
//           v_exp, causal, window, sinks) -> out | status | None
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Cache c;
        at::Tensor q, table, lens, starts;
        if4_kv_attention_args p;
        if (n != 13 || !c.from(a[1], a[8], a[9]) || !tensor(a[0], q) || q.dim() != 3 ||
            !vectors(a[0], q, at::kBFloat16, c.device, {q.size(0), q.size(1), c.c.head_dim}) ||
            !tensor(a[2], table) || table.dim() != 2)
            Py_RETURN_NONE;
        p.total_q = q.size(0);
        p.heads = q.size(1);
        p.batch = table.size(0);
        p.table_stride = table.size(1);
        if (p.heads == 0 || p.heads % c.c.kv_heads ||
            !plain(a[2], table, at::kInt, c.device, table.sizes()) ||
            !plain(a[3], lens, at::kInt, c.device, {p.batch}) ||
            !plain(a[4], starts, at::kInt, c.device, {p.batch + 1}))
            Py_RETURN_NONE;
        p.max_len = p.table_stride * c.c.page_size;
        double scale = 1.0 / sqrt((double)c.c.head_dim);
        if (a[7] != Py_None) {
            scale = PyFloat_Check(a[7]) ? PyFloat_AS_DOUBLE(a[7]) : -1.0;
        }
        if (!integer(a[5], p.max_q) || (a[6] != Py_None && !integer(a[6], p.max_len)) ||
            !(scale >= 0.0 && scale < 3e38) || !PyBool_Check(a[10]) || !integer(a[11], p.window) ||
            !integer(a[12], p.sinks) || p.window < 0 || p.sinks < 0)
            Py_RETURN_NONE;
        p.causal = a[10] == Py_True;
        if (!p.causal && (p.window || p.sinks)) Py_RETURN_NONE;
        p.scale = (float)scale;
        const at::Tensor out = at::empty(q.sizes(), q.options());
        p.q = q.data_ptr();
        p.out = out.data_ptr();
        p.q_stride_token = q.stride(0);
        p.q_stride_head = q.stride(1);
        p.out_stride_token = out.stride(0);
        p.out_stride_head = out.stride(1);
        p.page_table = (const int32_t*)table.data_ptr();
        p.seq_lens = (const int32_t*)lens.data_ptr();
        p.q_starts = (const int32_t*)starts.data_ptr();
        const int64_t need = kv_attention_workspace(&c.c, &p);
        if (need < 0) return PyLong_FromLong(-need);
        at::Tensor ws;
        if (need > 0) ws = at::empty({need}, q.options().dtype(at::kByte));
        const int st =
            kv_attention(&c.c, &p, need > 0 ? ws.data_ptr() : nullptr, need, c.stream());
        if (st != IF4_OK) return PyLong_FromLong(st);
        return THPVariable_Wrap(out);
    });
}

// bind(append, read, attention, workspace): the library's entry points, as addresses
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* f[4];
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "bind() takes four addresses");
        return nullptr;
    }
    for (int i = 0; i < 4; i++) {
        f[i] = PyLong_AsVoidPtr(a[i]);
        if (!f[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    kv_append = (decltype(kv_append))f[0];
    kv_read = (decltype(kv_read))f[1];
    kv_attention = (decltype(kv_attention))f[2];
    kv_attention_workspace = (decltype(kv_attention_workspace))f[3];
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"append", (PyCFunction)(void*)append, METH_FASTCALL, nullptr},
    {"read", (PyCFunction)(void*)read, METH_FASTCALL, nullptr},
    {"attention", (PyCFunction)(void*)attention, METH_FASTCALL, nullptr},
    {"bind", (PyCFunction)(void*)bind, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv_call", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv_call(void) { return PyModule_Create(&module); }
