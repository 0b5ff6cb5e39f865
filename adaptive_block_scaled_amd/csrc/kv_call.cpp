// Calls of the KV cache's entry points for arguments that are in order: the
// checks of kv_cache.py and kv_evict.py, the allocation of results and the call, in a few
// microseconds less than Python takes (a decode step's calls are shorter than
// that).  Anything out of order returns None, and the Python side then says what is
// wrong.  The entry points are those of the library that the binding loaded.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <math.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "../../include/if4_kv.h"
#include "../../include/if4_kv_evict.h"

namespace {

decltype(&if4_kv_append) kv_append;
decltype(&if4_kv_read) kv_read;
decltype(&if4_kv_attention) kv_attention;
decltype(&if4_kv_attention_workspace) kv_attention_workspace;
decltype(&if4_kv_weights) kv_weights;
decltype(&if4_kv_weights_workspace) kv_weights_workspace;
decltype(&if4_kv_select) kv_select;
decltype(&if4_kv_select_workspace) kv_select_workspace;
decltype(&if4_kv_compact) kv_compact;

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
    void* stream() const { return stream_of(device); }
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
        const On on(c.device);
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
        const On on(c.device);
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

// What attention and the sums of its weights are both given, and the tensors that hold it.
struct Batch {
    Cache c;
    at::Tensor q, table, lens, starts;
    if4_kv_attention_args p = {};

    // a: q, cache, page_table, seq_lens, q_starts, max_q, max_len | None, scale | None, causal, window, sinks
    bool from(PyObject* const* a, PyObject* k_exp, PyObject* v_exp) {
        if (!c.from(a[1], k_exp, v_exp) || !tensor(a[0], q) || q.dim() != 3 ||
            !vectors(a[0], q, at::kBFloat16, c.device, {q.size(0), q.size(1), c.c.head_dim}) ||
            !tensor(a[2], table) || table.dim() != 2)
            return false;
        p.total_q = q.size(0);
        p.heads = q.size(1);
        p.batch = table.size(0);
        p.table_stride = table.size(1);
        if (p.heads == 0 || p.heads % c.c.kv_heads ||
            !plain(a[2], table, at::kInt, c.device, table.sizes()) ||
            !plain(a[3], lens, at::kInt, c.device, {p.batch}) ||
            !plain(a[4], starts, at::kInt, c.device, {p.batch + 1}))
            return false;
        p.max_len = p.table_stride * c.c.page_size;
        double scale = 1.0 / sqrt((double)c.c.head_dim);
        if (a[7] != Py_None) {
            scale = PyFloat_Check(a[7]) ? PyFloat_AS_DOUBLE(a[7]) : -1.0;
        }
        if (!integer(a[5], p.max_q) || (a[6] != Py_None && !integer(a[6], p.max_len)) ||
            !(scale >= 0.0 && scale < 3e38) || !PyBool_Check(a[8]) || !integer(a[9], p.window) ||
            !integer(a[10], p.sinks) || p.window < 0 || p.sinks < 0)
            return false;
        p.causal = a[8] == Py_True;
        if (!p.causal && (p.window || p.sinks)) return false;
        p.scale = (float)scale;
        p.q = q.data_ptr();
        p.q_stride_token = q.stride(0);
        p.q_stride_head = q.stride(1);
        p.page_table = (const int32_t*)table.data_ptr();
        p.seq_lens = (const int32_t*)lens.data_ptr();
        p.q_starts = (const int32_t*)starts.data_ptr();
        return true;
    }
};

// attention(q, cache, page_table, seq_lens, q_starts, max_q, max_len | None, scale | None, k_exp,
//           v_exp, causal, window, sinks) -> out | status | None
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Batch b;
        if (n != 13) Py_RETURN_NONE;
        PyObject* const args[11] = {a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[10], a[11], a[12]};
        if (!b.from(args, a[8], a[9])) Py_RETURN_NONE;
        if4_kv_attention_args& p = b.p;
        const at::Tensor out = at::empty(b.q.sizes(), b.q.options());
        p.out = out.data_ptr();
        p.out_stride_token = out.stride(0);
        p.out_stride_head = out.stride(1);
        const int64_t need = kv_attention_workspace(&b.c.c, &p);
        if (need < 0) return PyLong_FromLong(-need);
        at::Tensor ws;
        if (need > 0) ws = at::empty({need}, b.q.options().dtype(at::kByte));
        const On on(b.c.device);
        const int st =
            kv_attention(&b.c.c, &p, need > 0 ? ws.data_ptr() : nullptr, need, b.c.stream());
        if (st != IF4_OK) return PyLong_FromLong(st);
        return THPVariable_Wrap(out);
    });
}

// [sequences, kv_heads, width] fp32 sums with unit stride along the last dim
bool sums(PyObject* o, at::Tensor& t, int64_t device) {
    return tensor(o, t) && t.dim() == 3 && t.scalar_type() == at::kFloat && t.device().index() == device &&
           t.stride(2) == 1;
}

// rows of sums that do not overlap: strides as of some order of sequences and heads
bool apart(const at::Tensor& t) {
    const int64_t n = t.size(0), h = t.size(1), w = t.size(2), sn = t.stride(0), sh = t.stride(1);
    return (n <= 1 || sn >= w) && (h <= 1 || sh >= w) &&
           (n <= 1 || h <= 1 || sn >= sh * (h - 1) + w || sh >= sn * (n - 1) + w);
}

// mass, out | None and rows | None
struct Mass {
    if4_kv_mass m = {};
    at::Tensor in, out, rows;

    bool from(PyObject* mass, PyObject* to, PyObject* at_rows, int64_t batch, int64_t device) {
        if (!sums(mass, in, device)) return false;
        m.in = (const float*)in.data_ptr();
        m.in_stride_row = in.stride(0);
        m.in_stride_head = in.stride(1);
        m.mass_rows = in.size(0);
        m.width = in.size(2);
        if (to != Py_None) {
            if (!sums(to, out, device) || !apart(out)) return false;
            m.out = (float*)out.data_ptr();
            m.out_stride_row = out.stride(0);
            m.out_stride_head = out.stride(1);
        }
        if (at_rows == Py_None) return m.mass_rows >= batch;
        if (!plain(at_rows, rows, at::kInt, device, {batch})) return false;
        m.rows = (const int32_t*)rows.data_ptr();
        return true;
    }
};

// weights(mass, out, rows | None, q, cache, page_table, seq_lens, q_starts, max_q, max_len | None, scale | None,
//         k_exp, causal, window, sinks) -> status | None
PyObject* weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Batch b;
        Mass m;
        if (n != 15) Py_RETURN_NONE;
        PyObject* const args[11] = {a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[12], a[13], a[14]};
        if (!b.from(args, a[11], a[11]) || !m.from(a[0], a[1], a[2], b.p.batch, b.c.device) ||
            m.in.size(1) != b.c.c.kv_heads || m.out.sizes() != m.in.sizes())
            Py_RETURN_NONE;
        const int64_t need = kv_weights_workspace(&b.c.c, &b.p);
        if (need < 0) return PyLong_FromLong(-need);
        at::Tensor ws;
        if (need > 0) ws = at::empty({need}, b.q.options().dtype(at::kByte));
        const On on(b.c.device);
        return PyLong_FromLong(
            kv_weights(&b.c.c, &b.p, &m.m, need > 0 ? ws.data_ptr() : nullptr, need, b.c.stream()));
    });
}

// select(mass, seq_lens, keep, recent, sinks, rows | None, mass_out | None) -> kept | status | None
PyObject* select(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Mass m;
        at::Tensor lens;
        int64_t keep, recent, sinks;
        if (n != 7 || !tensor(a[1], lens) || lens.dim() != 1 || !integer(a[2], keep) || !integer(a[3], recent) ||
            !integer(a[4], sinks) || keep < 0 || recent < 0 || sinks < 0 || recent > keep || sinks > keep - recent)
            Py_RETURN_NONE;
        const int64_t batch = lens.size(0), device = lens.device().index();
        if (!plain(a[1], lens, at::kInt, device, {batch}) || !m.from(a[0], a[6], a[5], batch, device)) Py_RETURN_NONE;
        const int64_t heads = m.in.size(1);
        if (heads == 0 || (m.out.defined() && a[6] != a[0] &&
                           (m.out.size(0) != m.in.size(0) || m.out.size(1) != heads ||
                            m.out.size(2) < (keep < m.m.width ? keep : m.m.width))))
            Py_RETURN_NONE;
        const at::Tensor kept = at::empty({batch, heads, keep}, lens.options());
        const int64_t need = kv_select_workspace(&m.m, batch, heads, keep);
        if (need < 0) return PyLong_FromLong(-need);
        at::Tensor ws;
        if (need > 0) ws = at::empty({need}, lens.options().dtype(at::kByte));
        const On on(device);
        const int st = kv_select(&m.m, (const int32_t*)lens.data_ptr(), batch, heads, keep, recent, sinks,
                                 (int32_t*)kept.data_ptr(), need > 0 ? ws.data_ptr() : nullptr, need,
                                 stream_of(device));
        if (st != IF4_OK) return PyLong_FromLong(st);
        return THPVariable_Wrap(kept);
    });
}

// compact(cache, page_table, kept, new_table, 0) -> status | None
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Cache c;
        at::Tensor table, kept, fresh;
        if (n != 5 || !c.from(a[0], a[4], a[4]) || !tensor(a[1], table) || table.dim() != 2 || !tensor(a[2], kept) ||
            kept.dim() != 3 || !tensor(a[3], fresh) || fresh.dim() != 2)
            Py_RETURN_NONE;
        const int64_t batch = table.size(0), keep = kept.size(2);
        if (!plain(a[1], table, at::kInt, c.device, table.sizes()) ||
            !plain(a[2], kept, at::kInt, c.device, {batch, c.c.kv_heads, keep}) ||
            !plain(a[3], fresh, at::kInt, c.device, {batch, fresh.size(1)}))
            Py_RETURN_NONE;
        const On on(c.device);
        return PyLong_FromLong(kv_compact(&c.c, (const int32_t*)table.data_ptr(), table.size(1),
                                          (const int32_t*)kept.data_ptr(), batch, keep,
                                          (const int32_t*)fresh.data_ptr(), fresh.size(1), c.stream()));
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

// bind_evict(weights, weights_workspace, select, select_workspace, compact)
PyObject* bind_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* f[5];
    if (!addresses(a, n, f, 5)) return nullptr;
    kv_weights = (decltype(kv_weights))f[0];
    kv_weights_workspace = (decltype(kv_weights_workspace))f[1];
    kv_select = (decltype(kv_select))f[2];
    kv_select_workspace = (decltype(kv_select_workspace))f[3];
    kv_compact = (decltype(kv_compact))f[4];
    Py_RETURN_NONE;
}

// bind(append, read, attention, workspace): the library's entry points, as addresses
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* f[4];
    if (!addresses(a, n, f, 4)) return nullptr;
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
    {"weights", (PyCFunction)(void*)weights, METH_FASTCALL, nullptr},
    {"select", (PyCFunction)(void*)select, METH_FASTCALL, nullptr},
    {"compact", (PyCFunction)(void*)compact, METH_FASTCALL, nullptr},
    {"bind", (PyCFunction)(void*)bind, METH_FASTCALL, nullptr},
    {"bind_evict", (PyCFunction)(void*)bind_evict, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv_call", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv_call(void) { return PyModule_Create(&module); }
