// paged_host.cpp -- the host side of the paged calls as a Python extension: checks the
// tensors of a call and passes their addresses to the C entry points.
//
// A serving loop makes these calls every step, on a few KB.  Checked in Python, an
// argument costs 0.4 us and a call of 17 through ctypes 2 us more, together three
// times the launch; here a call's checks take well under one.  The entry points'
// addresses come from the library that Python has loaded (init).
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "kvq.h"

namespace {

decltype(&kv_pages_reserve) g_reserve;
decltype(&kv_pages_trim) g_trim;
decltype(&kv_rope_append) g_rope;
decltype(&kv_attn_paged) g_attn;

struct Error {};   // a Python exception is set

[[noreturn]] void refuse(const std::string& what) {
    PyErr_SetString(PyExc_ValueError, what.c_str());
    throw Error{};
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Error{};
    return v;
}
// Into an int32 argument; the entry points refuse what is too large.
int32_t narrow(int64_t v) {
    return v > INT32_MAX ? INT32_MAX : v < INT32_MIN ? INT32_MIN : (int32_t)v;
}

const at::Tensor& tensor(PyObject* o, int64_t dev, const char* name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        throw Error{};
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    if (t.get_device() != dev) refuse(std::string(name) + " is on " + t.device().str() + ", not on the current device");
    return t;
}
// Address of a contiguous tensor on the current device; its type and shape are checked.
void* address(PyObject* o, at::ScalarType type, int64_t dev, const char* name, at::IntArrayRef shape) {
    const at::Tensor& t = tensor(o, dev, name);
    if (t.scalar_type() != type)
        refuse(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (t.sizes() != shape) {
        std::string want, got;
        for (int64_t n : shape) want += " " + std::to_string(n);
        for (int64_t n : t.sizes()) got += " " + std::to_string(n);
        refuse(std::string(name) + " must have shape (" + want + " ), got (" + got + " )");
    }
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    return t.data_ptr();
}
const at::Tensor& workspace(PyObject* o, int64_t dev) {
    const at::Tensor& t = tensor(o, dev, "workspace");
    if (t.scalar_type() != at::kByte || !t.is_contiguous()) refuse("workspace must be a contiguous uint8 tensor");
    return t;
}
// A tensor on the current device whose last dimension is contiguous.
const at::Tensor& strided(PyObject* o, int64_t dims, int64_t dev, const char* name) {
    const at::Tensor& t = tensor(o, dev, name);
    if (t.dim() != dims || (t.size(dims - 1) > 1 && t.stride(dims - 1) != 1))
        refuse(std::string(name) + " must have " + std::to_string(dims) + " dimensions, the last one contiguous");
    return t;
}
int64_t count(PyObject* o, int64_t dev, const char* name) { return tensor(o, dev, name).numel(); }
int64_t last_size(const at::Tensor& t) { return t.dim() > 0 ? t.size(t.dim() - 1) : 0; }

kvq_dtype query_type(const at::Tensor& t) {
    if (t.scalar_type() == at::kFloat) return KVQ_F32;
    if (t.scalar_type() == at::kBFloat16) return KVQ_BF16;
    refuse("queries and rows must be float32 or bfloat16");
}

// A ctypes structure.
template <class T>
T structure(PyObject* o) {
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Error{};
    T v;
    const bool ok = b.len == (Py_ssize_t)sizeof(T);
    if (ok) memcpy(&v, b.buf, sizeof(T));
    PyBuffer_Release(&b);
    if (!ok) refuse("a layout of the wrong kind");
    return v;
}

struct Rows {
    int64_t dims, bytes;
};
Rows row_of(kvq_format fmt, const kvq_mla_layout& L) {
    const int64_t d = (int64_t)L.block_dim[0] + (L.n_blocks > 1 ? L.block_dim[1] : 0);
    return {d, fmt == KVQ_KV8 ? d : d / 2};
}

template <class F>
PyObject* call(Py_ssize_t n, Py_ssize_t want, F body) {
    try {
        if (n != want) {
            PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
            return nullptr;
        }
        return PyLong_FromLong(body());
    } catch (const Error&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown exception");
    }
    return nullptr;
}

// kv_lens, new_lens, block_table, free_pages, n_free, page_rows, lens_out, cu_new,
// slot_map, positions or None, workspace, device, stream
PyObject* reserve(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return call(n_args, 13, [&]() -> int {
        const int64_t dev = integer(a[11]);
        const int64_t n = count(a[0], dev, "kv_lens"), m = count(a[8], dev, "slot_map"), pages = count(a[3], dev, "free_pages");
        const int64_t stride = last_size(tensor(a[2], dev, "block_table"));
        const at::Tensor& ws = workspace(a[10], dev);
        return g_reserve(narrow(n), narrow(integer(a[5])), (const int64_t*)address(a[0], at::kLong, dev, "kv_lens", {n}),
                         (const int64_t*)address(a[1], at::kLong, dev, "new_lens", {n}),
                         (int32_t*)address(a[2], at::kInt, dev, "block_table", {n, stride}), narrow(stride),
                         (int32_t*)address(a[3], at::kInt, dev, "free_pages", {pages}),
                         (int32_t*)address(a[4], at::kInt, dev, "n_free", {1}), narrow(pages),
                         (int64_t*)address(a[6], at::kLong, dev, "lens_out", {n}),
                         (int64_t*)address(a[7], at::kLong, dev, "cu_new", {n + 1}),
                         (int64_t*)address(a[8], at::kLong, dev, "slot_map", {m}),
                         a[9] == Py_None ? nullptr : (int64_t*)address(a[9], at::kLong, dev, "positions", {m}), m,
                         ws.data_ptr(), (size_t)ws.numel(), (void*)integer(a[12]));
    });
}

// kv_lens, keep_lens, block_table, free_pages, n_free, page_rows, workspace, device, stream
PyObject* trim(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return call(n_args, 9, [&]() -> int {
        const int64_t dev = integer(a[7]);
        const int64_t n = count(a[0], dev, "kv_lens"), pages = count(a[3], dev, "free_pages");
        const int64_t stride = last_size(tensor(a[2], dev, "block_table"));
        const at::Tensor& ws = workspace(a[6], dev);
        return g_trim(narrow(n), narrow(integer(a[5])), (int64_t*)address(a[0], at::kLong, dev, "kv_lens", {n}),
                      (const int64_t*)address(a[1], at::kLong, dev, "keep_lens", {n}),
                      (int32_t*)address(a[2], at::kInt, dev, "block_table", {n, stride}), narrow(stride),
                      (int32_t*)address(a[3], at::kInt, dev, "free_pages", {pages}),
                      (int32_t*)address(a[4], at::kInt, dev, "n_free", {1}), narrow(pages), ws.data_ptr(),
                      (size_t)ws.numel(), (void*)integer(a[8]));
    });
}

// fmt, rope, x_new or None, positions, slot_map, q_in or None, q_out, codes, scales,
// layout, err_word or None, device, stream
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return call(n_args, 13, [&]() -> int {
        const int64_t dev = integer(a[11]);
        const kvq_format fmt = (kvq_format)narrow(integer(a[0]));
        const kvq_rope rope = structure<kvq_rope>(a[1]);
        const kvq_mla_layout L = structure<kvq_mla_layout>(a[9]);
        const Rows row = row_of(fmt, L);
        const at::Tensor* x = a[2] == Py_None ? nullptr : &strided(a[2], 2, dev, "x_new");
        const at::Tensor* q = a[5] == Py_None ? nullptr : &strided(a[5], 3, dev, "q_in");
        if (!x && !q) refuse("neither rows nor queries");
        const int64_t n = x ? x->size(0) : q->size(0), axes = rope.n_axes;
        const int64_t* pos = axes == 1 && tensor(a[3], dev, "positions").dim() == 1
                                 ? (const int64_t*)address(a[3], at::kLong, dev, "positions", {n})
                                 : (const int64_t*)address(a[3], at::kLong, dev, "positions", {axes, n});
        kvq_dtype xt = KVQ_F32, qt = KVQ_F32;
        int64_t x_stride = 0, rows = 0, heads = 0, it = 0, ih = 0, ot = 0, oh = 0;
        const int64_t* slots = nullptr;
        uint8_t* codes = nullptr;
        float* scales = nullptr;
        if (x) {
            xt = query_type(*x);
            if (x->size(1) != row.dims) refuse("x_new must have " + std::to_string(row.dims) + " columns");
            x_stride = n > 1 ? x->stride(0) : row.dims;
            const at::Tensor& c = tensor(a[7], dev, "codes");
            rows = c.dim() > 0 ? c.size(0) : 0;
            slots = (const int64_t*)address(a[4], at::kLong, dev, "slot_map", {n});
            codes = (uint8_t*)address(a[7], at::kByte, dev, "codes", {rows, row.bytes});
            scales = (float*)address(a[8], at::kFloat, dev, "scales", {rows, (int64_t)L.n_blocks});
        }
        const void* qi = nullptr;
        void* qo = nullptr;
        if (q) {
            const at::Tensor& o = strided(a[6], 3, dev, "q_out");
            qt = query_type(*q);
            heads = q->size(1);
            const int64_t width = o.size(2);
            if (q->size(0) != n || q->size(2) != rope.dim || o.size(0) != n || o.size(1) != heads ||
                (width != rope.dim && width != row.dims) || o.scalar_type() != q->scalar_type())
                refuse("q_in must be [" + std::to_string(n) + "][n_heads][" + std::to_string(rope.dim) + "] and q_out match it");
            if (n > 1) {   // the stride of a dimension of size one says nothing
                it = q->stride(0);
                ot = o.stride(0);
            }
            if (heads > 1) {
                ih = q->stride(1);
                oh = o.stride(1);
            }
            qi = q->data_ptr();
            qo = (char*)o.data_ptr() + (width - rope.dim) * o.element_size();
        }
        int32_t* err = nullptr;
        if (a[10] != Py_None) {
            const at::Tensor& e = tensor(a[10], dev, "err_word");
            if ((e.scalar_type() != at::kInt && e.scalar_type() != at::kByte) || !e.is_contiguous() ||
                e.numel() * (int64_t)e.element_size() < 4)
                refuse("err_word must be an int32 tensor or a uint8 workspace");
            err = (int32_t*)e.data_ptr();
        }
        return g_rope(fmt, &L, &rope, x ? x->data_ptr() : nullptr, xt, x_stride, n, pos, n, slots, qi, qt, it, ih, qo, ot, oh,
                      narrow(heads), codes, scales, rows, err, (void*)integer(a[12]));
    });
}

// fmt, q, cu_q, codes, scales, block_table, kv_lens, page_rows, out, workspace,
// sm_scale, layout, path, device, stream
PyObject* attn_paged(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return call(n_args, 15, [&]() -> int {
        const int64_t dev = integer(a[13]);
        const kvq_format fmt = (kvq_format)narrow(integer(a[0]));
        const kvq_mla_layout L = structure<kvq_mla_layout>(a[11]);
        const at::Tensor &q = tensor(a[1], dev, "q"), &c = tensor(a[3], dev, "codes"), &ws = workspace(a[9], dev);
        if (q.dim() != 3) refuse("q must be [n_tokens][n_heads][576]");
        const int64_t n = q.size(0), heads = q.size(1), seqs = count(a[6], dev, "kv_lens");
        const int64_t rows = c.dim() > 0 ? c.size(0) : 0, page = integer(a[7]);
        const int64_t stride = last_size(tensor(a[5], dev, "block_table"));
        if (page <= 0 || rows % page != 0) refuse("the pool must hold whole pages");
        const kvq_dtype qt = query_type(q);
        const double sm = PyFloat_AsDouble(a[10]);
        if (sm == -1.0 && PyErr_Occurred()) throw Error{};
        return g_attn(fmt, &L, address(a[1], q.scalar_type(), dev, "q", {n, heads, 576}), qt, n, narrow(heads), narrow(seqs),
                      (const int64_t*)address(a[2], at::kLong, dev, "cu_q", {seqs + 1}),
                      (const uint8_t*)address(a[3], at::kByte, dev, "codes", {rows, row_of(fmt, L).bytes}),
                      (const float*)address(a[4], at::kFloat, dev, "scales", {rows, (int64_t)L.n_blocks}),
                      (const int32_t*)address(a[5], at::kInt, dev, "block_table", {seqs, stride}), narrow(stride),
                      (const int64_t*)address(a[6], at::kLong, dev, "kv_lens", {seqs}), narrow(page), narrow(rows / page),
                      (float)sm, address(a[8], q.scalar_type(), dev, "out", {n, heads, 512}), ws.data_ptr(),
                      (size_t)ws.numel(), (kvq_path)narrow(integer(a[12])), (void*)integer(a[14]));
    });
}

// The addresses of kv_pages_reserve, kv_pages_trim, kv_rope_append, kv_attn_paged.
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return call(n_args, 4, [&]() -> int {
        g_reserve = (decltype(g_reserve))integer(a[0]);
        g_trim = (decltype(g_trim))integer(a[1]);
        g_rope = (decltype(g_rope))integer(a[2]);
        g_attn = (decltype(g_attn))integer(a[3]);
        return 0;
    });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, (PyCFunction)(void (*)(void))F, METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<init>("init"),           method<reserve>("reserve"),       method<trim>("trim"),
                         method<rope_append>("rope_append"), method<attn_paged>("attn_paged"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_host() { return PyModule_Create(&module); }
