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
#include <vector>

#include "kvq.h"

namespace {

decltype(&kv_pages_reserve) g_reserve;
decltype(&kv_pages_trim) g_trim;
decltype(&kv_rope_append) g_rope;
decltype(&kv_attn_paged) g_attn;
decltype(&kv_gqa_append) g_gqa_append;
decltype(&kv_gqa_attn_paged) g_gqa_attn;
decltype(&kv_beam_select) g_beam;
decltype(&kv_pages_fork) g_fork;
decltype(&kv_pages_copy) g_copy;

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

int32_t* error_word(PyObject* o, int64_t dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor& e = tensor(o, dev, "err_word");
    if ((e.scalar_type() != at::kInt && e.scalar_type() != at::kByte) || !e.is_contiguous() ||
        e.numel() * (int64_t)e.element_size() < 4)
        refuse("err_word must be an int32 tensor or a uint8 workspace");
    return (int32_t*)e.data_ptr();
}

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
        return g_rope(fmt, &L, &rope, x ? x->data_ptr() : nullptr, xt, x_stride, n, pos, n, slots, qi, qt, it, ih, qo, ot, oh,
                      narrow(heads), codes, scales, rows, error_word(a[10], dev), (void*)integer(a[12]));
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

// The pools of grouped query heads: [n_pages][n_kv_heads][page_rows][head_dim] twice, scales.
struct HeadPools {
    int64_t pages, heads, page_rows, dim;
    uint8_t *k, *v;
    float* scales;
};
HeadPools head_pools(PyObject* k, PyObject* v, PyObject* scales, int64_t dev) {
    const at::Tensor& t = tensor(k, dev, "k_codes");
    if (t.dim() != 4) refuse("k_codes must be [n_pages][n_kv_heads][page_rows][head_dim]");
    HeadPools p{t.size(0), t.size(1), t.size(2), t.size(3), nullptr, nullptr, nullptr};
    p.k = (uint8_t*)address(k, at::kByte, dev, "k_codes", {p.pages, p.heads, p.page_rows, p.dim});
    p.v = (uint8_t*)address(v, at::kByte, dev, "v_codes", {p.pages, p.heads, p.page_rows, p.dim});
    p.scales = (float*)address(scales, at::kFloat, dev, "scales", {p.pages, p.heads, p.page_rows, 2});
    return p;
}

// rope or None, k_new or None, v_new or None, positions or None, slot_map or None, q_in or
// None, q_out or None, k_codes, v_codes, scales (None without rows), err_word or None, device, stream
PyObject* gqa_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return call(n_args, 13, [&]() -> int {
        const int64_t dev = integer(a[11]);
        kvq_rope rope{};
        const bool turns = a[0] != Py_None;
        if (turns) rope = structure<kvq_rope>(a[0]);
        const at::Tensor* k = a[1] == Py_None ? nullptr : &strided(a[1], 3, dev, "k_new");
        const at::Tensor* v = a[2] == Py_None ? nullptr : &strided(a[2], 3, dev, "v_new");
        const at::Tensor* q = a[5] == Py_None ? nullptr : &strided(a[5], 3, dev, "q_in");
        if (!k != !v) refuse("keys and values come together");
        if (!k && !q) refuse("neither rows nor queries");
        const at::Tensor& x = k ? *k : *q;
        const int64_t n = x.size(0), dim = x.size(2);
        const kvq_dtype type = query_type(x);
        HeadPools pool{0, 0, 16, dim, nullptr, nullptr, nullptr};
        const int64_t* slots = nullptr;
        if (k) {
            pool = head_pools(a[7], a[8], a[9], dev);
            if (k->size(1) != pool.heads || k->size(2) != pool.dim || v->sizes() != k->sizes() ||
                v->scalar_type() != k->scalar_type())
                refuse("k_new and v_new must be [n][n_kv_heads][head_dim] of one type, as the pool's heads");
            slots = (const int64_t*)address(a[4], at::kLong, dev, "slot_map", {n});
        }
        int64_t it = 0, ih = 0, ot = 0, oh = 0, heads = 0;
        const void* qi = nullptr;
        void* qo = nullptr;
        if (q) {
            const at::Tensor& o = strided(a[6], 3, dev, "q_out");
            if (q->size(0) != n || q->size(2) != dim || q->scalar_type() != x.scalar_type() || o.sizes() != q->sizes() ||
                o.scalar_type() != q->scalar_type())
                refuse("q_in and q_out must be [n][n_heads][head_dim], of the keys' type");
            heads = q->size(1);
            if (n > 1) {   // the stride of a dimension of size one says nothing
                it = q->stride(0);
                ot = o.stride(0);
            }
            if (heads > 1) {
                ih = q->stride(1);
                oh = o.stride(1);
            }
            qi = q->data_ptr();
            qo = o.data_ptr();
        }
        const int64_t* pos = nullptr;
        if (turns) {
            const int64_t axes = rope.n_axes;
            pos = axes == 1 && tensor(a[3], dev, "positions").dim() == 1
                      ? (const int64_t*)address(a[3], at::kLong, dev, "positions", {n})
                      : (const int64_t*)address(a[3], at::kLong, dev, "positions", {axes, n});
        }
        const auto step = [&](const at::Tensor* t, int d) { return t && t->size(d) > 1 ? t->stride(d) : 0; };
        return g_gqa_append(turns ? &rope : nullptr, type, n, narrow(heads), narrow(k ? pool.heads : 1), narrow(dim),
                            k ? k->data_ptr() : nullptr, step(k, 0), step(k, 1), v ? v->data_ptr() : nullptr, step(v, 0),
                            step(v, 1), pos, n, slots, qi, it, ih, qo, ot, oh, pool.k, pool.v, pool.scales,
                            narrow(pool.page_rows), narrow(pool.pages), error_word(a[10], dev), (void*)integer(a[12]));
    });
}

// q, cu_q, k_codes, v_codes, scales, block_table, kv_lens, out, workspace, sm_scale, causal,
// device, stream
PyObject* gqa_attn(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return call(n_args, 13, [&]() -> int {
        const int64_t dev = integer(a[11]);
        const at::Tensor &q = tensor(a[0], dev, "q"), &ws = workspace(a[8], dev);
        if (q.dim() != 3) refuse("q must be [n_tokens][n_heads][head_dim]");
        const HeadPools pool = head_pools(a[2], a[3], a[4], dev);
        const int64_t n = q.size(0), heads = q.size(1), seqs = count(a[6], dev, "kv_lens");
        const int64_t stride = last_size(tensor(a[5], dev, "block_table"));
        const kvq_dtype qt = query_type(q);
        const double sm = PyFloat_AsDouble(a[9]);
        if (sm == -1.0 && PyErr_Occurred()) throw Error{};
        return g_gqa_attn(address(a[0], q.scalar_type(), dev, "q", {n, heads, pool.dim}), qt, n, narrow(heads),
                          narrow(pool.heads), narrow(pool.dim), narrow(seqs),
                          (const int64_t*)address(a[1], at::kLong, dev, "cu_q", {seqs + 1}), pool.k, pool.v, pool.scales,
                          (const int32_t*)address(a[5], at::kInt, dev, "block_table", {seqs, stride}), narrow(stride),
                          (const int64_t*)address(a[6], at::kLong, dev, "kv_lens", {seqs}), narrow(pool.page_rows),
                          narrow(pool.pages), (float)sm, narrow(integer(a[10])),
                          address(a[7], q.scalar_type(), dev, "out", {n, heads, pool.dim}), ws.data_ptr(),
                          (size_t)ws.numel(), (void*)integer(a[12]));
    });
}

// logits, scores, out_scores, parents, tokens, workspace, device, stream
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return call(n_args, 8, [&]() -> int {
        const int64_t dev = integer(a[6]);
        const at::Tensor& x = strided(a[0], 3, dev, "logits");
        const at::Tensor& ws = workspace(a[5], dev);
        const int64_t n = x.size(0), beams = x.size(1), vocab = x.size(2), keep = last_size(tensor(a[2], dev, "out_scores"));
        const int64_t step = beams > 1 ? x.stride(1) : n > 1 ? x.stride(0) : vocab;
        if (n > 1 && beams > 1 && x.stride(0) != beams * step) refuse("logits' rows must lie at one distance");
        return g_beam(x.data_ptr(), query_type(x), step, narrow(n), narrow(beams), vocab,
                      (const float*)address(a[1], at::kFloat, dev, "scores", {n, beams}), narrow(keep),
                      (float*)address(a[2], at::kFloat, dev, "out_scores", {n, keep}),
                      (int32_t*)address(a[3], at::kInt, dev, "parents", {n, keep}),
                      (int32_t*)address(a[4], at::kInt, dev, "tokens", {n, keep}), ws.data_ptr(), (size_t)ws.numel(),
                      (void*)integer(a[7]));
    });
}

// parents, kv_lens, block_table, free_pages, n_free, page_rows, copies, workspace, device, stream
PyObject* fork_pages(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return call(n_args, 10, [&]() -> int {
        const int64_t dev = integer(a[8]);
        const int64_t n = count(a[1], dev, "kv_lens"), pages = count(a[3], dev, "free_pages");
        const int64_t stride = last_size(tensor(a[2], dev, "block_table"));
        const at::Tensor& ws = workspace(a[7], dev);
        return g_fork(narrow(n), narrow(integer(a[5])), (const int32_t*)address(a[0], at::kInt, dev, "parents", {n}),
                      (int64_t*)address(a[1], at::kLong, dev, "kv_lens", {n}),
                      (int32_t*)address(a[2], at::kInt, dev, "block_table", {n, stride}), narrow(stride),
                      (int32_t*)address(a[3], at::kInt, dev, "free_pages", {pages}),
                      (int32_t*)address(a[4], at::kInt, dev, "n_free", {1}), narrow(pages),
                      (int32_t*)address(a[6], at::kInt, dev, "copies", {n, 2}), ws.data_ptr(), (size_t)ws.numel(),
                      (void*)integer(a[9]));
    });
}

// copies, pools (a sequence of tensors [n_pages][...]), err_word or None, n_pages or -1, device, stream
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return call(n_args, 6, [&]() -> int {
        const int64_t dev = integer(a[4]);
        int64_t pages = integer(a[3]);
        PyObject* list = PySequence_Fast(a[1], "pools must be a sequence of tensors");
        if (!list) throw Error{};
        struct Held {
            PyObject* o;
            ~Held() { Py_DECREF(o); }
        } held{list};
        std::vector<kvq_pool> pools((size_t)PySequence_Fast_GET_SIZE(list));
        for (size_t i = 0; i < pools.size(); ++i) {
            const at::Tensor& t = tensor(PySequence_Fast_GET_ITEM(list, (Py_ssize_t)i), dev, "a pool");
            if (t.dim() < 1 || !t.is_contiguous()) refuse("a pool must be contiguous");
            if (pages < 0) pages = t.size(0);
            // rows [n_pages * page_rows][*] count as pages too
            if (pages > 0 ? t.size(0) % pages != 0 : t.numel() != 0) refuse("the pools must hold the same pages");
            const int64_t bytes = t.numel() * (int64_t)t.element_size();
            pools[i] = kvq_pool{t.data_ptr(), pages > 0 ? bytes / pages : 0};
        }
        const int64_t n = tensor(a[0], dev, "copies").dim() > 0 ? tensor(a[0], dev, "copies").size(0) : 0;
        return g_copy(narrow(n), (const int32_t*)address(a[0], at::kInt, dev, "copies", {n, 2}), narrow(pages < 0 ? 0 : pages),
                      narrow((int64_t)pools.size()), pools.data(), error_word(a[2], dev), (void*)integer(a[5]));
    });
}

// The addresses of the entry points, in the order of their names here.
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return call(n_args, 9, [&]() -> int {
        g_reserve = (decltype(g_reserve))integer(a[0]);
        g_trim = (decltype(g_trim))integer(a[1]);
        g_rope = (decltype(g_rope))integer(a[2]);
        g_attn = (decltype(g_attn))integer(a[3]);
        g_gqa_append = (decltype(g_gqa_append))integer(a[4]);
        g_gqa_attn = (decltype(g_gqa_attn))integer(a[5]);
        g_beam = (decltype(g_beam))integer(a[6]);
        g_fork = (decltype(g_fork))integer(a[7]);
        g_copy = (decltype(g_copy))integer(a[8]);
        return 0;
    });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, (PyCFunction)(void (*)(void))F, METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<init>("init"),           method<reserve>("reserve"),       method<trim>("trim"),
                         method<rope_append>("rope_append"), method<attn_paged>("attn_paged"), method<gqa_append>("gqa_append"),
                         method<gqa_attn>("gqa_attn"), method<beam_select>("beam_select"), method<fork_pages>("fork_pages"),
                         method<copy_pages>("copy_pages"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_host() { return PyModule_Create(&module); }
