// The paged-cache calls' binding to PyTorch: checks the tensors, allocates what the caller did
// not give, and calls the C ABI on the current stream of the tensors' device.  A decode step makes
// several of these calls of a few microseconds each, and the same checks in Python took longer than
// the kernels (block tables: 20 us of host time a call, here about a third).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <string>

#include "li.h"

namespace {

PyObject* g_li_error = nullptr;  // api.LiError(name, status)

struct Refused {
    std::string why;
};
struct Raised {};  // a Python exception is set

[[noreturn]] void refuse(const std::string& why) { throw Refused{why}; }

const char* type_name(at::ScalarType t) { return c10::toString(t); }

std::string shape_text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// The device every tensor of a call has to be on: the leading tensor's, made current for the call.
struct Place {
    c10::Device dev;
    c10::cuda::OptionalCUDAGuard guard;
    explicit Place(const at::Tensor& lead, const char* call) : dev(lead.device()) {
        if (!dev.is_cuda()) refuse(std::string(call) + " takes CUDA tensors");
        guard.set_device(dev);
    }
    li_stream_t stream() const { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
        return at::empty(shape, at::TensorOptions().dtype(t).device(dev));
    }
    // a contiguous tensor of this type, here (and of this shape)
    void* take(const at::Tensor& x, const char* name, at::ScalarType t) const {
        if (x.scalar_type() != t || x.device() != dev || !x.is_contiguous())
            refuse(std::string(name) + " must be a contiguous " + type_name(t) + " tensor on " + dev.str() + ", got " +
                   type_name(x.scalar_type()) + " on " + x.device().str() + (x.is_contiguous() ? "" : ", not contiguous"));
        return x.data_ptr();
    }
    void* take(const at::Tensor& x, const char* name, at::ScalarType t, at::IntArrayRef shape) const {
        if (x.sizes() != shape)
            refuse(std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(x.sizes()));
        return take(x, name, t);
    }
    void* maybe(PyObject* o, const char* name, at::ScalarType t, at::IntArrayRef shape) const {
        return o == Py_None ? nullptr : take(tensor(o, name), name, t, shape);
    }
};

// A contiguous tensor from byte `offset` of a shared allocation.  (An allocation costs the host half a microsecond, a
// tensor over one that is there a tenth.)
at::Tensor part_of(const at::Tensor& shared, int64_t offset, at::ScalarType t, at::IntArrayRef shape) {
    at::Tensor x = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(shared.storage()), shared.key_set(),
                                                            c10::scalarTypeToTypeMeta(t));
    x.unsafeGetTensorImpl()->set_storage_offset(offset / (int64_t)c10::elementSize(t));
    x.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    return x;
}

// An output: the caller's tensor, or a new one.  `object` is a new reference.
struct Out {
    PyObject* object = nullptr;
    void* ptr = nullptr;
    Out(const Place& p, PyObject* given, const char* name, at::ScalarType t, at::IntArrayRef shape) {
        if (given != Py_None) {
            ptr = p.take(tensor(given, name), name, t, shape);
            object = Py_NewRef(given);
        } else {
            wrap(p.empty(shape, t));
        }
    }
    // ... or a new vector from byte `offset` of an allocation that several outputs share
    Out(const Place& p, PyObject* given, const char* name, at::ScalarType t, int64_t n, const at::Tensor& shared,
        int64_t offset) {
        if (given != Py_None) {
            ptr = p.take(tensor(given, name), name, t, {n});
            object = Py_NewRef(given);
        } else {
            wrap(part_of(shared, offset, t, {n}));
        }
    }
    Out(const Out&) = delete;
    ~Out() { Py_XDECREF(object); }
    void wrap(at::Tensor&& x) {
        ptr = x.data_ptr();
        object = THPVariable_Wrap(std::move(x));
        if (!object) throw Raised{};
    }
    PyObject* give() {
        PyObject* o = object;
        object = nullptr;
        return o;
    }
};

int64_t whole(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
int small(PyObject* o, const char* name) {
    const int64_t v = whole(o);
    if (v < INT_MIN || v > INT_MAX) refuse(std::string(name) + " is out of range");
    return (int)v;
}
int clamped(PyObject* o) {  // sizes beyond int mean "all of it"
    int overflow = 0;
    const int64_t v = PyLong_AsLongLongAndOverflow(o, &overflow);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (overflow) return overflow > 0 ? INT_MAX : INT_MIN;
    return v > INT_MAX ? INT_MAX : v < INT_MIN ? INT_MIN : (int)v;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)v;
}
int size_of(int64_t n, const char* name) {
    if (n > INT_MAX) refuse(std::string(name) + " is too large");
    return (int)n;
}

void check(const char* call, li_status s) {
    if (s == LI_OK) return;
    PyObject* e = g_li_error ? PyObject_CallFunction(g_li_error, "si", call, (int)s) : nullptr;
    if (e) {
        PyErr_SetObject(g_li_error, e);
        Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
        PyErr_Format(PyExc_RuntimeError, "%s failed: %s", call, li_status_string(s));
    }
    throw Raised{};
}

// Runs a call's body; its refusals and errors become Python exceptions.
template <typename F>
PyObject* guarded(F&& body) {
    try {
        return body();
    } catch (const Refused& r) {
        PyErr_SetString(PyExc_ValueError, r.why.c_str());
    } catch (const Raised&) {
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type) PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}
void arity(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) refuse("wrong number of arguments");
}

constexpr auto I32 = at::kInt, I64 = at::kLong, U8 = at::kByte, BF16 = at::kBFloat16, F32 = at::kFloat;

PyObject* block_tables(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        arity(n, 13);
        const at::Tensor &seq = tensor(v[0], "seq_lens"), &add = tensor(v[1], "new_lens"),
                         &table = tensor(v[2], "block_table"), &pool = tensor(v[3], "free_pages");
        const Place p(seq, "li_block_tables");
        if (table.dim() != 2) refuse("block_table must be [requests, max_blocks]");
        const int64_t R = table.size(0);
        if (pool.dim() != 1) refuse("free_pages must be one-dimensional");
        const int page = small(v[4], "page_size"), pages = small(v[5], "num_pages"), tokens = small(v[6], "max_tokens");
        const int64_t t = tokens > 0 ? tokens : 0;
        auto* sp = static_cast<int32_t*>(p.take(seq, "seq_lens", I32, {R}));
        auto* np = static_cast<int32_t*>(p.take(add, "new_lens", I32, {R}));
        auto* tp = static_cast<int32_t*>(p.take(table, "block_table", I32));
        auto* fp = static_cast<int32_t*>(p.take(pool, "free_pages", I32));
        auto* at0 = static_cast<int32_t*>(p.maybe(v[7], "free_start", I32, {1}));
        // new outputs lie one behind the other in one allocation (slots first: 8 bytes each)
        const int64_t wide = v[8] == Py_None ? 8 * t : 0, one = v[9] == Py_None ? 4 * t : 0;
        const int64_t two = v[10] == Py_None ? 4 * t : 0, ends = v[11] == Py_None ? 4 * (R + 1) : 0;
        const int64_t last = v[12] == Py_None ? 4 : 0;
        const int64_t bytes = wide + one + two + ends + last;
        at::Tensor shared;
        if (bytes) shared = p.empty({bytes}, U8);
        Out slots(p, v[8], "slots", I64, t, shared, 0), pos(p, v[9], "positions", I32, t, shared, wide),
            req(p, v[10], "requests", I32, t, shared, wide + one),
            starts(p, v[11], "starts", I32, R + 1, shared, wide + one + two),
            next(p, v[12], "free_next", I32, 1, shared, wide + one + two + ends);
        check("li_block_tables",
              li_block_tables(sp, np, size_of(R, "requests"), tp, size_of(table.size(1), "max_blocks"), page, pages, fp,
                              size_of(pool.numel(), "free_pages"), at0, tokens, static_cast<int64_t*>(slots.ptr),
                              static_cast<int32_t*>(pos.ptr), static_cast<int32_t*>(req.ptr),
                              static_cast<int32_t*>(starts.ptr), static_cast<int32_t*>(next.ptr), p.stream()));
        PyObject* r = PyTuple_New(5);
        if (!r) throw Raised{};
        Out* outs[5] = {&slots, &pos, &req, &starts, &next};
        for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(r, i, outs[i]->give());
        return r;
    });
}

int layout_of(PyObject* o) {
    if (PyUnicode_Check(o)) {
        if (PyUnicode_CompareWithASCIIString(o, "interleaved") == 0) return LI_ROPE_INTERLEAVED;
        if (PyUnicode_CompareWithASCIIString(o, "half") == 0) return LI_ROPE_HALF;
    }
    refuse("layout must be \"interleaved\" or \"half\"");
}

constexpr int64_t ROPE_SHARED = 1 << 21;
int64_t share_bytes(const at::Tensor& x) { return (x.numel() * (int64_t)x.element_size() + 255) / 256 * 256; }

// rope(xs, positions, table, layout, offset, mscale, outs or None): xs a list, layout and offset one value or a list
PyObject* rope(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        arity(n, 7);
        if (!PyList_Check(v[0]) || (v[6] != Py_None && !PyList_Check(v[6]))) refuse("x and out must be tensors or lists");
        const Py_ssize_t count = PyList_GET_SIZE(v[0]);
        if (count < 1 || count > LI_ROPE_MAX_TENSORS) refuse("one to four tensors");
        const bool layouts = PyList_Check(v[3]) || PyTuple_Check(v[3]), offsets = PyList_Check(v[4]) || PyTuple_Check(v[4]);
        if ((layouts && PySequence_Fast_GET_SIZE(v[3]) != count) || (offsets && PySequence_Fast_GET_SIZE(v[4]) != count) ||
            (v[6] != Py_None && PyList_GET_SIZE(v[6]) != count))
            refuse("one layout, offset and out per tensor");
        const at::Tensor &lead = tensor(PyList_GET_ITEM(v[0], 0), "x"), &pos = tensor(v[1], "positions"),
                         &table = tensor(v[2], "table");
        const Place p(lead, "li_rope");
        if (pos.dim() != 1 || table.dim() != 1) refuse("positions and table must be one-dimensional");
        const int64_t tokens = pos.size(0);
        auto* pp = static_cast<int32_t*>(p.take(pos, "positions", I32));
        auto* tp = static_cast<uint64_t*>(p.take(table, "table", I64));
        li_rope_tensor d[LI_ROPE_MAX_TENSORS];
        // New outputs of a small call share an allocation (a decode step's four: 6.1 -> 5.4 us of host time); large ones
        // have their own, so that each can be freed by itself.
        at::Tensor shared;
        int64_t used = 0;
        if (v[6] == Py_None && count > 1) {
            int64_t bytes = 0;
            for (Py_ssize_t i = 0; i < count; ++i) bytes += share_bytes(tensor(PyList_GET_ITEM(v[0], i), "x"));
            if (bytes <= ROPE_SHARED) shared = p.empty({bytes}, U8);
        }
        PyObject* outs = PyList_New(count);
        if (!outs) throw Raised{};
        struct Drop {
            PyObject* o;
            ~Drop() { Py_XDECREF(o); }
        } drop{outs};
        for (Py_ssize_t i = 0; i < count; ++i) {
            PyObject* xo = PyList_GET_ITEM(v[0], i);
            const at::Tensor& x = tensor(xo, "x");
            const at::ScalarType t = x.scalar_type();
            if (t != BF16 && t != F32) refuse(std::string("x has dtype ") + type_name(t) + ", expected BFloat16 or Float");
            const int64_t dims = x.dim();
            if (dims != 2 && dims != 3) refuse("x must be [tokens, heads, dim] or [tokens, dim]");
            if (x.size(0) != tokens || x.device() != p.dev) refuse("x and positions must have the same tokens and device");
            PyObject* oo = v[6] == Py_None ? nullptr : PyList_GET_ITEM(v[6], i);
            if (oo) {
                const at::Tensor& o = tensor(oo, "out");
                if (o.sizes() != x.sizes() || o.scalar_type() != t || o.device() != p.dev)
                    refuse("out must have x's shape, dtype and device");
                Py_INCREF(oo);
            } else {
                oo = THPVariable_Wrap(shared.defined() ? part_of(shared, used, t, x.sizes()) : p.empty(x.sizes(), t));
                if (!oo) throw Raised{};
                used += share_bytes(x);
            }
            PyList_SET_ITEM(outs, i, oo);
            const at::Tensor& o = THPVariable_Unpack(oo);
            if (x.stride(dims - 1) != 1 || o.stride(dims - 1) != 1) refuse("a head's elements must be next to each other");
            d[i] = li_rope_tensor{x.data_ptr(), o.data_ptr(), x.stride(0), dims == 3 ? x.stride(1) : 0, o.stride(0),
                                  dims == 3 ? o.stride(1) : 0, dims == 3 ? size_of(x.size(1), "heads") : 1,
                                  size_of(x.size(dims - 1), "dim"),
                                  small(offsets ? PySequence_Fast_GET_ITEM(v[4], i) : v[4], "offset"),
                                  layout_of(layouts ? PySequence_Fast_GET_ITEM(v[3], i) : v[3]),
                                  t == BF16 ? LI_DTYPE_BF16 : LI_DTYPE_F32};
        }
        check("li_rope", li_rope(d, (int)count, size_of(tokens, "tokens"), pp, tp, size_of(2 * table.size(0), "table"),
                                 real(v[5]), p.stream()));
        drop.o = nullptr;
        return outs;
    });
}

int64_t kv4_slots(const at::Tensor& cache) {
    if (cache.dim() != 3 || cache.size(2) != LI_KV4_ROW_BYTES)
        refuse("a 4-bit cache is uint8 [pages, page_size, " + std::to_string(LI_KV4_ROW_BYTES) + "]");
    return cache.size(0) * cache.size(1);
}

PyObject* kv4_write(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        arity(n, 3);
        const at::Tensor &rows = tensor(v[0], "rows"), &slots = tensor(v[1], "slots"), &cache = tensor(v[2], "cache");
        const Place p(rows, "li_kv4_write");
        if (slots.dim() != 1) refuse("slots must be one-dimensional");
        const int64_t count = slots.size(0);
        if (rows.scalar_type() != BF16 || rows.dim() != 2 || rows.size(0) != count || rows.size(1) != 576)
            refuse("rows must be BFloat16 (" + std::to_string(count) + ", 576)");
        if (count && rows.stride(1) != 1) refuse("a row's elements must be next to each other");
        const int64_t num = kv4_slots(cache);
        check("li_kv4_write",
              li_kv4_write(rows.data_ptr(), count > 1 ? rows.stride(0) : 576,
                           static_cast<int64_t*>(p.take(slots, "slots", I64)), count, p.take(cache, "cache", U8), num,
                           p.stream()));
        return Py_NewRef(v[2]);
    });
}

PyObject* kv4_read(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        arity(n, 3);
        const at::Tensor &cache = tensor(v[0], "cache"), &slots = tensor(v[1], "slots");
        const Place p(cache, "li_kv4_read");
        if (slots.dim() != 1) refuse("slots must be one-dimensional");
        const int64_t num = kv4_slots(cache), count = slots.size(0);
        void* cp = p.take(cache, "cache", U8);
        auto* sp = static_cast<int64_t*>(p.take(slots, "slots", I64));
        Out out(p, v[2], "out", BF16, {count, 576});
        check("li_kv4_read", li_kv4_read(cp, num, sp, count, out.ptr, p.stream()));
        return out.give();
    });
}

// What the two attention calls share: q, cache, block_table, requests, scale, out, workspace.
struct Attention {
    Place p;
    li_attn_desc d{};
    void *q, *cache;
    int32_t *table = nullptr, *requests;
    Attention(const at::Tensor& qt, PyObject* co, PyObject* to, PyObject* ro, PyObject* scale, const char* call)
        : p(qt, call) {
        const at::Tensor& c = tensor(co, "cache");
        if (qt.dim() != 3 || qt.size(2) != 576) refuse("q must be [rows, heads, 576]");
        const bool four = c.scalar_type() == U8;
        if (c.dim() != 3 || c.size(2) != (four ? LI_KV4_ROW_BYTES : 576))
            refuse("cache must be uint8 [pages, page_size, 416] (4 bits) or bfloat16 [pages, page_size, 576]");
        q = p.take(qt, "q", BF16);
        cache = p.take(c, "cache", four ? U8 : BF16);
        d.rows = size_of(qt.size(0), "rows");
        d.heads = size_of(qt.size(1), "heads");
        d.num_pages = size_of(c.size(0), "pages");
        d.page_size = size_of(c.size(1), "page_size");
        d.cache_dtype = four ? LI_DTYPE_E2M1 : LI_DTYPE_BF16;
        d.scale = real(scale);
        if (to == Py_None) {  // a dense cache: request r's positions are page r
            d.requests = d.num_pages;
            d.max_blocks = 1;
        } else {
            const at::Tensor& t = tensor(to, "block_table");
            if (t.dim() != 2) refuse("block_table must be [requests, max_blocks]");
            table = static_cast<int32_t*>(p.take(t, "block_table", I32));
            d.requests = size_of(t.size(0), "requests");
            d.max_blocks = size_of(t.size(1), "max_blocks");
        }
        requests = static_cast<int32_t*>(p.maybe(ro, "requests", I32, {d.rows}));
    }
};

// The caller's workspace where it is large enough, else one of the call's own.
struct Work {
    at::Tensor own;
    void* ptr = nullptr;
    size_t bytes;
    Work(const Attention& a, PyObject* given, int positions)
        : bytes(li_paged_attention_workspace(a.d.rows, a.d.heads, positions)) {
        if (!bytes) return;
        if (given != Py_None) {
            const at::Tensor& w = tensor(given, "workspace");
            if (w.device() != a.p.dev || !w.is_contiguous()) refuse("workspace must be contiguous, on " + a.p.dev.str());
            if ((size_t)w.numel() * w.element_size() >= bytes) {
                ptr = w.data_ptr();
                return;
            }
        }
        own = a.p.empty({(int64_t)bytes}, U8);
        ptr = own.data_ptr();
    }
};

// sparse(q, cache, sel, scale, block_table, requests, out, workspace)
PyObject* sparse(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        arity(n, 8);
        const Attention a(tensor(v[0], "q"), v[1], v[4], v[5], v[3], "li_paged_sparse_attention");
        const at::Tensor& sel = tensor(v[2], "sel");
        if (sel.dim() != 2) refuse("sel must be [rows, k]");
        const int k = size_of(sel.size(1), "k");
        auto* sp = static_cast<int32_t*>(a.p.take(sel, "sel", I32, {a.d.rows, k}));
        Out out(a.p, v[6], "out", BF16, {a.d.rows, a.d.heads, 512});
        const Work w(a, v[7], k);
        check("li_paged_sparse_attention",
              li_paged_sparse_attention(a.q, a.cache, a.table, a.requests, sp, k, &a.d, out.ptr, w.ptr, w.bytes,
                                        a.p.stream()));
        return out.give();
    });
}

// window(q, cache, positions, scale, window, sinks, block_table, requests, max_len or None, out, workspace)
PyObject* window(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        arity(n, 11);
        const Attention a(tensor(v[0], "q"), v[1], v[6], v[7], v[3], "li_window_attention");
        auto* pp = static_cast<int32_t*>(a.p.take(tensor(v[2], "positions"), "positions", I32, {a.d.rows}));
        const int wide = clamped(v[4]), sinks = clamped(v[5]);
        int64_t top = (int64_t)a.d.max_blocks * a.d.page_size;
        if (v[8] != Py_None) top = clamped(v[8]);
        const int max_len = top > INT_MAX ? INT_MAX : (int)top;
        int64_t seen = (int64_t)wide + sinks;
        if (seen > max_len) seen = max_len;
        Out out(a.p, v[9], "out", BF16, {a.d.rows, a.d.heads, 512});
        const Work w(a, v[10], seen > 0 ? (int)seen : 0);
        check("li_window_attention",
              li_window_attention(a.q, a.cache, a.table, a.requests, pp, wide, sinks, max_len, &a.d, out.ptr, w.ptr,
                                  w.bytes, a.p.stream()));
        return out.give();
    });
}

PyObject* set_error(PyObject*, PyObject* e) {
    Py_XSETREF(g_li_error, Py_NewRef(e));
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}

PyMethodDef methods[] = {{"block_tables", fast(block_tables), METH_FASTCALL, nullptr},
                         {"rope", fast(rope), METH_FASTCALL, nullptr},
                         {"kv4_write", fast(kv4_write), METH_FASTCALL, nullptr},
                         {"kv4_read", fast(kv4_read), METH_FASTCALL, nullptr},
                         {"sparse", fast(sparse), METH_FASTCALL, nullptr},
                         {"window", fast(window), METH_FASTCALL, nullptr},
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
