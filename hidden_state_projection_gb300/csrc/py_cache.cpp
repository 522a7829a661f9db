// py_cache.cpp -- the Python side of the paged cache's calls: tensors to the C ABI.
//
// A decode step makes these calls for every layer, and through ctypes a small one cost more on
// the host (10 to 19 us: attribute by attribute, packed structs, outputs from torch.empty)
// than on the GPU (2 to 10 us).  Here the tensors are read in place.  The module only checks and
// marshals: sizes, strides, types and devices of the tensors, outputs and workspaces that the
// caller did not pass, one C call with the interpreter lock released.  Every refusal raises
// ProjError with the status and the text that the C ABI uses.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <vector>

#include "proj.h"

namespace {

PyObject *g_error = nullptr;       // ProjError
PyObject *g_no_memory = nullptr;   // torch.OutOfMemoryError
PyObject *g_get_device = nullptr;  // torch._C._cuda_getDevice
PyObject *g_get_stream = nullptr;  // torch._C._cuda_getCurrentRawStream

struct Refusal {
    int status;
    char text[384];
};
struct PythonError {};  // an exception is set already

[[noreturn]] void refuse(int status, const char *fmt, ...) {
    Refusal r;
    r.status = status;
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(r.text, sizeof r.text, fmt, ap);
    va_end(ap);
    throw r;
}

// Runs `body`, turning what it throws into a Python exception.
template <typename Body>
PyObject *guarded(Body body) {
    try {
        return body();
    } catch (const Refusal &r) {
        PyObject *e = PyObject_CallFunction(g_error, "is", r.status, r.text);
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
    } catch (const PythonError &) {
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(g_no_memory, e.what_without_backtrace());
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PROJ_ERR_INVALID_ARG, "%s must be a tensor", name);
    return THPVariable_Unpack(o);
}
// None: an undefined tensor.
at::Tensor optional(PyObject *o, const char *name) { return o == Py_None ? at::Tensor() : tensor(o, name); }

int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    return v;
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError();
    return v;
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError();
    return v != 0;
}
// Sizes that the C ABI takes as 32 bits: what does not fit is out of its range anyway.
int32_t narrow(int64_t v) { return static_cast<int32_t>(std::min<int64_t>(std::max<int64_t>(v, INT32_MIN), INT32_MAX)); }

// The current CUDA device, which every tensor must be on.
int device_of(std::initializer_list<const at::Tensor *> tensors) {
    int dev = -2;
    for (const at::Tensor *t : tensors) {
        if (!t->defined()) continue;
        const int d = t->is_cuda() ? t->get_device() : -1;
        if (dev == -2) dev = d;
        if (d != dev || d < 0)
            refuse(PROJ_ERR_INVALID_ARG, "every tensor must be on the current CUDA device (one is on %s)", t->device().str().c_str());
    }
    PyObject *o = PyObject_CallNoArgs(g_get_device);
    if (!o) throw PythonError();
    const long cur = PyLong_AsLong(o);
    Py_DECREF(o);
    if (cur != dev) refuse(PROJ_ERR_INVALID_ARG, "every tensor must be on the current CUDA device (%ld; they are on %d)", cur, dev);
    return dev;
}

// The stream of the call: the given raw pointer, or the device's current stream.
proj_stream_t stream_of(PyObject *stream, int dev) {
    PyObject *o = stream;
    if (stream == Py_None) {
        PyObject *d = PyLong_FromLong(dev);
        o = d ? PyObject_CallOneArg(g_get_stream, d) : nullptr;
        Py_XDECREF(d);
        if (!o) throw PythonError();
    } else {
        Py_INCREF(o);
    }
    void *p = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    if (!p && PyErr_Occurred()) throw PythonError();
    return static_cast<proj_stream_t>(p);
}

at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, int dev) {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<at::DeviceIndex>(dev)));
}

const int32_t *ints(const char *name, const at::Tensor &t, int64_t n) {
    if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
        refuse(PROJ_ERR_INVALID_ARG, "%s must be a dense 1-D int32 tensor of %lld elements", name, (long long)n);
    return static_cast<const int32_t *>(t.data_ptr());
}
int32_t *ints_out(const char *name, const at::Tensor &t, int64_t n) { return const_cast<int32_t *>(ints(name, t, n)); }

proj_page_index page_index(const at::Tensor &table, const at::Tensor &lens, const at::Tensor &refs, int64_t num_pages,
                           int64_t page_size) {
    if (table.scalar_type() != at::kInt || table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1))
        refuse(PROJ_ERR_INVALID_ARG, "block_table must be a 2-D int32 tensor with dense rows");
    proj_page_index ix;
    ix.block_table = static_cast<int32_t *>(table.data_ptr());
    ix.num_rows = narrow(table.size(0));
    ix.max_pages = narrow(table.size(1));
    ix.table_stride = table.size(0) > 1 ? table.stride(0) : std::max<int64_t>(table.stride(0), table.size(1));
    ix.seq_lens = ints_out("seq_lens", lens, table.size(0));
    ix.ref_counts = refs.defined() ? ints_out("ref_counts", refs, num_pages) : nullptr;
    ix.num_pages = narrow(num_pages);
    ix.page_size = narrow(page_size);
    return ix;
}

// v_dim None: the values' columns, or 512 of a latent cache.
proj_kv_pages kv_pages(const at::Tensor &k, const at::Tensor &v, PyObject *v_dim_or_none) {
    const bool given = v_dim_or_none != Py_None;
    const int64_t v_dim = given ? integer(v_dim_or_none) : 512;
    if (k.dim() != 4 || k.stride(3) != 1)
        refuse(PROJ_ERR_INVALID_ARG, "k_pages must be a [num_pages, page_size, kv_heads, k_dim] tensor with dense columns");
    if (k.scalar_type() != at::kBFloat16 || (v.defined() && v.scalar_type() != at::kBFloat16))
        refuse(PROJ_ERR_UNSUPPORTED_DTYPE, "the cache holds bf16");
    proj_kv_pages p = {};
    p.k = k.data_ptr();
    p.kv_heads = narrow(k.size(2));
    p.k_dim = narrow(k.size(3));
    p.k_page_stride = k.stride(0);
    p.k_token_stride = k.stride(1);
    p.k_head_stride = k.stride(2);
    if (!v.defined()) {
        p.v_dim = narrow(v_dim);
        return p;
    }
    if (v.dim() != 4 || v.stride(3) != 1 || v.size(0) != k.size(0) || v.size(1) != k.size(1) || v.size(2) != k.size(2))
        refuse(PROJ_ERR_INVALID_ARG, "v_pages must be a [num_pages, page_size, kv_heads, v_dim] tensor like k_pages");
    if (given && v_dim != v.size(3))
        refuse(PROJ_ERR_INVALID_ARG, "v_dim=%lld, but v_pages has %lld columns", (long long)v_dim, (long long)v.size(3));
    p.v = v.data_ptr();
    p.v_dim = narrow(v.size(3));
    p.v_page_stride = v.stride(0);
    p.v_token_stride = v.stride(1);
    p.v_head_stride = v.stride(2);
    return p;
}

// A sequence of pools [layers, num_pages, ...] with dense pages.
struct Pools {
    std::vector<at::Tensor> tensors;
    std::vector<proj_page_pool> pools;
    int64_t num_pages = -1;  // -1: not known yet
};
void read_pools(PyObject *seq, Pools *out) {
    PyObject *fast = PySequence_Fast(seq, "pools must be a sequence of tensors");
    if (!fast) throw PythonError();
    try {
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(fast);
        for (Py_ssize_t i = 0; i < n; ++i) {
            const at::Tensor &t = tensor(PySequence_Fast_GET_ITEM(fast, i), "a pool");
            if (t.dim() < 3 || (out->num_pages >= 0 && t.size(1) != out->num_pages))
                refuse(PROJ_ERR_INVALID_ARG, "a pool is a [layers, num_pages, ...] tensor");
            int64_t page = 1;
            for (int64_t d = t.dim() - 1; d >= 2; --d) {
                if (t.size(d) != 1 && t.stride(d) != page) refuse(PROJ_ERR_INVALID_ARG, "the pages of a pool must be dense");
                page *= t.size(d);
            }
            out->num_pages = t.size(1);
            const int64_t e = t.element_size();
            proj_page_pool p = {};
            p.base = t.data_ptr();
            p.layers = narrow(t.size(0));
            p.page_bytes = page * e;
            p.layer_stride = t.size(0) > 1 ? t.stride(0) * e : page * e;
            p.page_stride = t.size(1) > 1 ? t.stride(1) * e : page * e;
            out->pools.push_back(p);
            out->tensors.push_back(t);
        }
    } catch (...) {
        Py_DECREF(fast);
        throw;
    }
    Py_DECREF(fast);
}
void same_device(const Pools &p, int dev) {
    for (const at::Tensor &t : p.tensors)
        if (!t.is_cuda() || t.get_device() != dev)
            refuse(PROJ_ERR_INVALID_ARG, "every tensor must be on the current CUDA device (a pool is on %s)", t.device().str().c_str());
}

// The C call with the interpreter lock released.
template <typename Call>
void run(Call call) {
    proj_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = call();
    Py_END_ALLOW_THREADS;
    if (st != PROJ_OK) refuse(st, "%s", proj_last_error_string());
}

struct Workspace {
    c10::DataPtr own;  // (torch's allocator, on the current stream, like a tensor of its own but quicker to have)
    void *ptr = nullptr;
    size_t bytes = 0;
};
// `need` of 0: sizes that the C call refuses, which then says why.
void use(Workspace *w, const at::Tensor &given, size_t need) {
    if (!given.defined()) {
        if (need == 0) return;
        w->own = c10::GetAllocator(c10::kCUDA)->allocate(need);
        w->ptr = w->own.get();
        w->bytes = need;
        return;
    }
    if (!given.is_contiguous()) refuse(PROJ_ERR_INVALID_ARG, "workspace must be dense");
    w->ptr = given.data_ptr();
    w->bytes = given.nbytes();
}

void arguments(Py_ssize_t have, Py_ssize_t want) {
    if (have != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", have, want);
        throw PythonError();
    }
}

// (q, k_pages, v_pages, block_table, seq_lens, scale, v_dim, rows, out, lse, return_lse, workspace, stream)
PyObject *paged_attention(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject * {
        arguments(nargs, 13);
        const at::Tensor &q = tensor(args[0], "q"), &k = tensor(args[1], "k_pages");
        const at::Tensor v = optional(args[2], "v_pages");
        const at::Tensor &table = tensor(args[3], "block_table"), &lens = tensor(args[4], "seq_lens");
        const float scale = static_cast<float>(number(args[5]));
        const at::Tensor rows = optional(args[7], "rows");
        at::Tensor out = optional(args[8], "out"), lse = optional(args[9], "lse");
        const bool return_lse = truth(args[10]);
        const at::Tensor given = optional(args[11], "workspace");
        const int dev = device_of({&q, &k, &v, &table, &lens, &rows, &out, &lse, &given});
        const proj_kv_pages kv = kv_pages(k, v, args[6]);
        if (q.dim() != 3 || q.size(2) != kv.k_dim || q.stride(2) != 1)
            refuse(PROJ_ERR_INVALID_ARG, "q must be a [batch, heads, k_dim] tensor with dense columns");
        if (q.scalar_type() != at::kBFloat16) refuse(PROJ_ERR_UNSUPPORTED_DTYPE, "unsupported tensor dtype %s", c10::toString(q.scalar_type()));
        const int64_t batch = q.size(0), heads = q.size(1), dv = kv.v_dim;
        if (dv < 1 || dv > kv.k_dim)  // (before out is made)
            refuse(PROJ_ERR_UNSUPPORTED_SHAPE, "k_dim=%d, v_dim=%d: the values are at most as wide as the keys", kv.k_dim, kv.v_dim);
        const proj_page_index ix = page_index(table, lens, at::Tensor(), k.size(0), k.size(1));
        if (!out.defined()) out = make({batch, heads, dv}, at::kBFloat16, dev);
        else if (out.sizes() != at::IntArrayRef({batch, heads, dv}) || out.scalar_type() != at::kBFloat16 || !out.is_contiguous())
            refuse(PROJ_ERR_INVALID_ARG, "out must be a dense [%lld, %lld, %lld] bf16 tensor", (long long)batch, (long long)heads, (long long)dv);
        if (!lse.defined()) {
            if (return_lse) lse = make({batch, heads}, at::kFloat, dev);
        } else if (lse.sizes() != at::IntArrayRef({batch, heads}) || lse.scalar_type() != at::kFloat || !lse.is_contiguous()) {
            refuse(PROJ_ERR_INVALID_ARG, "lse must be a dense [%lld, %lld] float32 tensor", (long long)batch, (long long)heads);
        }
        const int32_t *rp = rows.defined() ? ints("rows", rows, batch) : nullptr;
        Workspace ws;
        if (given.defined() || static_cast<int64_t>(ix.max_pages) * ix.page_size > PROJ_UNCUT_TOKENS)
            use(&ws, given, given.defined() ? 0 : proj_paged_attention_workspace_bytes(narrow(heads), kv.kv_heads, kv.k_dim, kv.v_dim, !v.defined()));
        const proj_stream_t stream = stream_of(args[12], dev);
        const void *qp = q.data_ptr();
        void *op = out.data_ptr();
        float *lp = lse.defined() ? static_cast<float *>(lse.data_ptr()) : nullptr;
        const int64_t qs = q.stride(0), qh = q.stride(1);
        run([&] {
            return proj_paged_attention(qp, qs, qh, &kv, &ix, rp, narrow(batch), narrow(heads), scale, op, lp, ws.ptr, ws.bytes, stream);
        });
        if (!return_lse) return THPVariable_Wrap(out);
        PyObject *a = THPVariable_Wrap(out), *b = THPVariable_Wrap(lse);
        PyObject *both = a && b ? PyTuple_Pack(2, a, b) : nullptr;
        Py_XDECREF(a);
        Py_XDECREF(b);
        return both;
    });
}

// Pointer and token stride of new rows [tokens, heads, dim] or [tokens, heads * dim].
const void *new_rows(const char *name, const at::Tensor &t, int64_t tokens, int64_t heads, int64_t dim, int64_t *stride) {
    if (t.scalar_type() != at::kBFloat16) refuse(PROJ_ERR_UNSUPPORTED_DTYPE, "unsupported tensor dtype %s", c10::toString(t.scalar_type()));
    const bool flat = t.dim() == 2 && t.size(0) == tokens && t.size(1) == heads * dim && t.stride(1) == 1;
    const bool deep = t.dim() == 3 && t.size(0) == tokens && t.size(1) == heads && t.size(2) == dim && t.stride(2) == 1 &&
                      (heads == 1 || t.stride(1) == dim);
    if (!flat && !deep)
        refuse(PROJ_ERR_INVALID_ARG, "%s must be [tokens, %lld, %lld] with dense tokens", name, (long long)heads, (long long)dim);
    *stride = tokens > 1 ? t.stride(0) : heads * dim;
    return t.data_ptr();
}

// (k_new, v_new, k_pages, v_pages, block_table, seq_lens, rows, positions, cos_sin, interleaved, q, q_out, stream, ref_counts)
PyObject *cache_append(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject * {
        arguments(nargs, 14);
        const at::Tensor &kn = tensor(args[0], "k_new"), &k = tensor(args[2], "k_pages");
        const at::Tensor vn = optional(args[1], "v_new"), v = optional(args[3], "v_pages");
        const at::Tensor &table = tensor(args[4], "block_table"), &lens = tensor(args[5], "seq_lens");
        const at::Tensor rows = optional(args[6], "rows"), pos = optional(args[7], "positions"), cs = optional(args[8], "cos_sin");
        const at::Tensor q = optional(args[10], "q");
        at::Tensor q_out = optional(args[11], "q_out");
        const at::Tensor refs = optional(args[13], "ref_counts");
        const int dev = device_of({&kn, &vn, &k, &v, &table, &lens, &rows, &pos, &cs, &q, &q_out, &refs});
        const proj_kv_pages kv = kv_pages(k, v, Py_None);
        if (kn.dim() < 1) refuse(PROJ_ERR_INVALID_ARG, "k_new must be [tokens, ...]");
        const int64_t tokens = kn.size(0), dim = kv.k_dim;
        if (vn.defined() != v.defined()) refuse(PROJ_ERR_INVALID_ARG, "v_new goes with a cache that has values of its own");
        int64_t ks = 0, vs = 0;
        const void *kp = new_rows("k_new", kn, tokens, kv.kv_heads, dim, &ks);
        const void *vp = vn.defined() ? new_rows("v_new", vn, tokens, kv.kv_heads, kv.v_dim, &vs) : nullptr;
        const proj_page_index ix = page_index(table, lens, refs, k.size(0), k.size(1));
        proj_rotary rot = {};
        if (cs.defined()) {
            if (cs.scalar_type() != at::kFloat || cs.dim() != 2 || !cs.is_contiguous())
                refuse(PROJ_ERR_INVALID_ARG, "cos_sin must be a dense [max_pos, rot] float32 tensor");
            rot.cos_sin = static_cast<const float *>(cs.data_ptr());
            rot.max_pos = narrow(cs.size(0));
            rot.dim = narrow(cs.size(1));
            rot.interleaved = truth(args[9]);
        }
        int64_t heads = 0, qs = 0, qh = 0, os = 0, oh = 0;
        if (q.defined()) {
            if (!q_out.defined()) q_out = make(q.sizes(), at::kBFloat16, dev);
            if (q.dim() != 3 || q.size(0) != tokens || q.size(2) != dim || q_out.sizes() != q.sizes() || q.stride(2) != 1 ||
                q_out.stride(2) != 1)
                refuse(PROJ_ERR_INVALID_ARG, "q and q_out must be [tokens, heads, %lld] with dense columns", (long long)dim);
            if (q.scalar_type() != at::kBFloat16 || q_out.scalar_type() != at::kBFloat16)
                refuse(PROJ_ERR_UNSUPPORTED_DTYPE, "unsupported tensor dtype %s", c10::toString(q.scalar_type()));
            heads = q.size(1);
            qs = q.stride(0);
            qh = q.stride(1);
            os = q_out.stride(0);
            oh = q_out.stride(1);
        }
        const int32_t *rp = rows.defined() ? ints("rows", rows, tokens) : nullptr;
        const int32_t *pp = pos.defined() ? ints("positions", pos, tokens) : nullptr;
        const proj_stream_t stream = stream_of(args[12], dev);
        const void *qp = q.defined() ? q.data_ptr() : nullptr;
        void *op = q.defined() ? q_out.data_ptr() : nullptr;
        run([&] {
            return proj_cache_append(kp, ks, vp, vs, &kv, &ix, rp, pp, narrow(tokens), cs.defined() ? &rot : nullptr, qp, qs, qh, op,
                                     os, oh, narrow(heads), stream);
        });
        if (!q.defined()) Py_RETURN_NONE;
        if (args[11] != Py_None) return Py_NewRef(args[11]);
        return THPVariable_Wrap(q_out);
    });
}

// (block_table, seq_lens, ref_counts, rows, new_lens, page_size, pools, status, workspace, stream)
PyObject *cache_resize(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject * {
        arguments(nargs, 10);
        const at::Tensor &table = tensor(args[0], "block_table"), &lens = tensor(args[1], "seq_lens"), &refs = tensor(args[2], "ref_counts");
        const at::Tensor &rows = tensor(args[3], "rows"), &want = tensor(args[4], "new_lens");
        at::Tensor status = optional(args[7], "status");
        const at::Tensor given = optional(args[8], "workspace");
        const int dev = device_of({&table, &lens, &refs, &rows, &want, &status, &given});
        Pools pools;
        pools.num_pages = refs.dim() > 0 ? refs.size(0) : 0;
        read_pools(args[6], &pools);
        same_device(pools, dev);
        const proj_page_index ix = page_index(table, lens, refs, refs.numel(), integer(args[5]));
        const int64_t n = rows.numel();
        if (!status.defined()) status = make({n}, at::kInt, dev);
        int32_t *sp = ints_out("status", status, n);
        const int32_t *rp = ints("rows", rows, n), *wp = ints("new_lens", want, n);
        Workspace ws;
        use(&ws, given, given.defined() ? 0 : proj_cache_workspace_bytes(&ix, narrow(n)));
        const proj_stream_t stream = stream_of(args[9], dev);
        run([&] {
            return proj_cache_resize(&ix, rp, wp, narrow(n), pools.pools.data(), narrow(static_cast<int64_t>(pools.pools.size())), sp,
                                     ws.ptr, ws.bytes, stream);
        });
        return args[7] != Py_None ? Py_NewRef(args[7]) : THPVariable_Wrap(status);
    });
}

// (block_table, seq_lens, ref_counts, parents, children, page_size, status, stream)
PyObject *cache_fork(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject * {
        arguments(nargs, 8);
        const at::Tensor &table = tensor(args[0], "block_table"), &lens = tensor(args[1], "seq_lens"), &refs = tensor(args[2], "ref_counts");
        const at::Tensor &parents = tensor(args[3], "parents"), &children = tensor(args[4], "children");
        at::Tensor status = optional(args[6], "status");
        const int dev = device_of({&table, &lens, &refs, &parents, &children, &status});
        const proj_page_index ix = page_index(table, lens, refs, refs.numel(), integer(args[5]));
        const int64_t n = parents.numel();
        if (!status.defined()) status = make({n}, at::kInt, dev);
        int32_t *sp = ints_out("status", status, n);
        const int32_t *pp = ints("parents", parents, n), *cp = ints("children", children, n);
        const proj_stream_t stream = stream_of(args[7], dev);
        run([&] { return proj_cache_fork(&ix, pp, cp, narrow(n), sp, stream); });
        return args[6] != Py_None ? Py_NewRef(args[6]) : THPVariable_Wrap(status);
    });
}

// (block_table, seq_lens, ref_counts, page_size, pools, live, workspace, stream)
PyObject *cache_compact(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject * {
        arguments(nargs, 8);
        const at::Tensor &table = tensor(args[0], "block_table"), &lens = tensor(args[1], "seq_lens"), &refs = tensor(args[2], "ref_counts");
        at::Tensor live = optional(args[5], "live");
        const at::Tensor given = optional(args[6], "workspace");
        const int dev = device_of({&table, &lens, &refs, &live, &given});
        Pools pools;
        pools.num_pages = refs.dim() > 0 ? refs.size(0) : 0;
        read_pools(args[4], &pools);
        same_device(pools, dev);
        const proj_page_index ix = page_index(table, lens, refs, refs.numel(), integer(args[3]));
        if (!live.defined()) live = make({1}, at::kInt, dev);
        int32_t *lp = ints_out("live", live, 1);
        Workspace ws;
        use(&ws, given, given.defined() ? 0 : proj_cache_workspace_bytes(&ix, 0));
        const proj_stream_t stream = stream_of(args[7], dev);
        run([&] {
            return proj_cache_compact(&ix, pools.pools.data(), narrow(static_cast<int64_t>(pools.pools.size())), lp, ws.ptr, ws.bytes, stream);
        });
        return args[5] != Py_None ? Py_NewRef(args[5]) : THPVariable_Wrap(live);
    });
}

// (pools, src, dst, stream); src and dst are CPU tensors
PyObject *cache_copy_pages(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject * {
        arguments(nargs, 4);
        Pools pools;
        read_pools(args[0], &pools);
        if (pools.tensors.empty()) refuse(PROJ_ERR_INVALID_ARG, "no pools");
        const int dev = device_of({&pools.tensors[0]});
        same_device(pools, dev);
        const at::Tensor &src = tensor(args[1], "src"), &dst = tensor(args[2], "dst");
        if (!src.device().is_cpu() || !dst.device().is_cpu()) refuse(PROJ_ERR_INVALID_ARG, "src and dst must be on the host");
        const int64_t n = src.numel();
        const int32_t *sp = ints("src", src, n), *dp = ints("dst", dst, n);
        const proj_stream_t stream = stream_of(args[3], dev);
        run([&] {
            return proj_cache_copy_pages(pools.pools.data(), narrow(static_cast<int64_t>(pools.pools.size())), narrow(pools.num_pages), sp,
                                         dp, narrow(n), stream);
        });
        Py_RETURN_NONE;
    });
}

// (ProjError)
PyObject *set_error(PyObject *, PyObject *cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(paged_attention)), METH_FASTCALL, nullptr},
    {"cache_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(cache_append)), METH_FASTCALL, nullptr},
    {"cache_resize", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(cache_resize)), METH_FASTCALL, nullptr},
    {"cache_fork", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(cache_fork)), METH_FASTCALL, nullptr},
    {"cache_compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(cache_compact)), METH_FASTCALL, nullptr},
    {"cache_copy_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(cache_copy_pages)), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "hsp_cache_py", "Tensors to the C ABI of the paged cache.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_hsp_cache_py() {
    PyObject *c = PyImport_ImportModule("torch._C");
    if (!c) return nullptr;
    g_get_device = PyObject_GetAttrString(c, "_cuda_getDevice");
    g_get_stream = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
    g_no_memory = PyObject_GetAttrString(c, "OutOfMemoryError");
    Py_DECREF(c);
    if (!g_get_device || !g_get_stream || !g_no_memory) return nullptr;
    g_error = Py_NewRef(PyExc_RuntimeError);
    return PyModule_Create(&kModule);
}
