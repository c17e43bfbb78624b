// q8_torch.cpp -- the tensor helpers of the paged cache, the attention and the calls around a layer's projections
// (attn_decode, kv_append, residual_norm, lora, ...) as a CPython module: argument checks, output tensors and the call, nothing else.  These calls take 3 to 10 us on
// the GPU, and the same marshalling through ctypes and tensor methods took 10 to 14 us of host time a call
// (measured on Grace; here 5 to 7 us, of which the launch itself is 3).
//
// The module does not link libq8.so: the package hands it the entry points it loaded (init).
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/q8.h"

namespace {

PyObject *g_error = nullptr;   // Q8Error

decltype(&q8_kv_page_bytes) f_page_bytes;
decltype(&q8_kv_append) f_append;
decltype(&q8_attn_decode) f_decode;
decltype(&q8_attn_prompt) f_prompt;
decltype(&q8_kv_reserve) f_reserve;
decltype(&q8_kv_fork) f_fork;
decltype(&q8_kv_free) f_free;
decltype(&q8_kv_compact) f_compact;
decltype(&q8_kv_copy) f_copy;
decltype(&q8_kv_read) f_read;
decltype(&q8_residual_norm) f_residual;
decltype(&q8_lora) f_lora;

struct Raised {};   // a Python exception is set

[[noreturn]] void raise(PyObject *kind, const char *what) {
    PyErr_SetString(kind, what);
    throw Raised{};
}

[[noreturn]] void raise_status(int rc, const char *what) {
    PyObject *e = PyObject_CallFunction(g_error, "is", rc, what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s: a tensor expected", name);
        throw Raised{};
    }
    return THPVariable_Unpack(o);
}

long long integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

uint32_t word(PyObject *o, const char *name) {
    const long long v = integer(o);
    if (v < 0 || v > 0xffffffffll) {
        PyErr_Format(PyExc_ValueError, "%s: out of range", name);
        throw Raised{};
    }
    return (uint32_t)v;
}

// Contiguous int32 GPU tensor (None: null).
const int32_t *ints(PyObject *o, const char *name, int64_t *n = nullptr) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != at::kInt || !t.is_cuda() || !t.is_contiguous()) {
        PyErr_Format(PyExc_TypeError, "%s: contiguous int32 on the GPU expected", name);
        throw Raised{};
    }
    if (n) *n = t.numel();
    return static_cast<const int32_t *>(t.data_ptr());
}

int64_t length(PyObject *o, const char *name) {
    const at::Tensor &t = tensor(o, name);
    return t.dim() == 1 ? t.size(0) : -1;
}

struct Table {
    int32_t *p = nullptr;
    int64_t stride = 0, width = 0, rows = 0;
};

Table table_of(PyObject *o) {
    const at::Tensor &t = tensor(o, "table");
    if (t.dim() != 2 || t.scalar_type() != at::kInt || !t.is_cuda() || (t.stride(1) != 1 && t.size(1) != 1))
        raise(PyExc_TypeError, "table: int32 [rows, max_pages] on the GPU with contiguous rows expected");
    Table r;
    r.p = static_cast<int32_t *>(t.data_ptr());
    r.rows = t.size(0);
    r.width = t.size(1);
    r.stride = r.rows > 1 ? t.stride(0) : r.width;
    return r;
}

// [rows, heads, dim] GPU tensor whose heads lie back to back: its row stride.
int64_t row_stride(const at::Tensor &t, const char *name) {
    if (t.dim() != 3 || !t.is_cuda() || t.stride(2) != 1 || (t.stride(1) != t.size(2) && t.size(1) != 1)) {
        PyErr_Format(PyExc_ValueError, "%s: a GPU tensor whose heads lie back to back expected", name);
        throw Raised{};
    }
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
}

int type16(at::ScalarType t) {
    if (t == at::kBFloat16) return Q8_TYPE_BF16;
    if (t == at::kHalf) return Q8_TYPE_F16;
    raise(PyExc_TypeError, "float16 or bfloat16 expected");
}

const float *sinks_of(PyObject *o, int64_t heads) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, "sinks");
    if (t.scalar_type() != at::kFloat || t.numel() != heads || !t.is_contiguous() || !t.is_cuda())
        raise(PyExc_TypeError, "sinks: contiguous float32 [heads] on the GPU expected");
    return static_cast<const float *>(t.data_ptr());
}

// Output [rows, heads, dim], or [rows, heads, dim / 32 * 34] Q8_0 blocks; out_type None: q's type.
at::Tensor output(const at::Tensor &q, int64_t rows, int64_t heads, int64_t dim, int kind, PyObject *o, int &out_type) {
    out_type = o == Py_None ? kind : (int)integer(o);
    if (out_type == kind) return at::empty({rows, heads, dim}, q.options());
    if (out_type == Q8_TYPE_F32) return at::empty({rows, heads, dim}, q.options().dtype(at::kFloat));
    if (out_type == Q8_TYPE_Q8_0) return at::empty({rows, heads, dim / Q8_BLOCK * Q8_BLOCK_BYTES}, q.options().dtype(at::kByte));
    raise_status(Q8_EINVAL, "out_type");
}

// What a KVCache's address points to: the cache, and the device of its pages (-1: the host).
struct Cache {
    q8_kv_cache c;
    int32_t device;
};

const q8_kv_cache *cache_of(PyObject *o) { return o == Py_None ? nullptr : &static_cast<const Cache *>(PyLong_AsVoidPtr(o))->c; }

int device_of(const q8_kv_cache *c) { return reinterpret_cast<const Cache *>(c)->device; }

void on_gpu(const q8_kv_cache *c) {
    if (c && device_of(c) < 0) raise(PyExc_TypeError, "cache: pages on the GPU expected");
}

// The current stream, for a call on these tensors (None among them) and the cache: all on its device.
void *stream_for(const q8_kv_cache *c, PyObject *const *a, std::initializer_list<int> tensors) {
    const c10::cuda::CUDAStream st = c10::cuda::getCurrentCUDAStream();
    bool here = !c || device_of(c) == st.device_index();
    for (const int i : tensors) here = here && (a[i] == Py_None || THPVariable_Unpack(a[i]).get_device() == st.device_index());
    if (!here) raise(PyExc_ValueError, "tensors and a cache on the current device expected");
    return st.stream();
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }

// A tensor of the caller's that a call wrote: autograd has to see that it changed, or a gradient that needs its old values
// would be computed from the new ones.
void written(const at::Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

PyObject *none_or(const at::Tensor &t) {
    if (t.defined()) return wrap(t);
    Py_RETURN_NONE;
}

template <class F> void call(const char *what, F f) {
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = f();
    Py_END_ALLOW_THREADS;
    if (rc) raise_status(rc, what);
}

void arity(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) raise(PyExc_TypeError, "wrong number of arguments");
}

// fill_cache(address, k, v, type, page_tokens, n_kv_heads, head_dim)
PyObject *fill_cache(PyObject *const *a, Py_ssize_t n) {
    arity(n, 7);
    Cache *const cache = static_cast<Cache *>(PyLong_AsVoidPtr(a[0]));
    q8_kv_cache *const c = &cache->c;
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const int type = (int)integer(a[3]);
    const uint32_t tokens = word(a[4], "page_tokens"), kv = word(a[5], "n_kv_heads"), dim = word(a[6], "head_dim");
    const uint64_t page = f_page_bytes(type, tokens, kv, dim);
    if (!page) raise_status(Q8_EINVAL, "q8_kv_page_bytes");
    if (k.dim() < 3 || k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type() || k.strides() != v.strides() ||
        k.device() != v.device())
        raise(PyExc_ValueError, "k and v must have the same shape, type, strides and device: [n_layers, n_pages, ...]");
    // bytes (any integer type) hold every format; values only their own
    if (at::isFloatingType(k.scalar_type()) &&
        !(type == Q8_TYPE_F16 && k.scalar_type() == at::kHalf) && !(type == Q8_TYPE_BF16 && k.scalar_type() == at::kBFloat16))
        raise(PyExc_TypeError, "k and v: values of the cache's type, or bytes, expected");
    int64_t want = 1;
    for (int64_t i = k.dim() - 1; i >= 2; --i) {
        if (k.stride(i) != want && k.size(i) != 1) raise(PyExc_ValueError, "a page must be contiguous");
        want *= k.size(i);
    }
    const int64_t size = k.element_size();
    if ((uint64_t)(want * size) != page) {
        PyErr_Format(PyExc_ValueError, "a page has %lld bytes, its layout %llu", (long long)(want * size), (unsigned long long)page);
        throw Raised{};
    }
    c->k = k.data_ptr();
    c->v = v.data_ptr();
    c->page_stride = k.size(1) > 1 ? k.stride(1) * size : page;
    c->layer_stride = k.size(0) > 1 ? k.stride(0) * size : k.size(1) * c->page_stride;
    c->n_layers = (uint32_t)k.size(0);
    c->n_pages = (uint32_t)k.size(1);
    c->page_tokens = tokens;
    c->n_kv_heads = kv;
    c->head_dim = dim;
    c->type = type;
    cache->device = k.is_cuda() ? k.get_device() : -1;
    Py_RETURN_NONE;
}

// kv_append(cache, layer, q, k, v, positions, seq_of, table, cos_sin, rope, out_type, want_kv)
PyObject *kv_append(PyObject *const *a, Py_ssize_t n) {
    arity(n, 12);
    const q8_kv_cache *c = cache_of(a[0]);
    on_gpu(c);
    const uint32_t layer = word(a[1], "layer");
    const at::Tensor &k = tensor(a[3], "k"), &v = tensor(a[4], "v");
    const int rope = (int)integer(a[9]), kind = (int)integer(a[10]);
    if (k.scalar_type() != at::kFloat || v.scalar_type() != at::kFloat) raise(PyExc_TypeError, "k and v: float32 expected");
    if (k.dim() != 3 || v.sizes() != k.sizes() || length(a[5], "positions") != k.size(0))
        raise(PyExc_ValueError, "k, v and positions disagree");
    const int64_t tok = k.size(0), kv = k.size(1), dim = k.size(2);
    const auto opt = k.options().dtype(kind == Q8_TYPE_BF16 ? at::kBFloat16 : at::kHalf);
    at::Tensor qo, ko, vo;
    const float *qp = nullptr;
    int64_t qs = 0, heads = 0;
    if (a[2] != Py_None) {
        const at::Tensor &q = tensor(a[2], "q");
        if (q.scalar_type() != at::kFloat) raise(PyExc_TypeError, "q: float32 expected");
        if (q.dim() != 3 || q.size(0) != tok || q.size(2) != dim) raise(PyExc_ValueError, "q and k disagree");
        heads = q.size(1);
        qs = row_stride(q, "q");
        qp = static_cast<const float *>(q.data_ptr());
        qo = at::empty({tok, heads, dim}, opt);
    }
    const int64_t kst = row_stride(k, "k"), vst = row_stride(v, "v");
    if (a[11] == Py_True) {
        ko = at::empty({tok, kv, dim}, opt);
        vo = at::empty({tok, kv, dim}, opt);
    }
    Table t;
    const int32_t *seq = nullptr;
    if (c) {
        if (a[6] == Py_None || a[7] == Py_None || length(a[6], "seq_of") != tok)
            raise(PyExc_ValueError, "a cache write needs seq_of [n] and table");
        seq = ints(a[6], "seq_of");
        t = table_of(a[7]);
    }
    const float *cs = nullptr;
    int64_t n_pos = 0, rot = 0;
    if (rope) {
        if (a[8] == Py_None) raise(PyExc_ValueError, "rope needs cos_sin");
        const at::Tensor &x = tensor(a[8], "cos_sin");
        if (x.dim() != 2 || x.scalar_type() != at::kFloat || !x.is_contiguous() || !x.is_cuda())
            raise(PyExc_ValueError, "rope needs a contiguous float32 cos_sin [n_pos, rot_dim] on the GPU");
        cs = static_cast<const float *>(x.data_ptr());
        n_pos = x.size(0);
        rot = x.size(1);
    }
    const int32_t *pos = ints(a[5], "positions");
    const float *kp = static_cast<const float *>(k.data_ptr()), *vp = static_cast<const float *>(v.data_ptr());
    void *qop = qo.defined() ? qo.data_ptr() : nullptr, *kop = ko.defined() ? ko.data_ptr() : nullptr,
         *vop = vo.defined() ? vo.data_ptr() : nullptr;
    void *st = c ? stream_for(c, a, {2, 3, 4, 5, 6, 7}) : stream_for(c, a, {2, 3, 4, 5});
    if (rope) stream_for(c, a, {8});
    call("q8_kv_append", [&] {
        return f_append(qop, kop, vop, kind, c, layer, qp, qs, kp, kst, vp, vst, (uint32_t)heads, (uint32_t)kv, (uint32_t)dim, pos,
                        seq, t.p, t.stride, (uint32_t)t.width, (uint32_t)t.rows, cs, (uint32_t)n_pos, (uint32_t)rot, rope, tok, st);
    });
    if (a[11] != Py_True) return none_or(qo);
    return Py_BuildValue("(NNN)", none_or(qo), wrap(ko), wrap(vo));
}

// attn_decode(q, cache, layer, table, seq_lens, scale, window, sinks, out_type, want_lse)
PyObject *attn_decode(PyObject *const *a, Py_ssize_t n) {
    arity(n, 10);
    const at::Tensor &q = tensor(a[0], "q");
    const q8_kv_cache *c = cache_of(a[1]);
    const uint32_t layer = word(a[2], "layer"), window = word(a[6], "window");
    if (q.dim() != 3 || q.size(2) != c->head_dim || tensor(a[3], "table").dim() != 2 || tensor(a[3], "table").size(0) != q.size(0) ||
        length(a[4], "seq_lens") != q.size(0))
        raise(PyExc_ValueError, "q, cache, table and seq_lens disagree");
    on_gpu(c);
    const int64_t seqs = q.size(0), heads = q.size(1), dim = q.size(2);
    const Table t = table_of(a[3]);
    const int32_t *lens = ints(a[4], "seq_lens");
    const int kind = type16(q.scalar_type());
    const int64_t qs = row_stride(q, "q");
    const float *sk = sinks_of(a[7], heads);
    const double scale = a[5] == Py_None ? 1.0 / std::sqrt((double)dim) : PyFloat_AsDouble(a[5]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    int out_type;
    const at::Tensor out = output(q, seqs, heads, dim, kind, a[8], out_type);
    at::Tensor lse;
    if (a[9] == Py_True) lse = at::empty({seqs, heads}, q.options().dtype(at::kFloat));
    void *op = out.data_ptr(), *qp = q.data_ptr(), *st = stream_for(c, a, {0, 3, 4, 7});
    float *lp = lse.defined() ? static_cast<float *>(lse.data_ptr()) : nullptr;
    call("q8_attn_decode", [&] {
        return f_decode(op, out_type, lp, qp, qs, kind, c, layer, t.p, t.stride, (uint32_t)t.width, lens, (uint32_t)seqs, (uint32_t)heads,
                        (float)scale, window, sk, st);
    });
    return lp ? Py_BuildValue("(NN)", wrap(out), wrap(lse)) : wrap(out);
}

// attn_prompt(q, k, v, q_start, k_start, scale, window, sinks, out_type, want_lse)
PyObject *attn_prompt(PyObject *const *a, Py_ssize_t n) {
    arity(n, 10);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const uint32_t window = word(a[6], "window");
    if (q.dim() != 3 || k.dim() != 3 || k.sizes() != v.sizes() || k.size(2) != q.size(2) || k.scalar_type() != q.scalar_type() ||
        v.scalar_type() != q.scalar_type())
        raise(PyExc_ValueError, "q, k and v disagree");
    const int64_t rows = q.size(0), heads = q.size(1), dim = q.size(2), n_start = length(a[3], "q_start");
    if (n_start < 1 || (a[4] != Py_None && length(a[4], "k_start") != n_start)) raise(PyExc_ValueError, "q_start and k_start disagree");
    const int32_t *qst = ints(a[3], "q_start"), *kst = ints(a[4], "k_start");
    const int kind = type16(q.scalar_type());
    const int64_t qs = row_stride(q, "q"), ks = row_stride(k, "k"), vs = row_stride(v, "v");
    const float *sk = sinks_of(a[7], heads);
    const double scale = a[5] == Py_None ? 1.0 / std::sqrt((double)dim) : PyFloat_AsDouble(a[5]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    int out_type;
    const at::Tensor out = output(q, rows, heads, dim, kind, a[8], out_type);
    at::Tensor lse;
    if (a[9] == Py_True) lse = at::empty({rows, heads}, q.options().dtype(at::kFloat));
    void *op = out.data_ptr(), *qp = q.data_ptr(), *kp = k.data_ptr(), *vp = v.data_ptr(), *st = stream_for(nullptr, a, {0, 1, 2, 3, 4, 7});
    float *lp = lse.defined() ? static_cast<float *>(lse.data_ptr()) : nullptr;
    const uint64_t n_k = k.size(0);
    const uint32_t kv = (uint32_t)k.size(1);
    call("q8_attn_prompt", [&] {
        return f_prompt(op, out_type, lp, qp, kp, vp, kind, qs, ks, vs, qst, kst, (uint32_t)(n_start - 1), rows, n_k, (uint32_t)heads, kv,
                        (uint32_t)dim, (float)scale, window, sk, st);
    });
    return lp ? Py_BuildValue("(NN)", wrap(out), wrap(lse)) : wrap(out);
}

// The arguments that the page calls share: cache, table, lens, refs.
struct Pages {
    const q8_kv_cache *c;
    Table t;
    int32_t *lens, *refs;
};

Pages pages_of(PyObject *const *a) {
    Pages p;
    p.c = cache_of(a[0]);
    on_gpu(p.c);
    p.t = table_of(a[1]);
    int64_t n_lens = 0, n_refs = 0;
    p.lens = const_cast<int32_t *>(ints(a[2], "lens", &n_lens));
    p.refs = const_cast<int32_t *>(ints(a[3], "refs", &n_refs));
    if (!p.lens || !p.refs || n_lens != p.t.rows || n_refs != p.c->n_pages)
        raise(PyExc_ValueError, "table, lens, refs and cache disagree");
    return p;
}

// kv_reserve / kv_fork(cache, table, lens, refs, rows, second list)
template <class F> PyObject *pages_two(PyObject *const *a, Py_ssize_t n, F f, const char *what) {
    arity(n, 6);
    const Pages p = pages_of(a);
    int64_t na = 0, nb = 0;
    const int32_t *x = ints(a[4], "rows", &na), *y = ints(a[5], "second list", &nb);
    if (na != nb) raise(PyExc_ValueError, "the two lists disagree");
    void *st = stream_for(p.c, a, {1, 2, 3, 4, 5});
    call(what, [&] { return f(p.c, p.t.p, p.t.stride, (uint32_t)p.t.width, (uint32_t)p.t.rows, p.lens, p.refs, x, y, (uint32_t)na, st); });
    Py_RETURN_NONE;
}

PyObject *kv_reserve(PyObject *const *a, Py_ssize_t n) { return pages_two(a, n, f_reserve, "q8_kv_reserve"); }
PyObject *kv_fork(PyObject *const *a, Py_ssize_t n) { return pages_two(a, n, f_fork, "q8_kv_fork"); }

// kv_free(cache, table, lens, refs, rows)
PyObject *kv_free(PyObject *const *a, Py_ssize_t n) {
    arity(n, 5);
    const Pages p = pages_of(a);
    int64_t na = 0;
    const int32_t *x = ints(a[4], "seqs", &na);
    void *st = stream_for(p.c, a, {1, 2, 3, 4});
    call("q8_kv_free", [&] {
        return f_free(p.c, p.t.p, p.t.stride, (uint32_t)p.t.width, (uint32_t)p.t.rows, p.lens, p.refs, x, (uint32_t)na, st);
    });
    Py_RETURN_NONE;
}

// kv_compact(cache, table, lens, refs) -> table, refs, used
PyObject *kv_compact(PyObject *const *a, Py_ssize_t n) {
    arity(n, 4);
    const Pages p = pages_of(a);
    const at::Tensor &t = tensor(a[1], "table");
    const at::Tensor nt = at::empty_strided({p.t.rows, p.t.width}, {p.t.stride, 1}, t.options());
    const at::Tensor nr = at::empty({(int64_t)p.c->n_pages}, t.options()), used = at::empty({}, t.options());
    int32_t *ntp = static_cast<int32_t *>(nt.data_ptr()), *nrp = static_cast<int32_t *>(nr.data_ptr()),
            *up = static_cast<int32_t *>(used.data_ptr());
    void *st = stream_for(p.c, a, {1, 2, 3});
    call("q8_kv_compact", [&] {
        return f_compact(p.c, ntp, p.t.p, p.t.stride, (uint32_t)p.t.width, (uint32_t)p.t.rows, nrp, p.refs, up, st);
    });
    return Py_BuildValue("(NNN)", wrap(nt), wrap(nr), wrap(used));
}

// kv_copy(cache, src, dst)
PyObject *kv_copy(PyObject *const *a, Py_ssize_t n) {
    arity(n, 3);
    const q8_kv_cache *c = cache_of(a[0]);
    on_gpu(c);
    int64_t na = 0, nb = 0;
    const int32_t *x = ints(a[1], "src", &na), *y = ints(a[2], "dst", &nb);
    if (na != nb) raise(PyExc_ValueError, "src and dst disagree");
    void *st = stream_for(c, a, {1, 2});
    call("q8_kv_copy", [&] { return f_copy(c, x, y, (uint32_t)na, st); });
    Py_RETURN_NONE;
}

// kv_read(cache, layer, table, k_start, n_k, seqs, first, out_type, k_out, v_out)
PyObject *kv_read(PyObject *const *a, Py_ssize_t n) {
    arity(n, 10);
    const q8_kv_cache *c = cache_of(a[0]);
    if (!c) raise(PyExc_TypeError, "cache: a KVCache expected");
    on_gpu(c);
    const uint32_t layer = word(a[1], "layer");
    const Table t = table_of(a[2]);
    const int64_t n_start = length(a[3], "k_start"), rows = word(a[4], "n_k");
    if (n_start < 1) raise(PyExc_ValueError, "k_start: [n_seq + 1] expected");
    if ((a[5] != Py_None && length(a[5], "seqs") != n_start - 1) || (a[6] != Py_None && length(a[6], "first") != n_start - 1) ||
        (a[5] == Py_None && n_start - 1 > t.rows))
        raise(PyExc_ValueError, "table, k_start, seqs and first disagree");
    const int32_t *start = ints(a[3], "k_start"), *seqs = ints(a[5], "seqs"), *first = ints(a[6], "first");
    int out_type = a[7] != Py_None ? (int)integer(a[7]) : c->type == Q8_TYPE_Q8_0 ? Q8_TYPE_BF16 : c->type;
    const int64_t heads = c->n_kv_heads, dim = c->head_dim;
    at::Tensor k, v;
    if (a[8] != Py_None || a[9] != Py_None) {
        if (a[8] == Py_None || a[9] == Py_None) raise(PyExc_ValueError, "out: both k and v expected");
        k = tensor(a[8], "k");
        v = tensor(a[9], "v");
        const int kind = k.scalar_type() == at::kFloat ? Q8_TYPE_F32 : type16(k.scalar_type());
        if (v.scalar_type() != k.scalar_type() || (a[7] != Py_None && kind != out_type)) raise(PyExc_TypeError, "out: k, v and out_type disagree");
        for (const at::Tensor *x : {&k, &v})
            if (x->dim() != 3 || x->size(0) < rows || x->size(1) != heads || x->size(2) != dim)
                raise(PyExc_ValueError, "out: k and v of at least n_k rows [n_kv_heads, head_dim] expected");
        out_type = kind;
    } else {
        const auto type = out_type == Q8_TYPE_F32 ? at::kFloat : out_type == Q8_TYPE_BF16 ? at::kBFloat16 : at::kHalf;
        if (out_type != Q8_TYPE_F32 && out_type != Q8_TYPE_BF16 && out_type != Q8_TYPE_F16) raise_status(Q8_EINVAL, "out_type");
        const auto opt = tensor(a[2], "table").options().dtype(type);
        k = at::empty({rows, heads, dim}, opt);
        v = at::empty({rows, heads, dim}, opt);
    }
    const int64_t ks = row_stride(k, "k"), vs = row_stride(v, "v");
    void *kp = k.data_ptr(), *vp = v.data_ptr(), *st = stream_for(c, a, {2, 3, 5, 6, 8, 9});
    call("q8_kv_read", [&] {
        return f_read(kp, ks, vp, vs, out_type, c, layer, t.p, t.stride, (uint32_t)t.width, (uint32_t)t.rows, seqs, first, start,
                      (uint32_t)(n_start - 1), rows, st);
    });
    if (a[8] != Py_None) {
        written(k);
        written(v);
    }
    return Py_BuildValue("(NN)", wrap(k), wrap(v));
}

// [rows, n] GPU tensor with contiguous rows: its row stride.
int64_t matrix_stride(const at::Tensor &t, int64_t rows, int64_t n, const char *name) {
    if (t.dim() != 2 || !t.is_cuda() || t.size(0) != rows || t.size(1) != n || (t.stride(1) != 1 && n != 1)) {
        PyErr_Format(PyExc_ValueError, "%s: a GPU tensor [%lld, %lld] with contiguous rows expected", name, (long long)rows, (long long)n);
        throw Raised{};
    }
    return rows > 1 ? t.stride(0) : n;
}

int value_type(const at::Tensor &t) { return t.scalar_type() == at::kFloat ? Q8_TYPE_F32 : type16(t.scalar_type()); }

const float *floats(PyObject *o, int64_t n, const char *name) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != at::kFloat || t.numel() != n || !t.is_contiguous() || !t.is_cuda()) {
        PyErr_Format(PyExc_TypeError, "%s: contiguous float32 of %lld values on the GPU expected", name, (long long)n);
        throw Raised{};
    }
    return static_cast<const float *>(t.data_ptr());
}

float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)v;
}

// residual_norm(h, y, gamma_next, eps, gamma_post, post, gate, residual_scale, out_type, h_out) -> n, h_out
// out_type None: no n; h_out None: a new tensor, False: not stored
PyObject *residual_norm(PyObject *const *a, Py_ssize_t n) {
    arity(n, 10);
    const at::Tensor &h = tensor(a[0], "h"), &y = tensor(a[1], "y");
    if (h.dim() != 2) raise(PyExc_ValueError, "h: [n_tok, dim] expected");
    const int64_t tok = h.size(0), dim = h.size(1);
    const int64_t hs = matrix_stride(h, tok, dim, "h"), ys = matrix_stride(y, tok, dim, "y");
    const int ht = value_type(h), yt = value_type(y), post = PyObject_IsTrue(a[5]);
    if (post < 0) throw Raised{};
    const float *next = floats(a[2], dim, "gamma_next"), *before = floats(a[4], dim, "gamma_post"), *gate = nullptr;
    const float eps = real(a[3]), scale = real(a[7]);
    int64_t gs = 0;
    if (a[6] != Py_None) {
        const at::Tensor &g = tensor(a[6], "gate");
        if (g.dim() == 1) gate = floats(a[6], dim, "gate");
        else {
            if (g.scalar_type() != at::kFloat) raise(PyExc_TypeError, "gate: float32 expected");
            gs = matrix_stride(g, tok, dim, "gate");
            gate = static_cast<const float *>(g.data_ptr());
        }
    }
    at::Tensor out, ho;
    int out_type = Q8_TYPE_F32;
    if (a[8] != Py_None) {
        out_type = (int)integer(a[8]);
        if (out_type == Q8_TYPE_Q8_0) out = at::empty({tok, dim / Q8_BLOCK * Q8_BLOCK_BYTES}, h.options().dtype(at::kByte));
        else if (out_type == Q8_TYPE_F32) out = at::empty({tok, dim}, h.options().dtype(at::kFloat));
        else if (out_type == Q8_TYPE_BF16) out = at::empty({tok, dim}, h.options().dtype(at::kBFloat16));
        else if (out_type == Q8_TYPE_F16) out = at::empty({tok, dim}, h.options().dtype(at::kHalf));
        else raise_status(Q8_EINVAL, "out_type");
    }
    int64_t hos = 0;
    if (a[9] == Py_None) {
        ho = at::empty({tok, dim}, h.options());
        hos = dim;
    } else if (a[9] != Py_False) {
        ho = tensor(a[9], "h_out");
        if (ho.scalar_type() != h.scalar_type()) raise(PyExc_TypeError, "h_out: h's type expected");
        hos = matrix_stride(ho, tok, dim, "h_out");
    }
    void *op = out.defined() ? out.data_ptr() : nullptr, *hop = ho.defined() ? ho.data_ptr() : nullptr;
    const void *hp = h.data_ptr(), *yp = y.data_ptr();
    void *st = a[9] == Py_False ? stream_for(nullptr, a, {0, 1, 2, 4, 6}) : stream_for(nullptr, a, {0, 1, 2, 4, 6, 9});
    call("q8_residual_norm", [&] {
        return f_residual(op, out_type, hop, hos, hp, ht, hs, yp, yt, ys, post, before, gate, gs, scale, next, eps, dim, tok, st);
    });
    if (a[9] != Py_None && a[9] != Py_False) written(ho);
    return Py_BuildValue("(NN)", none_or(out), none_or(ho));
}

// lora(x, a, b, adapter_of, ranks, scales, base, out) -> out
PyObject *lora(PyObject *const *a, Py_ssize_t n) {
    arity(n, 8);
    const at::Tensor &x = tensor(a[0], "x"), &wa = tensor(a[1], "a"), &wb = tensor(a[2], "b");
    if (x.dim() != 2 || wa.dim() != 3 || wb.dim() != 3 || wa.size(0) != wb.size(0) || wa.size(1) != wb.size(2))
        raise(PyExc_ValueError, "x [n_tok, in_dim], a [n, rank, in_dim] and b [n, out_dim, rank] expected");
    if (wa.scalar_type() != wb.scalar_type()) raise(PyExc_TypeError, "a and b: one type expected");
    const int64_t tok = x.size(0), in = wa.size(2), od = wb.size(1), rank = wa.size(1), count = wa.size(0);
    for (const at::Tensor *w : {&wa, &wb})
        if (!w->is_cuda() || (w->stride(2) != 1 && w->size(2) != 1) || (w->stride(1) != w->size(2) && w->size(1) != 1))
            raise(PyExc_ValueError, "a and b: adapters of contiguous rows on the GPU expected");
    q8_adapters ad{};
    ad.a = wa.data_ptr();
    ad.b = wb.data_ptr();
    ad.a_stride = count > 1 ? wa.stride(0) : rank * in;
    ad.b_stride = count > 1 ? wb.stride(0) : rank * od;
    ad.ranks = a[4] == Py_None ? nullptr : ints(a[4], "ranks");
    if (ad.ranks && length(a[4], "ranks") != count) raise(PyExc_ValueError, "ranks: [n] expected");
    ad.scales = floats(a[5], count, "scales");
    ad.in_dim = in;
    ad.out_dim = od;
    if (count > 0xffffffffll || rank > 0xffffffffll) raise(PyExc_ValueError, "a: out of range");
    ad.n_adapters = (uint32_t)count;
    ad.max_rank = (uint32_t)rank;
    ad.type = type16(wa.scalar_type());
    int xt;
    int64_t xs;
    if (x.scalar_type() == at::kByte) {
        xt = Q8_TYPE_Q8_0;
        if (!x.is_cuda() || !x.is_contiguous() || in % Q8_BLOCK || x.size(1) != in / Q8_BLOCK * Q8_BLOCK_BYTES)
            raise(PyExc_ValueError, "x: contiguous Q8_0 rows of in_dim values on the GPU expected");
        xs = in;
    } else {
        xt = value_type(x);
        xs = matrix_stride(x, tok, in, "x");
    }
    if (length(a[3], "adapter_of") != tok) raise(PyExc_ValueError, "adapter_of: [n_tok] expected");
    const int32_t *ids = ints(a[3], "adapter_of");
    const float *base = nullptr;
    int64_t bs = 0, os = od;
    if (a[6] != Py_None) {
        const at::Tensor &t = tensor(a[6], "base");
        if (t.scalar_type() != at::kFloat) raise(PyExc_TypeError, "base: float32 expected");
        bs = matrix_stride(t, tok, od, "base");
        base = static_cast<const float *>(t.data_ptr());
    }
    at::Tensor out;
    if (a[7] == Py_None) out = at::empty({tok, od}, x.options().dtype(at::kFloat));
    else {
        out = tensor(a[7], "out");
        if (out.scalar_type() != at::kFloat) raise(PyExc_TypeError, "out: float32 expected");
        os = matrix_stride(out, tok, od, "out");
    }
    float *op = static_cast<float *>(out.data_ptr());
    const void *xp = x.data_ptr();
    void *st = stream_for(nullptr, a, {0, 1, 2, 3, 4, 5, 6, 7});
    call("q8_lora", [&] { return f_lora(op, os, base, bs, xp, xt, xs, &ad, ids, tok, st); });
    if (a[7] != Py_None) written(out);
    return wrap(out);
}

// init(Q8Error, addresses of the twelve entry points)
PyObject *init(PyObject *const *a, Py_ssize_t n) {
    arity(n, 13);
    Py_INCREF(a[0]);
    g_error = a[0];
    f_page_bytes = reinterpret_cast<decltype(f_page_bytes)>(PyLong_AsVoidPtr(a[1]));
    f_append = reinterpret_cast<decltype(f_append)>(PyLong_AsVoidPtr(a[2]));
    f_decode = reinterpret_cast<decltype(f_decode)>(PyLong_AsVoidPtr(a[3]));
    f_prompt = reinterpret_cast<decltype(f_prompt)>(PyLong_AsVoidPtr(a[4]));
    f_reserve = reinterpret_cast<decltype(f_reserve)>(PyLong_AsVoidPtr(a[5]));
    f_fork = reinterpret_cast<decltype(f_fork)>(PyLong_AsVoidPtr(a[6]));
    f_free = reinterpret_cast<decltype(f_free)>(PyLong_AsVoidPtr(a[7]));
    f_compact = reinterpret_cast<decltype(f_compact)>(PyLong_AsVoidPtr(a[8]));
    f_copy = reinterpret_cast<decltype(f_copy)>(PyLong_AsVoidPtr(a[9]));
    f_read = reinterpret_cast<decltype(f_read)>(PyLong_AsVoidPtr(a[10]));
    f_residual = reinterpret_cast<decltype(f_residual)>(PyLong_AsVoidPtr(a[11]));
    f_lora = reinterpret_cast<decltype(f_lora)>(PyLong_AsVoidPtr(a[12]));
    Py_RETURN_NONE;
}

// No C++ exception leaves the module: torch's become its Python errors.
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)> PyObject *guarded(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(a, n);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define Q8_METHOD(f) {#f, (PyCFunction)(void (*)(void))guarded<f>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {Q8_METHOD(init),       Q8_METHOD(fill_cache), Q8_METHOD(kv_append), Q8_METHOD(attn_decode),
                         Q8_METHOD(attn_prompt), Q8_METHOD(kv_reserve), Q8_METHOD(kv_fork),   Q8_METHOD(kv_free),
                         Q8_METHOD(kv_compact),  Q8_METHOD(kv_copy),    Q8_METHOD(kv_read),   Q8_METHOD(residual_norm),
                         Q8_METHOD(lora),        {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_q8torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__q8torch(void) { return PyModule_Create(&module); }
