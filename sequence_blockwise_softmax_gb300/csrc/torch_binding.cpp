// torch_binding.cpp -- argument checks and marshalling, in C++, for the calls
// that serve single tokens or short sequences, where a Python binding's checks
// cost more than the kernel: about 13 us a call on the Grace host against 1 us
// here.  Nothing is computed and nothing kept: each function checks its
// tensors' types, shapes, layouts and device, takes their pointers and the
// current CUDA stream, and calls the C entry point (whose address bind() was
// given), returning its status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>

#include "ra.h"

namespace {

struct Refused : std::exception {};   // the Python error is set

template <class... A>
[[noreturn]] void refuse(PyObject *type, const char *fmt, A... a) {
    PyErr_Format(type, fmt, a...);
    throw Refused();
}

enum Types : unsigned { kBF16 = 1, kF32 = 2, kI32 = 4, kAny = 8 };

const char *type_names(unsigned t) {
    switch (t) {
        case kBF16: return "bf16";
        case kF32: return "fp32";
        case kI32: return "int32";
        default: return "bf16 or fp32";
    }
}

unsigned type_of(const at::Tensor &t) {
    switch (t.scalar_type()) {
        case at::kBFloat16: return kBF16;
        case at::kFloat: return kF32;
        case at::kInt: return kI32;
        default: return 0;
    }
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

// The device of a call: its first tensor's, which has to be the current one.
int call_device(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
    const int dev = t.get_device();
    if (dev != (int)c10::cuda::current_device())
        refuse(PyExc_ValueError, "%s must be on the current CUDA device", name);
    return dev;
}

void check_type(const at::Tensor &t, const char *name, unsigned types, int dev) {
    if (!(types & kAny) && !(type_of(t) & types)) refuse(PyExc_TypeError, "%s must be %s", name, type_names(types));
    if (!t.is_cuda() || t.get_device() != dev)
        refuse(PyExc_ValueError, "%s must be on the call's CUDA device", name);
}

void check_shape(const at::Tensor &t, const char *name, std::initializer_list<int64_t> shape) {
    bool same = t.dim() == (int64_t)shape.size();
    int i = 0;
    for (int64_t n : shape) same = same && t.size(i++) == n;
    if (!same) refuse(PyExc_ValueError, "%s does not have the call's shape", name);
}

void *contiguous(PyObject *o, const char *name, unsigned types, int dev, std::initializer_list<int64_t> shape) {
    const at::Tensor &t = tensor(o, name);
    check_type(t, name, types, dev);
    check_shape(t, name, shape);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return t.data_ptr();
}

struct Workspace {
    void *ptr;
    size_t bytes;
};
Workspace workspace(PyObject *o, int dev) {
    if (o == Py_None) refuse(PyExc_ValueError, "workspace is needed (see new_workspace)");
    const at::Tensor &t = tensor(o, "workspace");
    check_type(t, "workspace", kAny, dev);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
    return {t.data_ptr(), (size_t)t.nbytes()};
}

struct Boundaries {
    const int32_t *ptr = nullptr;
    int n_seqs = 0;
};
Boundaries boundaries(PyObject *o, int dev) {
    Boundaries b;
    if (o == Py_None) return b;
    const at::Tensor &t = tensor(o, "cu_seqlens");
    check_type(t, "cu_seqlens", kI32, dev);
    if (t.dim() != 1 || !t.is_contiguous()) refuse(PyExc_ValueError, "cu_seqlens must be a contiguous vector");
    if (t.numel() - 1 > 0x7fffffff) refuse(PyExc_ValueError, "too many sequences");
    b.ptr = t.const_data_ptr<int32_t>();
    b.n_seqs = (int)t.numel() - 1;
    return b;
}

int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}
int small_integer(PyObject *o) {
    const int64_t v = integer(o);
    if (v != (int)v) refuse(PyExc_OverflowError, "an argument does not fit in 32 bits");
    return (int)v;
}
float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return (float)v;
}
void *stream_of(PyObject *o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    return reinterpret_cast<void *>((uintptr_t)integer(o));
}

// The C entry points' addresses.
decltype(&ra_window_attn_fwd) window_fwd_fn;
decltype(&ra_window_attn_bwd) window_bwd_fn;
decltype(&ra_paged_attn_fwd) paged_fwd_fn;
decltype(&ra_paged_append) append_fn;
decltype(&ra_paged_tree_attn_fwd) tree_fwd_fn;
decltype(&ra_paged_append_rotary) append_rotary_fn;
decltype(&ra_paged_keep_path) keep_path_fn;

template <class F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F f) {
    if (got != want) return PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    try {
        return PyLong_FromLong((long)f());
    } catch (const Refused &) {
        return nullptr;
    } catch (const std::exception &e) {
        return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
    }
}

// q, k, v, o, lse, B, L, H, H_kv, d, window, sinks, scale, cu_seqlens, workspace, stream
PyObject *window_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 16, [&] {
        const int64_t B = integer(a[5]), L = integer(a[6]), H = integer(a[7]), Hkv = integer(a[8]);
        const int d = small_integer(a[9]);
        const int dev = call_device(tensor(a[0], "q"), "q");
        const void *q = contiguous(a[0], "q", kBF16, dev, {B, L, H, d});
        const void *k = contiguous(a[1], "k", kBF16, dev, {B, L, Hkv, d});
        const void *v = contiguous(a[2], "v", kBF16, dev, {B, L, Hkv, d});
        void *o = contiguous(a[3], "o", kBF16 | kF32, dev, {B, L, H, d});
        void *lse = contiguous(a[4], "lse", kF32, dev, {B, H, L});
        const Boundaries cu = boundaries(a[13], dev);
        const Workspace ws = workspace(a[14], dev);
        const unsigned flags = type_of(tensor(a[3], "o")) == kBF16 ? RA_FLAG_O_BF16 : 0;
        return window_fwd_fn(q, k, v, o, static_cast<float *>(lse), cu.ptr, cu.n_seqs, B, L, H, Hkv, d, integer(a[10]),
                             integer(a[11]), real(a[12]), flags, ws.ptr, ws.bytes, stream_of(a[15]));
    });
}

// q, k, v, o, dout, lse, dq, dk, dv, B, L, H, H_kv, d, window, sinks, scale, cu_seqlens, workspace, stream
PyObject *window_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 20, [&] {
        const int64_t B = integer(a[9]), L = integer(a[10]), H = integer(a[11]), Hkv = integer(a[12]);
        const int d = small_integer(a[13]);
        const int dev = call_device(tensor(a[0], "q"), "q");
        const void *q = contiguous(a[0], "q", kBF16, dev, {B, L, H, d});
        const void *k = contiguous(a[1], "k", kBF16, dev, {B, L, Hkv, d});
        const void *v = contiguous(a[2], "v", kBF16, dev, {B, L, Hkv, d});
        const void *o = contiguous(a[3], "o", kBF16 | kF32, dev, {B, L, H, d});
        const void *dout = contiguous(a[4], "dout", kBF16, dev, {B, L, H, d});
        const void *lse = contiguous(a[5], "lse", kF32, dev, {B, H, L});
        void *dq = contiguous(a[6], "dq", kBF16 | kF32, dev, {B, L, H, d});
        const unsigned g = type_of(tensor(a[6], "dq"));      // all three alike
        void *dk = contiguous(a[7], "dk", g, dev, {B, L, Hkv, d});
        void *dv = contiguous(a[8], "dv", g, dev, {B, L, Hkv, d});
        const Boundaries cu = boundaries(a[17], dev);
        const Workspace ws = workspace(a[18], dev);
        const unsigned flags = (type_of(tensor(a[3], "o")) == kBF16 ? RA_FLAG_O_BF16 : 0) |
                               (g == kBF16 ? RA_FLAG_GRAD_BF16 : 0);
        return window_bwd_fn(q, k, v, o, dout, static_cast<const float *>(lse), dq, dk, dv, cu.ptr, cu.n_seqs, B, L, H,
                             Hkv, d, integer(a[14]), integer(a[15]), real(a[16]), flags, ws.ptr, ws.bytes,
                             stream_of(a[19]));
    });
}

// [n_pages, page, H_kv, d] views of one shape and page stride, each page without gaps.
struct Pool {
    void *k, *v;
    int64_t n_pages, page, Hkv, d, stride;
};
// Whether t[0] (t[0][0] with `from` 2) has no gaps.
bool gapless(const at::Tensor &t, int64_t from = 1) {
    if (t.is_contiguous()) return true;
    int64_t next = 1;
    for (int64_t i = t.dim() - 1; i >= from; --i) {
        if (t.size(i) != 1 && t.stride(i) != next) return false;
        next *= t.size(i);
    }
    return t.size(0) > 0;
}
// ... and of the layers [layers, n_pages, page, H_kv, d] with one layer stride, or of one pool.
struct Layers {
    Pool pool;
    int64_t n, stride;
};
// (`axis`: that of the pages)
Pool pool_of(const at::Tensor &k, const at::Tensor &v, int64_t axis) {
    Pool p{k.data_ptr(), v.data_ptr(), k.size(axis), k.size(axis + 1), k.size(axis + 2), k.size(axis + 3), 0};
    p.stride = p.n_pages > 1 ? k.stride(axis) : p.page * p.Hkv * p.d;
    if (!gapless(k, axis + 1) || !gapless(v, axis + 1) || (p.n_pages > 1 && v.stride(axis) != p.stride))
        refuse(PyExc_ValueError, "k_pages and v_pages: a page must be contiguous, and both pools have one page stride");
    return p;
}
Pool pool(PyObject *ko, PyObject *vo) {
    const at::Tensor &k = tensor(ko, "k_pages"), &v = tensor(vo, "v_pages");
    if (k.dim() != 4 || v.sizes() != k.sizes())
        refuse(PyExc_ValueError, "k_pages and v_pages must have one shape, [n_pages, page, H_kv, d]");
    return pool_of(k, v, 0);
}
Layers layers(PyObject *ko, PyObject *vo) {
    const at::Tensor &k = tensor(ko, "k_pages"), &v = tensor(vo, "v_pages");
    if (k.dim() != 5) return {pool(ko, vo), 1, 0};
    if (v.sizes() != k.sizes() || k.size(0) < 1 || (k.size(0) > 1 && v.stride(0) != k.stride(0)))
        refuse(PyExc_ValueError, "k_pages and v_pages must have one shape and layer stride, and a layer at least");
    return {pool_of(k, v, 1), k.size(0), k.size(0) > 1 ? k.stride(0) : 0};
}

int pool_device(PyObject *first, const char *name, PyObject *ko, PyObject *vo) {
    const int dev = call_device(tensor(first, name), name);
    check_type(tensor(ko, "k_pages"), "k_pages", kBF16, dev);
    check_type(tensor(vo, "v_pages"), "v_pages", kBF16, dev);
    return dev;
}

// The token stride of a bf16 [T, heads, d] view whose tokens are contiguous.
int64_t token_stride(const at::Tensor &t, const char *name, int64_t heads, int64_t d, int dev) {
    check_type(t, name, kBF16, dev);
    if (t.dim() != 3 || t.size(1) != heads || t.size(2) != d)
        refuse(PyExc_ValueError, "%s must be [T, heads, d] with the call's heads and d", name);
    if (!gapless(t) && t.size(0) > 0) refuse(PyExc_ValueError, "%s: a token's heads must be contiguous", name);
    return t.size(0) > 1 ? t.stride(0) : heads * d;
}

struct Sequences {
    const int32_t *table, *lens, *cu;
    int64_t n, max_pages;
};
Sequences sequences(PyObject *table, PyObject *lens, PyObject *cu, const char *cu_name, int dev) {
    const at::Tensor &t = tensor(table, "block_table");
    check_type(t, "block_table", kI32, dev);
    if (t.dim() != 2 || !t.is_contiguous()) refuse(PyExc_ValueError, "block_table must be contiguous, [n_seqs, max_pages]");
    const int64_t n = t.size(0);
    return {t.const_data_ptr<int32_t>(), static_cast<const int32_t *>(contiguous(lens, "seq_lens", kI32, dev, {n})),
            static_cast<const int32_t *>(contiguous(cu, cu_name, kI32, dev, {n + 1})), n, t.size(1)};
}

// q, k_pages, v_pages, block_table, seq_lens, cu_q, o, lse, max_new, max_len, window, sinks, scale, workspace, stream
PyObject *paged_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        const at::Tensor &q = tensor(a[0], "q");
        const Pool p = pool(a[1], a[2]);
        const int dev = pool_device(a[0], "q", a[1], a[2]);
        if (q.dim() != 3) refuse(PyExc_ValueError, "q must be [T, H, d]");
        const int64_t T = q.size(0), H = q.size(1);
        const int64_t q_stride = token_stride(q, "q", H, p.d, dev);
        const Sequences s = sequences(a[3], a[4], a[5], "cu_q", dev);
        void *o = contiguous(a[6], "o", kBF16 | kF32, dev, {T, H, p.d});
        void *lse = a[7] == Py_None ? nullptr : contiguous(a[7], "lse", kF32, dev, {H, T});
        const Workspace ws = workspace(a[13], dev);
        if (p.d != (int)p.d) refuse(PyExc_ValueError, "d does not fit in 32 bits");
        return paged_fwd_fn(q.data_ptr(), p.k, p.v, s.table, s.lens, s.cu, o, static_cast<float *>(lse), T, s.n, H, p.Hkv,
                            (int)p.d, p.n_pages, p.page, p.stride, s.max_pages, q_stride, integer(a[8]), integer(a[9]),
                            integer(a[10]), integer(a[11]), real(a[12]),
                            type_of(tensor(a[6], "o")) == kBF16 ? RA_FLAG_O_BF16 : 0, ws.ptr, ws.bytes,
                            stream_of(a[14]));
    });
}

// k_new, v_new, k_pages, v_pages, block_table, seq_lens, cu_new, workspace, stream
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        const at::Tensor &k = tensor(a[0], "k_new"), &v = tensor(a[1], "v_new");
        const Pool p = pool(a[2], a[3]);
        const int dev = pool_device(a[0], "k_new", a[2], a[3]);
        const int64_t stride = token_stride(k, "k_new", p.Hkv, p.d, dev);
        if (v.sizes() != k.sizes() || token_stride(v, "v_new", p.Hkv, p.d, dev) != stride)
            refuse(PyExc_ValueError, "k_new and v_new must have one shape and token stride");
        const Sequences s = sequences(a[4], a[5], a[6], "cu_new", dev);
        const Workspace ws = workspace(a[7], dev);
        if (p.d != (int)p.d) refuse(PyExc_ValueError, "d does not fit in 32 bits");
        return append_fn(k.data_ptr(), v.data_ptr(), p.k, p.v, s.table, s.lens, s.cu, k.size(0), s.n, p.Hkv, (int)p.d,
                         p.n_pages, p.page, p.stride, s.max_pages, stride, ws.ptr, ws.bytes, stream_of(a[8]));
    });
}

const int32_t *vector(PyObject *o, const char *name, int dev, int64_t n) {
    return static_cast<const int32_t *>(contiguous(o, name, kI32, dev, {n}));
}

// q, k_pages, v_pages, block_table, seq_lens, cu_q, parents, o, lse, max_new, max_len, window, sinks, scale, workspace,
// stream
PyObject *tree_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 16, [&] {
        const at::Tensor &q = tensor(a[0], "q");
        const Pool p = pool(a[1], a[2]);
        const int dev = pool_device(a[0], "q", a[1], a[2]);
        if (q.dim() != 3) refuse(PyExc_ValueError, "q must be [T, H, d]");
        const int64_t T = q.size(0), H = q.size(1);
        const int64_t q_stride = token_stride(q, "q", H, p.d, dev);
        const Sequences s = sequences(a[3], a[4], a[5], "cu_q", dev);
        const int32_t *parents = vector(a[6], "parents", dev, T);
        void *o = contiguous(a[7], "o", kBF16 | kF32, dev, {T, H, p.d});
        void *lse = a[8] == Py_None ? nullptr : contiguous(a[8], "lse", kF32, dev, {H, T});
        const Workspace ws = workspace(a[14], dev);
        if (p.d != (int)p.d) refuse(PyExc_ValueError, "d does not fit in 32 bits");
        return tree_fwd_fn(q.data_ptr(), p.k, p.v, s.table, s.lens, s.cu, parents, o, static_cast<float *>(lse), T, s.n, H,
                           p.Hkv, (int)p.d, p.n_pages, p.page, p.stride, s.max_pages, q_stride, integer(a[9]),
                           integer(a[10]), integer(a[11]), integer(a[12]), real(a[13]),
                           type_of(tensor(a[7], "o")) == kBF16 ? RA_FLAG_O_BF16 : 0, ws.ptr, ws.bytes, stream_of(a[15]));
    });
}

// q, k_new, v_new, q_out, k_pages, v_pages, block_table, seq_lens, cu_new, inv_freq, parents, pairs, workspace, stream
PyObject *append_rotary(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 14, [&] {
        const at::Tensor &k = tensor(a[1], "k_new"), &v = tensor(a[2], "v_new");
        const Pool p = pool(a[4], a[5]);
        const int dev = pool_device(a[1], "k_new", a[4], a[5]);
        const int64_t T = k.dim() > 0 ? k.size(0) : 0, stride = token_stride(k, "k_new", p.Hkv, p.d, dev);
        if (v.sizes() != k.sizes() || token_stride(v, "v_new", p.Hkv, p.d, dev) != stride)
            refuse(PyExc_ValueError, "k_new and v_new must have one shape and token stride");
        int64_t H = 0, q_stride = 0, out_stride = 0;
        void *q = nullptr, *q_out = nullptr;
        if ((a[0] == Py_None) != (a[3] == Py_None)) refuse(PyExc_ValueError, "q and q_out are given both or neither");
        if (a[0] != Py_None) {
            const at::Tensor &x = tensor(a[0], "q"), &y = tensor(a[3], "q_out");
            if (x.dim() != 3 || x.size(0) != T || y.sizes() != x.sizes())
                refuse(PyExc_ValueError, "q and q_out must be [T, H, d] with k_new's T");
            H = x.size(1);
            q_stride = token_stride(x, "q", H, p.d, dev);
            out_stride = token_stride(y, "q_out", H, p.d, dev);
            q = x.data_ptr();
            q_out = y.data_ptr();
        }
        const Sequences s = sequences(a[6], a[7], a[8], "cu_new", dev);
        const at::Tensor &f = tensor(a[9], "inv_freq");
        if (f.dim() != 1) refuse(PyExc_ValueError, "inv_freq must be a vector");
        const void *freq = contiguous(a[9], "inv_freq", kF32, dev, {f.size(0)});
        const int32_t *parents = a[10] == Py_None ? nullptr : vector(a[10], "parents", dev, T);
        const int pairs = PyObject_IsTrue(a[11]);
        if (pairs < 0) throw Refused();
        const Workspace ws = workspace(a[12], dev);
        if (p.d != (int)p.d || f.size(0) > p.d) refuse(PyExc_ValueError, "d or inv_freq is too large");
        return append_rotary_fn(q, k.data_ptr(), v.data_ptr(), q_out, p.k, p.v, s.table, s.lens, s.cu, parents,
                                static_cast<const float *>(freq), T, s.n, H, p.Hkv, (int)p.d, (int)(2 * f.size(0)),
                                p.n_pages, p.page, p.stride, s.max_pages, q_stride, out_stride, stride,
                                pairs ? RA_FLAG_ROTARY_PAIRS : 0, ws.ptr, ws.bytes, stream_of(a[13]));
    });
}

// k_pages, v_pages, block_table, seq_lens, cu_new, parents, last, new_lens, path, workspace, stream
PyObject *keep_path(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const Layers l = layers(a[0], a[1]);
        const Pool &p = l.pool;
        const int dev = pool_device(a[0], "k_pages", a[0], a[1]);
        const Sequences s = sequences(a[2], a[3], a[4], "cu_new", dev);
        const at::Tensor &t = tensor(a[5], "parents");
        if (t.dim() != 1) refuse(PyExc_ValueError, "parents must be a vector");
        const int64_t T = t.size(0);
        const int32_t *parents = vector(a[5], "parents", dev, T);
        const int32_t *last = vector(a[6], "last", dev, s.n);
        const int32_t *lens = vector(a[7], "new_lens", dev, s.n);
        const int32_t *path = a[8] == Py_None ? nullptr : vector(a[8], "path", dev, T);
        const Workspace ws = workspace(a[9], dev);
        if (p.d != (int)p.d) refuse(PyExc_ValueError, "d does not fit in 32 bits");
        return keep_path_fn(p.k, p.v, s.table, s.lens, s.cu, parents, last, const_cast<int32_t *>(lens),
                            const_cast<int32_t *>(path), T, s.n, l.n, p.Hkv, (int)p.d, p.n_pages, p.page, p.stride,
                            l.stride, s.max_pages, ws.ptr, ws.bytes, stream_of(a[10]));
    });
}

// The addresses of ra_window_attn_fwd, ra_window_attn_bwd, ra_paged_attn_fwd, ra_paged_append,
// ra_paged_tree_attn_fwd, ra_paged_append_rotary, ra_paged_keep_path
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 7, [&] {
        window_fwd_fn = reinterpret_cast<decltype(window_fwd_fn)>((uintptr_t)integer(a[0]));
        window_bwd_fn = reinterpret_cast<decltype(window_bwd_fn)>((uintptr_t)integer(a[1]));
        paged_fwd_fn = reinterpret_cast<decltype(paged_fwd_fn)>((uintptr_t)integer(a[2]));
        append_fn = reinterpret_cast<decltype(append_fn)>((uintptr_t)integer(a[3]));
        tree_fwd_fn = reinterpret_cast<decltype(tree_fwd_fn)>((uintptr_t)integer(a[4]));
        append_rotary_fn = reinterpret_cast<decltype(append_rotary_fn)>((uintptr_t)integer(a[5]));
        keep_path_fn = reinterpret_cast<decltype(keep_path_fn)>((uintptr_t)integer(a[6]));
        return 0;
    });
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"window_fwd", fast(window_fwd), METH_FASTCALL, nullptr},
                         {"window_bwd", fast(window_bwd), METH_FASTCALL, nullptr},
                         {"paged_fwd", fast(paged_fwd), METH_FASTCALL, nullptr},
                         {"append", fast(append), METH_FASTCALL, nullptr},
                         {"tree_fwd", fast(tree_fwd), METH_FASTCALL, nullptr},
                         {"append_rotary", fast(append_rotary), METH_FASTCALL, nullptr},
                         {"keep_path", fast(keep_path), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "ra_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ra_torch() { return PyModule_Create(&module); }
