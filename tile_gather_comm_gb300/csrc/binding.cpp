// binding.cpp -- _ops, the argument marshalling of the transformer-block, attention and cache operators: torch tensors
// in, the C ABI's argument structs (include/tgc.h) out.  It checks what the C entry points cannot
// see -- device, type, shape, inner stride -- because they get addresses only, and computes
// nothing.  Native because a decoding step calls these for a few microseconds of GPU work: the
// same checks in Python took 5 to 18 us a call, on the GB300's host cores.
#include <Python.h>

#include <cstdint>
#include <optional>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/tgc.h"

namespace {

int (*g_linear)(const tgc_linear_args *);
int (*g_linear_bwd)(const tgc_linear_bwd_args *);
size_t (*g_linear_bwd_bytes)(const tgc_linear_bwd_args *);
int (*g_norm)(const tgc_block_norm_args *);
int (*g_norm_bwd)(const tgc_block_norm_bwd_args *);
size_t (*g_norm_bwd_bytes)(const tgc_block_norm_bwd_args *);
int (*g_rope)(const tgc_rope_args *);
int (*g_rope_bwd)(const tgc_rope_args *);
int (*g_append)(const tgc_kv_append_args *);
int (*g_attention)(const tgc_paged_attention_args *);
size_t (*g_attention_bytes)(const tgc_paged_attention_args *);
int (*g_kv[5])(const tgc_kv_args *);  // copy, reserve, fork, free, compact
size_t (*g_kv_bytes)(const tgc_kv_args *);

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(const char *name, const char *what) {
    PyErr_Format(PyExc_ValueError, "%s: %s", name, what);
    throw Refused{};
}

// The tensor in `o`, or null for None; it has to live on the current device.
const at::Tensor *tensor(PyObject *o, const char *name, int *dev) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(name, "expected a tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(name, "expected a CUDA tensor");
    if (*dev < 0) *dev = (int)c10::cuda::current_device();
    if (t.get_device() != *dev) refuse(name, "is not on the current device");
    return &t;
}

const at::Tensor *needed(PyObject *o, const char *name, int *dev) {
    const at::Tensor *t = tensor(o, name, dev);
    if (t == nullptr) refuse(name, "must be given");
    return t;
}

// A (rows, cols) operand whose rows are contiguous: its address and row stride.
void *rows_of(const at::Tensor *t, const char *name, at::ScalarType type, int64_t rows, int64_t cols, int64_t *ld) {
    *ld = 0;
    if (t == nullptr) return nullptr;
    if (t->scalar_type() != type || t->dim() != 2 || t->size(0) != rows || t->size(1) != cols)
        refuse(name, "has another type or shape than the call asks for");
    if (cols > 1 && t->stride(1) != 1) refuse(name, "its last dimension must be contiguous");
    if (rows > 1) {
        *ld = t->stride(0);
        if (*ld < 1) refuse(name, "its rows must not overlap");
    }
    return t->data_ptr();
}

// A contiguous operand of exactly this shape (lead < 0: no leading dimension).
void *dense_of(const at::Tensor *t, const char *name, at::ScalarType type, int64_t lead, int64_t a, int64_t b = -1) {
    if (t == nullptr) return nullptr;
    int64_t want[3];
    int n = 0;
    if (lead >= 0) want[n++] = lead;
    want[n++] = a;
    if (b >= 0) want[n++] = b;
    bool same = t->scalar_type() == type && t->dim() == n;
    for (int i = 0; same && i < n; ++i) same = t->size(i) == want[i];
    if (!same) refuse(name, "has another type or shape than the call asks for");
    if (!t->is_contiguous()) refuse(name, "must be contiguous");
    return t->data_ptr();
}

tgc_dtype dtype_of(at::ScalarType t) {
    switch (t) {
        case at::kByte: return TGC_U8;
        case at::kChar: return TGC_I8;
        case at::kHalf: return TGC_F16;
        case at::kBFloat16: return TGC_BF16;
        case at::kInt: return TGC_I32;
        case at::kFloat: return TGC_F32;
        case at::kLong: return TGC_I64;
        case at::kDouble: return TGC_F64;
        default: return (tgc_dtype)-1;
    }
}

// The stream given as an address, or torch's current one for None.
cudaStream_t stream_of(PyObject *o, int dev) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    if (PyErr_Occurred()) throw Refused{};
    return reinterpret_cast<cudaStream_t>((uintptr_t)v);
}

// The caller's workspace, or one from torch's allocator that belongs to the call's stream.
struct Workspace {
    at::Tensor own;
    void *ptr = nullptr;
    size_t bytes = 0;
    Workspace(PyObject *given, size_t need, const at::Tensor &like, PyObject *stream_arg, cudaStream_t stream, int *dev) {
        if (const at::Tensor *t = tensor(given, "workspace", dev)) {
            if (!t->is_contiguous()) refuse("workspace", "must be contiguous");
            ptr = t->data_ptr();
            bytes = (size_t)t->nbytes();
            return;
        }
        if (need == 0) return;
        std::optional<c10::cuda::CUDAStreamGuard> guard;
        if (stream_arg != Py_None) guard.emplace(c10::cuda::getStreamFromExternal(stream, (c10::DeviceIndex)*dev));
        own = at::empty({(int64_t)need}, like.options().dtype(at::kByte));
        ptr = own.data_ptr();
        bytes = need;
    }
};

struct Weight {
    void *p;
    int64_t N, ld, stride;
};

Weight weight_of(const at::Tensor &w, at::ScalarType type, int64_t K, int groups) {
    const int dims = groups > 0 ? 3 : 2;
    if (w.scalar_type() != type || w.dim() != dims || w.size(dims - 1) != K || (groups > 0 && w.size(0) != groups))
        refuse("w", "has another type or shape than the call asks for");
    if (K > 1 && w.stride(dims - 1) != 1) refuse("w", "its last dimension must be contiguous");
    Weight r{w.data_ptr(), w.size(dims - 2), 0, 0};
    if (r.N > 1) r.ld = w.stride(dims - 2);
    if (groups > 1) r.stride = w.stride(0);
    if ((r.N > 1 && r.ld < 1) || (groups > 1 && r.stride < 1)) refuse("w", "its rows must not overlap");
    return r;
}

const int32_t *offsets_of(const at::Tensor *t, int *groups) {
    *groups = 0;
    if (t == nullptr) return nullptr;
    if (t->scalar_type() != at::kInt || t->dim() != 1 || t->numel() < 2 || !t->is_contiguous())
        refuse("offsets", "expected contiguous int32 of ngroups + 1 row numbers");
    if (t->numel() - 1 > TGC_MAX_GROUPS) refuse("offsets", "too many groups");
    *groups = (int)(t->numel() - 1);
    return static_cast<const int32_t *>(t->data_ptr());
}

int int_of(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return (int)v;
}

float float_of(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return (float)v;
}

// Runs f; what it refuses or torch throws becomes a Python exception.
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F &&f) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return nullptr;
    }
    try {
        return PyLong_FromLongLong((long long)f());
    } catch (const Refused &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// x, w, y, bias, act, residual, z, offsets, stream
PyObject *linear(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        int dev = -1;
        const at::Tensor &x = *needed(o[0], "x", &dev), &w = *needed(o[1], "w", &dev);
        const at::Tensor *y = needed(o[2], "y", &dev), *bias = tensor(o[3], "bias", &dev);
        const at::Tensor *res = tensor(o[5], "residual", &dev), *z = tensor(o[6], "z", &dev);
        const auto type = x.scalar_type();
        if (x.dim() != 2) refuse("x", "expected (M, K)");
        tgc_linear_args a{};
        a.offsets = offsets_of(tensor(o[7], "offsets", &dev), &a.ngroups);
        a.M = x.size(0);
        a.K = x.size(1);
        const Weight k = weight_of(w, type, a.K, a.ngroups);
        a.w = k.p; a.N = k.N; a.ldw = k.ld; a.w_stride = k.stride;
        a.x = rows_of(&x, "x", type, a.M, a.K, &a.ldx);
        a.y = rows_of(y, "y", type, a.M, a.N, &a.ldy);
        a.residual = rows_of(res, "residual", type, a.M, a.N, &a.ldres);
        a.z = rows_of(z, "z", type, a.M, a.N, &a.ldz);
        a.bias = dense_of(bias, "bias", type, a.ngroups > 0 ? a.ngroups : -1, a.N);
        a.dtype = dtype_of(type);
        a.act = (tgc_act)int_of(o[4]);
        a.stream = stream_of(o[8], dev);
        return g_linear(&a);
    });
}

// dy, x, w, z, act, dx, dw, dbias, offsets, workspace, stream.  QUERY: the workspace's bytes, no call.
template <bool QUERY>
PyObject *linear_bwd(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> int64_t {
        int dev = -1;
        const at::Tensor *dy = needed(o[0], "dy", &dev);
        const at::Tensor &x = *needed(o[1], "x", &dev), &w = *needed(o[2], "w", &dev);
        const at::Tensor *z = tensor(o[3], "z", &dev), *dx = tensor(o[5], "dx", &dev);
        const at::Tensor *dw = tensor(o[6], "dw", &dev), *db = tensor(o[7], "dbias", &dev);
        const auto type = x.scalar_type();
        if (x.dim() != 2) refuse("x", "expected (M, K)");
        tgc_linear_bwd_args a{};
        a.offsets = offsets_of(tensor(o[8], "offsets", &dev), &a.ngroups);
        a.M = x.size(0);
        a.K = x.size(1);
        const Weight k = weight_of(w, type, a.K, a.ngroups);
        a.w = k.p; a.N = k.N; a.ldw = k.ld; a.w_stride = k.stride;
        const int64_t lead = a.ngroups > 0 ? a.ngroups : -1;
        a.dy = rows_of(dy, "dy", type, a.M, a.N, &a.lddy);
        a.x = rows_of(&x, "x", type, a.M, a.K, &a.ldx);
        a.z = rows_of(z, "z", type, a.M, a.N, &a.ldz);
        a.dx = rows_of(dx, "dx", type, a.M, a.K, &a.lddx);
        a.dw = dense_of(dw, "dw", type, lead, a.N, a.K);
        a.dbias = dense_of(db, "dbias", type, lead, a.N);
        a.dtype = dtype_of(type);
        a.act = (tgc_act)int_of(o[4]);
        a.stream = stream_of(o[10], dev);
        if (QUERY) return (int64_t)g_linear_bwd_bytes(&a);
        const Workspace ws(o[9], g_linear_bwd_bytes(&a), x, o[10], a.stream, &dev);
        a.workspace = ws.ptr;
        a.workspace_bytes = ws.bytes;
        return g_linear_bwd(&a);
    });
}

// y, r, h, x, gate, post, post_weight, post_bias, pre, pre_weight, pre_bias, res_scale, branch_scale, eps, stream
PyObject *block_norm(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        int dev = -1;
        const at::Tensor &y = *needed(o[0], "y", &dev);
        const auto type = y.scalar_type();
        if (y.dim() != 2) refuse("y", "expected (M, D)");
        tgc_block_norm_args a{};
        const int64_t M = a.M = y.size(0), D = a.D = y.size(1);
        a.y = rows_of(&y, "y", type, M, D, &a.ldy);
        a.r = rows_of(tensor(o[1], "r", &dev), "r", type, M, D, &a.ldr);
        a.h = rows_of(tensor(o[2], "h", &dev), "h", type, M, D, &a.ldh);
        a.x = rows_of(tensor(o[3], "x", &dev), "x", type, M, D, &a.ldx);
        if (const at::Tensor *g = tensor(o[4], "gate", &dev)) {
            a.gates = g->dim() == 2 ? g->size(0) : -1;
            a.gate = dense_of(g, "gate", type, a.gates, D);
        }
        a.post = (tgc_norm)int_of(o[5]);
        a.post_weight = dense_of(tensor(o[6], "post_weight", &dev), "post_weight", type, -1, D);
        a.post_bias = dense_of(tensor(o[7], "post_bias", &dev), "post_bias", type, -1, D);
        a.pre = (tgc_norm)int_of(o[8]);
        a.pre_weight = dense_of(tensor(o[9], "pre_weight", &dev), "pre_weight", type, -1, D);
        a.pre_bias = dense_of(tensor(o[10], "pre_bias", &dev), "pre_bias", type, -1, D);
        a.res_scale = float_of(o[11]);
        a.branch_scale = float_of(o[12]);
        a.eps = float_of(o[13]);
        a.dtype = dtype_of(type);
        a.stream = stream_of(o[14], dev);
        return g_norm(&a);
    });
}

// y, r, dr, dh, gate, post, post_weight, post_bias, pre, pre_weight, res_scale, branch_scale, eps,
// dx, dy, dgate, dpost_weight, dpost_bias, dpre_weight, dpre_bias, workspace, stream.  QUERY: as above.
template <bool QUERY>
PyObject *block_norm_bwd(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 22, [&]() -> int64_t {
        int dev = -1;
        static const char *const names[4] = {"y", "r", "dr", "dh"};
        const at::Tensor *in[4], *like = nullptr;
        for (int i = 0; i < 4; ++i) in[i] = tensor(o[i], names[i], &dev);
        for (int i = 3; i >= 0; --i)
            if (like == nullptr) like = in[i];
        if (like == nullptr || like->dim() != 2) refuse("dh", "expected (M, D) operands");
        const auto type = like->scalar_type();
        tgc_block_norm_bwd_args a{};
        const int64_t M = a.M = like->size(0), D = a.D = like->size(1);
        a.y = rows_of(in[0], "y", type, M, D, &a.ldy);
        a.r = rows_of(in[1], "r", type, M, D, &a.ldr);
        a.dr = rows_of(in[2], "dr", type, M, D, &a.lddr);
        a.dh = rows_of(in[3], "dh", type, M, D, &a.lddh);
        if (const at::Tensor *g = tensor(o[4], "gate", &dev)) {
            a.gates = g->dim() == 2 ? g->size(0) : -1;
            a.gate = dense_of(g, "gate", type, a.gates, D);
        }
        a.post = (tgc_norm)int_of(o[5]);
        a.post_weight = dense_of(tensor(o[6], "post_weight", &dev), "post_weight", type, -1, D);
        a.post_bias = dense_of(tensor(o[7], "post_bias", &dev), "post_bias", type, -1, D);
        a.pre = (tgc_norm)int_of(o[8]);
        a.pre_weight = dense_of(tensor(o[9], "pre_weight", &dev), "pre_weight", type, -1, D);
        a.res_scale = float_of(o[10]);
        a.branch_scale = float_of(o[11]);
        a.eps = float_of(o[12]);
        a.dx = rows_of(tensor(o[13], "dx", &dev), "dx", type, M, D, &a.lddx);
        a.dy = rows_of(tensor(o[14], "dy", &dev), "dy", type, M, D, &a.lddy);
        a.dgate = dense_of(tensor(o[15], "dgate", &dev), "dgate", type, a.gates, D);
        a.dpost_weight = dense_of(tensor(o[16], "dpost_weight", &dev), "dpost_weight", type, -1, D);
        a.dpost_bias = dense_of(tensor(o[17], "dpost_bias", &dev), "dpost_bias", type, -1, D);
        a.dpre_weight = dense_of(tensor(o[18], "dpre_weight", &dev), "dpre_weight", type, -1, D);
        a.dpre_bias = dense_of(tensor(o[19], "dpre_bias", &dev), "dpre_bias", type, -1, D);
        a.dtype = dtype_of(type);
        a.stream = stream_of(o[21], dev);
        if (QUERY) return (int64_t)g_norm_bwd_bytes(&a);
        const Workspace ws(o[20], g_norm_bwd_bytes(&a), *like, o[21], a.stream, &dev);
        a.workspace = ws.ptr;
        a.workspace_bytes = ws.bytes;
        return g_norm_bwd(&a);
    });
}

// ---------------------------------------------------------------- attention and cache operators

int64_t int64_of(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return (int64_t)v;
}

// A (T, heads, D) operand whose heads' elements are contiguous: its address and strides.
void *heads_of(const at::Tensor *t, const char *name, at::ScalarType type, int64_t T, int64_t H, int64_t D, int64_t *st,
               int64_t *sh) {
    *st = *sh = 0;
    if (t == nullptr) return nullptr;
    if (t->scalar_type() != type || t->dim() != 3 || t->size(0) != T || t->size(1) != H || t->size(2) != D)
        refuse(name, "has another type or shape than the call asks for");
    if (D > 1 && t->stride(2) != 1) refuse(name, "its last dimension must be contiguous");
    if (H > 1) *sh = t->stride(1);
    if (T > 1) *st = t->stride(0);
    if ((H > 1 && *sh < 1) || (T > 1 && *st < 1)) refuse(name, "its tokens and heads must not overlap");
    return t->data_ptr();
}

// A list of whole numbers; n < 0: of any length.
int32_t *ints_of(const at::Tensor *t, const char *name, int64_t n) {
    if (t == nullptr) return nullptr;
    if (t->scalar_type() != at::kInt || t->dim() != 1 || (n >= 0 && t->size(0) != n) || !t->is_contiguous())
        refuse(name, "expected contiguous int32 of as many numbers as the call asks for");
    return static_cast<int32_t *>(t->data_ptr());
}

int32_t *table_of(const at::Tensor *t, int64_t *num_seqs, int64_t *max_pages, int64_t *ld) {
    if (t->dim() != 2) refuse("table", "expected int32 (sequences, pages)");
    *num_seqs = t->size(0);
    *max_pages = t->size(1);
    return static_cast<int32_t *>(rows_of(t, "table", at::kInt, *num_seqs, *max_pages, ld));
}

// The pools of keys and values, (pages, page_size, heads, D) with the same strides in any order of pages,
// tokens and heads.
struct Pages {
    void *k, *v;
    int64_t num, size, heads, D, page_s, token_s, head_s;
};

Pages pages_of(const at::Tensor *k, const at::Tensor *v, at::ScalarType type) {
    if (k->dim() != 4 || k->scalar_type() != type) refuse("k_pages", "expected (pages, page size, heads, D) of the call's type");
    bool same = v->scalar_type() == type && v->sizes() == k->sizes();
    for (int i = 0; same && i < 4; ++i) same = k->size(i) < 2 || v->stride(i) == k->stride(i);  // of one entry it means nothing
    if (!same) refuse("v_pages", "has another type, shape or strides than k_pages");
    if (k->size(3) > 1 && k->stride(3) != 1) refuse("k_pages", "its last dimension must be contiguous");
    Pages p{k->data_ptr(), v->data_ptr(), k->size(0), k->size(1), k->size(2), k->size(3), 0, 0, 0};
    int64_t *const s[3] = {&p.page_s, &p.token_s, &p.head_s};
    for (int i = 0; i < 3; ++i)
        if (k->size(i) > 1) {
            *s[i] = k->stride(i);
            if (*s[i] < 1) refuse("k_pages", "its pages, tokens and heads must not overlap");
        }
    // where a dimension has one entry its stride means nothing: the C call's default would multiply what is given
    if (p.head_s == 0) p.head_s = p.D;
    if (p.token_s == 0) p.token_s = p.D;
    if (p.page_s == 0) p.page_s = p.D;
    return p;
}

const double *freqs_of(const at::Tensor *t, int64_t *R) {
    *R = 0;
    if (t == nullptr) return nullptr;
    if (t->scalar_type() != at::kDouble || t->dim() != 1 || t->numel() < 1 || !t->is_contiguous())
        refuse("freqs", "expected contiguous float64 of half as many numbers as elements turn");
    *R = 2 * t->numel();
    return static_cast<const double *>(t->data_ptr());
}

// q, q_out, pos, freqs, k, k_out, layout, scale, stream
template <bool BACK>
PyObject *rope(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        int dev = -1;
        const at::Tensor &q = *needed(o[0], BACK ? "dq_out" : "q", &dev);
        const at::Tensor *q_out = needed(o[1], BACK ? "dq" : "q_out", &dev), *pos = needed(o[2], "pos", &dev);
        const at::Tensor *freqs = needed(o[3], "freqs", &dev);
        const char *const kn = BACK ? "dk_out" : "k", *const kon = BACK ? "dk" : "k_out";
        const at::Tensor *k = tensor(o[4], kn, &dev), *k_out = tensor(o[5], kon, &dev);
        const auto type = q.scalar_type();
        if (q.dim() != 3) refuse(BACK ? "dq_out" : "q", "expected (tokens, heads, D)");
        if ((k == nullptr) != (k_out == nullptr)) refuse(kon, "must be given exactly with its input");
        if (k != nullptr && k->dim() != 3) refuse(kn, "expected (tokens, heads, D)");
        tgc_rope_args a{};
        a.T = q.size(0);
        a.heads_q = q.size(1);
        a.D = q.size(2);
        a.heads_k = k != nullptr ? k->size(1) : 0;
        a.q = heads_of(&q, BACK ? "dq_out" : "q", type, a.T, a.heads_q, a.D, &a.q_t, &a.q_h);
        a.q_out = heads_of(q_out, BACK ? "dq" : "q_out", type, a.T, a.heads_q, a.D, &a.qo_t, &a.qo_h);
        a.k = heads_of(k, kn, type, a.T, a.heads_k, a.D, &a.k_t, &a.k_h);
        a.k_out = heads_of(k_out, kon, type, a.T, a.heads_k, a.D, &a.ko_t, &a.ko_h);
        a.pos = ints_of(pos, "pos", a.T);
        a.freqs = freqs_of(freqs, &a.R);
        a.layout = (tgc_rope_layout)int_of(o[6]);
        a.scale = float_of(o[7]);
        a.dtype = dtype_of(type);
        a.stream = stream_of(o[8], dev);
        return (BACK ? g_rope_bwd : g_rope)(&a);
    });
}

// k, v, k_pages, v_pages, table, pos, seqs, q, q_out, freqs, layout, scale, stream
PyObject *kv_append(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        int dev = -1;
        const at::Tensor &k = *needed(o[0], "k", &dev), *v = needed(o[1], "v", &dev);
        const at::Tensor *kp = needed(o[2], "k_pages", &dev), *vp = needed(o[3], "v_pages", &dev);
        const at::Tensor *table = needed(o[4], "table", &dev), *pos = needed(o[5], "pos", &dev);
        const at::Tensor *seqs = tensor(o[6], "seqs", &dev), *q = tensor(o[7], "q", &dev), *q_out = tensor(o[8], "q_out", &dev);
        const auto type = k.scalar_type();
        if (k.dim() != 3) refuse("k", "expected (tokens, heads, D)");
        if ((q == nullptr) != (q_out == nullptr)) refuse("q_out", "must be given exactly with its input");
        if (q != nullptr && q->dim() != 3) refuse("q", "expected (tokens, heads, D)");
        tgc_kv_append_args a{};
        a.T = k.size(0);
        a.heads_k = k.size(1);
        a.D = k.size(2);
        a.heads_q = q != nullptr ? q->size(1) : 0;
        a.k = heads_of(&k, "k", type, a.T, a.heads_k, a.D, &a.k_t, &a.k_h);
        a.v = heads_of(v, "v", type, a.T, a.heads_k, a.D, &a.v_t, &a.v_h);
        a.q = heads_of(q, "q", type, a.T, a.heads_q, a.D, &a.q_t, &a.q_h);
        a.q_out = heads_of(q_out, "q_out", type, a.T, a.heads_q, a.D, &a.qo_t, &a.qo_h);
        const Pages p = pages_of(kp, vp, type);
        if (p.heads != a.heads_k || p.D != a.D) refuse("k_pages", "has other heads than k");
        a.k_pages = p.k; a.v_pages = p.v;
        a.num_pages = p.num; a.page_size = p.size;
        a.page_s = p.page_s; a.token_s = p.token_s; a.head_s = p.head_s;
        a.table = table_of(table, &a.num_seqs, &a.max_pages, &a.table_ld);
        a.pos = ints_of(pos, "pos", a.T);
        a.seqs = ints_of(seqs, "seqs", a.T);
        a.freqs = freqs_of(tensor(o[9], "freqs", &dev), &a.R);
        a.layout = (tgc_rope_layout)int_of(o[10]);
        a.scale = float_of(o[11]);
        a.dtype = dtype_of(type);
        a.stream = stream_of(o[12], dev);
        return g_append(&a);
    });
}

// q, out, k_pages, v_pages, table, lens, lse, scale, window, softcap, workspace, stream.  QUERY: as above.
template <bool QUERY>
PyObject *attention(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> int64_t {
        int dev = -1;
        const at::Tensor &q = *needed(o[0], "q", &dev), *out = needed(o[1], "out", &dev);
        const at::Tensor *kp = needed(o[2], "k_pages", &dev), *vp = needed(o[3], "v_pages", &dev);
        const at::Tensor *table = needed(o[4], "table", &dev), *lens = needed(o[5], "lens", &dev);
        const at::Tensor *lse = tensor(o[6], "lse", &dev);
        const auto type = q.scalar_type();
        if (q.dim() != 3) refuse("q", "expected (sequences, heads, D)");
        tgc_paged_attention_args a{};
        const int64_t S = q.size(0);
        a.heads_q = q.size(1);
        a.D = q.size(2);
        a.q = heads_of(&q, "q", type, S, a.heads_q, a.D, &a.q_s, &a.q_h);
        a.out = heads_of(out, "out", type, S, a.heads_q, a.D, &a.o_s, &a.o_h);
        const Pages p = pages_of(kp, vp, type);
        if (p.D != a.D) refuse("k_pages", "has another head size than q");
        a.k_pages = p.k; a.v_pages = p.v;
        a.heads_k = p.heads;
        a.num_pages = p.num; a.page_size = p.size;
        a.page_s = p.page_s; a.token_s = p.token_s; a.head_s = p.head_s;
        a.table = table_of(table, &a.num_seqs, &a.max_pages, &a.table_ld);
        if (a.num_seqs != S) refuse("table", "has another number of sequences than q");
        a.lens = ints_of(lens, "lens", S);
        a.lse = static_cast<float *>(dense_of(lse, "lse", at::kFloat, S, a.heads_q));
        a.scale = float_of(o[7]);
        a.window = int64_of(o[8]);
        a.softcap = float_of(o[9]);
        a.dtype = dtype_of(type);
        a.stream = stream_of(o[11], dev);
        if (QUERY) return (int64_t)g_attention_bytes(&a);
        const Workspace ws(o[10], g_attention_bytes(&a), q, o[11], a.stream, &dev);
        a.workspace = ws.ptr;
        a.workspace_bytes = ws.bytes;
        return g_attention(&a);
    });
}

// The pools of a cache: a sequence of contiguous tensors of the same number of pages and bytes a page.
struct Pools {
    void *at[TGC_KV_MAX_POOLS];
    int n = 0;
    int64_t pages = -1, page_bytes = -1;
    Pools(PyObject *o, const char *name, int *dev) {
        PyObject *seq = PySequence_Fast(o, "expected a list of tensors");
        if (seq == nullptr) throw Refused{};
        const struct Drop {
            PyObject *o;
            ~Drop() { Py_DECREF(o); }
        } drop{seq};
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(seq);
        if (count < 1 || count > TGC_KV_MAX_POOLS) refuse(name, "expected 1 to 256 tensors");
        for (Py_ssize_t i = 0; i < count; ++i) {
            const at::Tensor &t = *needed(PySequence_Fast_GET_ITEM(seq, i), name, dev);
            if (t.dim() < 1 || t.size(0) < 1 || t.numel() == 0 || !t.is_contiguous())
                refuse(name, "expected contiguous tensors of pages");
            const int64_t p = t.size(0), bytes = (int64_t)t.nbytes() / p;
            if (i > 0 && (p != pages || bytes != page_bytes)) refuse(name, "its pools must have pages of one number and size");
            pages = p;
            page_bytes = bytes;
            at[n++] = t.data_ptr();
        }
    }
};

// refs, table, lens of a cache; lens may be left out (null PyObject).
const at::Tensor &cache_of(PyObject *refs, PyObject *table, PyObject *lens, tgc_kv_args *a, int *dev) {
    const at::Tensor &r = *needed(refs, "refs", dev);
    a->refs = ints_of(&r, "refs", -1);
    a->num_pages = r.size(0);
    a->table = table_of(needed(table, "table", dev), &a->num_seqs, &a->max_pages, &a->table_ld);
    if (lens != nullptr) a->lens = ints_of(needed(lens, "lens", dev), "lens", a->num_seqs);
    return r;
}

int64_t page_size_of(PyObject *o) {
    const int64_t v = int64_of(o);
    if (v < 1) refuse("page_size", "must be positive");
    return v;
}

// pools, from, dst, src, stream
PyObject *kv_copy(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 5, [&] {
        int dev = -1;
        Pools to(o[0], "pools", &dev), from(o[1], "from_pools", &dev);
        if (to.n != from.n || to.page_bytes != from.page_bytes) refuse("from_pools", "has other pools than pools");
        tgc_kv_args a{};
        const at::Tensor *dst = needed(o[2], "dst", &dev);
        a.dst = ints_of(dst, "dst", -1);
        a.n = dst->size(0);
        a.src = ints_of(needed(o[3], "src", &dev), "src", a.n);
        a.pools = to.at;
        a.from = const_cast<const void *const *>(from.at);
        a.npools = to.n;
        a.page_bytes = to.page_bytes;
        a.num_pages = to.pages;
        a.from_pages = from.pages;
        a.stream = stream_of(o[4], dev);
        return g_kv[0](&a);
    });
}

// refs, table, lens, dst, add, page_size, ok, workspace, stream.  QUERY: as above.
template <bool QUERY>
PyObject *kv_reserve(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> int64_t {
        int dev = -1;
        tgc_kv_args a{};
        const at::Tensor &refs = cache_of(o[0], o[1], o[2], &a, &dev);
        const at::Tensor *dst = needed(o[3], "seqs", &dev);
        a.dst = ints_of(dst, "seqs", -1);
        a.n = dst->size(0);
        a.add = ints_of(needed(o[4], "add", &dev), "add", a.n);
        a.page_size = page_size_of(o[5]);
        a.ok = ints_of(tensor(o[6], "ok", &dev), "ok", a.n);
        a.stream = stream_of(o[8], dev);
        if (QUERY) return (int64_t)g_kv_bytes(&a);
        const Workspace ws(o[7], a.n > 0 ? g_kv_bytes(&a) : 0, refs, o[8], a.stream, &dev);
        a.workspace = ws.ptr;
        a.workspace_bytes = ws.bytes;
        return g_kv[1](&a);
    });
}

// pools, refs, table, lens, src, dst, page_size, ok, workspace, stream.  QUERY: as above.
template <bool QUERY>
PyObject *kv_fork(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> int64_t {
        int dev = -1;
        tgc_kv_args a{};
        Pools pools(o[0], "pools", &dev);
        const at::Tensor &refs = cache_of(o[1], o[2], o[3], &a, &dev);
        if (pools.pages != a.num_pages) refuse("refs", "has another number of pages than the pools");
        const at::Tensor *dst = needed(o[5], "dst", &dev);
        a.dst = ints_of(dst, "dst", -1);
        a.n = dst->size(0);
        a.src = ints_of(needed(o[4], "src", &dev), "src", a.n);
        a.page_size = page_size_of(o[6]);
        if (pools.page_bytes % a.page_size != 0) refuse("page_size", "does not divide the pools' pages");
        a.ok = ints_of(tensor(o[7], "ok", &dev), "ok", a.n);
        a.pools = pools.at;
        a.npools = pools.n;
        a.page_bytes = pools.page_bytes;
        a.stream = stream_of(o[9], dev);
        if (QUERY) return (int64_t)g_kv_bytes(&a);
        const Workspace ws(o[8], a.n > 0 ? g_kv_bytes(&a) : 0, refs, o[9], a.stream, &dev);
        a.workspace = ws.ptr;
        a.workspace_bytes = ws.bytes;
        return g_kv[2](&a);
    });
}

// refs, table, lens, seqs, stream
PyObject *kv_free(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 5, [&] {
        int dev = -1;
        tgc_kv_args a{};
        cache_of(o[0], o[1], o[2], &a, &dev);
        const at::Tensor *dst = needed(o[3], "seqs", &dev);
        a.dst = ints_of(dst, "seqs", -1);
        a.n = dst->size(0);
        a.page_size = 1;  // no matter here
        a.stream = stream_of(o[4], dev);
        return g_kv[3](&a);
    });
}

// pools, refs, table, used, workspace, stream.  QUERY: as above.
template <bool QUERY>
PyObject *kv_compact(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> int64_t {
        int dev = -1;
        tgc_kv_args a{};
        Pools pools(o[0], "pools", &dev);
        const at::Tensor &refs = cache_of(o[1], o[2], nullptr, &a, &dev);
        if (pools.pages != a.num_pages) refuse("refs", "has another number of pages than the pools");
        a.used = ints_of(tensor(o[3], "used", &dev), "used", 1);
        a.page_size = 1;  // no matter here
        a.pools = pools.at;
        a.npools = pools.n;
        a.page_bytes = pools.page_bytes;
        a.stream = stream_of(o[5], dev);
        if (QUERY) return (int64_t)g_kv_bytes(&a);
        const Workspace ws(o[4], g_kv_bytes(&a), refs, o[5], a.stream, &dev);
        a.workspace = ws.ptr;
        a.workspace_bytes = ws.bytes;
        return g_kv[4](&a);
    });
}

// The addresses of libtgc.so's entry points, in the order below.
PyObject *bind(PyObject *, PyObject *const *o, Py_ssize_t n) {
    constexpr int kEntries = 17;
    if (n != kEntries) {
        PyErr_SetString(PyExc_TypeError, "expected 17 addresses");
        return nullptr;
    }
    void *p[kEntries];
    for (int i = 0; i < kEntries; ++i) p[i] = PyLong_AsVoidPtr(o[i]);
    if (PyErr_Occurred()) return nullptr;
    g_linear = reinterpret_cast<decltype(g_linear)>(p[0]);
    g_linear_bwd = reinterpret_cast<decltype(g_linear_bwd)>(p[1]);
    g_linear_bwd_bytes = reinterpret_cast<decltype(g_linear_bwd_bytes)>(p[2]);
    g_norm = reinterpret_cast<decltype(g_norm)>(p[3]);
    g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(p[4]);
    g_norm_bwd_bytes = reinterpret_cast<decltype(g_norm_bwd_bytes)>(p[5]);
    g_rope = reinterpret_cast<decltype(g_rope)>(p[6]);
    g_rope_bwd = reinterpret_cast<decltype(g_rope_bwd)>(p[7]);
    g_append = reinterpret_cast<decltype(g_append)>(p[8]);
    g_attention = reinterpret_cast<decltype(g_attention)>(p[9]);
    g_attention_bytes = reinterpret_cast<decltype(g_attention_bytes)>(p[10]);
    for (int i = 0; i < 5; ++i) g_kv[i] = reinterpret_cast<int (*)(const tgc_kv_args *)>(p[11 + i]);
    g_kv_bytes = reinterpret_cast<decltype(g_kv_bytes)>(p[16]);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f));
}

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"linear", fast(linear), METH_FASTCALL, nullptr},
                         {"linear_bwd", fast(linear_bwd<false>), METH_FASTCALL, nullptr},
                         {"linear_bwd_bytes", fast(linear_bwd<true>), METH_FASTCALL, nullptr},
                         {"block_norm", fast(block_norm), METH_FASTCALL, nullptr},
                         {"block_norm_bwd", fast(block_norm_bwd<false>), METH_FASTCALL, nullptr},
                         {"block_norm_bwd_bytes", fast(block_norm_bwd<true>), METH_FASTCALL, nullptr},
                         {"rope", fast(rope<false>), METH_FASTCALL, nullptr},
                         {"rope_bwd", fast(rope<true>), METH_FASTCALL, nullptr},
                         {"kv_append", fast(kv_append), METH_FASTCALL, nullptr},
                         {"paged_attention", fast(attention<false>), METH_FASTCALL, nullptr},
                         {"paged_attention_bytes", fast(attention<true>), METH_FASTCALL, nullptr},
                         {"kv_copy", fast(kv_copy), METH_FASTCALL, nullptr},
                         {"kv_reserve", fast(kv_reserve<false>), METH_FASTCALL, nullptr},
                         {"kv_reserve_bytes", fast(kv_reserve<true>), METH_FASTCALL, nullptr},
                         {"kv_fork", fast(kv_fork<false>), METH_FASTCALL, nullptr},
                         {"kv_fork_bytes", fast(kv_fork<true>), METH_FASTCALL, nullptr},
                         {"kv_free", fast(kv_free), METH_FASTCALL, nullptr},
                         {"kv_compact", fast(kv_compact<false>), METH_FASTCALL, nullptr},
                         {"kv_compact_bytes", fast(kv_compact<true>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", "argument marshalling of the transformer-block, attention and cache operators", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops(void) { return PyModule_Create(&module); }
