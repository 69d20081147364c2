// binding.cpp -- _ops, the argument marshalling of the transformer-block operators: torch tensors
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

// The addresses of libtgc.so's entry points, in the order below.
PyObject *bind(PyObject *, PyObject *const *o, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "expected 6 addresses");
        return nullptr;
    }
    void *p[6];
    for (int i = 0; i < 6; ++i) p[i] = PyLong_AsVoidPtr(o[i]);
    if (PyErr_Occurred()) return nullptr;
    g_linear = reinterpret_cast<decltype(g_linear)>(p[0]);
    g_linear_bwd = reinterpret_cast<decltype(g_linear_bwd)>(p[1]);
    g_linear_bwd_bytes = reinterpret_cast<decltype(g_linear_bwd_bytes)>(p[2]);
    g_norm = reinterpret_cast<decltype(g_norm)>(p[3]);
    g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(p[4]);
    g_norm_bwd_bytes = reinterpret_cast<decltype(g_norm_bwd_bytes)>(p[5]);
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
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", "argument marshalling of the transformer-block operators", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops(void) { return PyModule_Create(&module); }
