// Python binding of the calls that make up a decode step of a few microseconds: rotary
// positions, per-head norms, trees of drafted tokens.  It does what the ctypes layer does
// (types, shapes, devices and contiguity of the tensors, the device's current stream, then
// the C entry point), in one native call: a dozen tensors checked in Python take longer
// than the launch.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <string>

#include "../../include/qsa.h"

namespace {

using at::ScalarType;
constexpr auto BF = ScalarType::BFloat16;
constexpr auto F32 = ScalarType::Float;
constexpr auto F64 = ScalarType::Double;
constexpr auto I32 = ScalarType::Int;
constexpr auto I64 = ScalarType::Long;
constexpr auto U8 = ScalarType::Byte;

const char *name_of(ScalarType t) {
    switch (t) {
        case BF: return "torch.bfloat16";
        case F32: return "torch.float32";
        case F64: return "torch.float64";
        case I32: return "torch.int32";
        case I64: return "torch.int64";
        default: return "torch.uint8";
    }
}

// What a refusal throws: the Python error is set.
struct Refused {};

std::string list_of(at::IntArrayRef s) {
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
        throw Refused();
    }
    return THPVariable_Unpack(o);
}

void of_type(const at::Tensor &t, ScalarType type, const char *name) {
    if (t.scalar_type() != type) {
        PyErr_Format(PyExc_TypeError, "%s must be %s, got %s", name, name_of(type),
                     c10::toString(t.scalar_type()));
        throw Refused();
    }
}

void of_rank(const at::Tensor &t, int rank, const char *name) {
    if (t.dim() != rank) {
        PyErr_Format(PyExc_ValueError, "%s must have %d dims, got %s", name, rank,
                     list_of(t.sizes()).c_str());
        throw Refused();
    }
}

// On device `dev`, or (dev < 0) on any; the device.
int on_device(const at::Tensor &t, int dev, const char *name) {
    if (!t.is_cuda()) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
        throw Refused();
    }
    if (dev >= 0 && t.get_device() != dev) {
        PyErr_Format(PyExc_ValueError, "%s is on cuda:%d, not on cuda:%d", name,
                     (int)t.get_device(), dev);
        throw Refused();
    }
    return (int)t.get_device();
}

void of_shape(const at::Tensor &t, at::IntArrayRef shape, const char *name) {
    if (t.sizes() != shape) {
        PyErr_Format(PyExc_ValueError, "%s must be %s, got %s", name, list_of(shape).c_str(),
                     list_of(t.sizes()).c_str());
        throw Refused();
    }
}

void contiguous(const at::Tensor &t, const char *name) {
    if (!t.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
        throw Refused();
    }
}

// The pointer of a contiguous tensor; None passes as NULL where it may.
void *data(PyObject *o, ScalarType type, at::IntArrayRef shape, int dev, const char *name) {
    const at::Tensor &t = tensor(o, name);
    of_type(t, type, name);
    on_device(t, dev, name);
    contiguous(t, name);
    of_rank(t, (int)shape.size(), name);
    of_shape(t, shape, name);
    return t.data_ptr();
}
template <typename T>
T *need(PyObject *o, ScalarType type, at::IntArrayRef shape, int dev, const char *name) {
    return static_cast<T *>(data(o, type, shape, dev, name));
}
template <typename T>
T *maybe(PyObject *o, ScalarType type, at::IntArrayRef shape, int dev, const char *name) {
    return o == Py_None ? nullptr : need<T>(o, type, shape, dev, name);
}

// A workspace of any size.
struct Space {
    void *p = nullptr;
    size_t n = 0;
    Space(PyObject *o, int dev, const char *name) {
        if (o == Py_None) return;
        const at::Tensor &t = tensor(o, name);
        of_rank(t, 1, name);
        p = data(o, U8, t.sizes(), dev, name);
        n = (size_t)t.numel();
    }
};

// A [B,T,H,D] tensor whose tokens lie at one stride, heads packed.
struct Rows {
    void *p;
    int64_t stride;
    Rows() : p(nullptr), stride(0) {}
    Rows(PyObject *o, ScalarType type, at::IntArrayRef shape, int dev, const char *name) {
        const at::Tensor &t = tensor(o, name);
        of_type(t, type, name);
        on_device(t, dev, name);
        of_rank(t, 4, name);
        of_shape(t, shape, name);
        p = t.data_ptr();
        const int64_t B = shape[0], T = shape[1], H = shape[2], D = shape[3];
        stride = H * D;
        if (t.is_contiguous()) return;
        const auto s = t.strides();
        int64_t st = s[1];
        if (T == 1) st = B > 1 ? s[0] : H * D;
        if ((D > 1 && s[3] != 1) || (H > 1 && s[2] != D) || (B > 1 && T > 0 && s[0] != T * st)) {
            PyErr_Format(PyExc_ValueError,
                         "%s's tokens must lie at one stride, its heads packed; strides %s", name,
                         list_of(s).c_str());
            throw Refused();
        }
        stride = B * T <= 1 && st < H * D ? H * D : st;
    }
};

struct Freq {
    const double *p = nullptr;
    int rot = 0;
    Freq(PyObject *o, int dev) {
        if (o == Py_None) return;
        const at::Tensor &t = tensor(o, "freq");
        of_rank(t, 1, "freq");
        p = need<double>(o, F64, t.sizes(), dev, "freq");
        // (more pairs than any head has are refused by the call, however many)
        rot = 2 * (int)std::min<int64_t>(t.numel(), 1 << 20);
    }
};

int layout(PyObject *o) {
    if (PyUnicode_Check(o)) {
        if (PyUnicode_CompareWithASCIIString(o, "half") == 0) return QSA_ROPE_HALF;
        if (PyUnicode_CompareWithASCIIString(o, "interleaved") == 0) return QSA_ROPE_INTERLEAVED;
    }
    PyErr_Format(PyExc_ValueError, "layout must be one of ['half', 'interleaved'], got %R", o);
    throw Refused();
}

float real(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Refused();
    return (float)x;
}

int integer(PyObject *o) {
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred()) throw Refused();
    if (x != (int)x) {
        PyErr_SetString(PyExc_OverflowError, "integer argument out of range");
        throw Refused();
    }
    return (int)x;
}

int truth(PyObject *o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw Refused();
    return x;
}

int dtype(const at::Tensor &t, const char *name) {
    if (t.scalar_type() == BF) return QSA_BF16;
    if (t.scalar_type() == F32) return QSA_F32;
    PyErr_Format(PyExc_TypeError, "%s must be a torch.bfloat16 or torch.float32 tensor", name);
    throw Refused();
}

// The given stream (an object with .cuda_stream) or the device's current one.
void *stream_of(PyObject *o, int dev) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    PyObject *v = PyObject_GetAttrString(o, "cuda_stream");
    if (!v) throw Refused();
    void *s = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (!s && PyErr_Occurred()) throw Refused();
    return s;
}

// Runs `call` with `dev` current (the library launches on the current device); its status.
template <typename F>
PyObject *launch(int dev, F call) {
    int rc;
    {
        c10::cuda::OptionalCUDAGuard guard;
        if (c10::cuda::current_device() != dev) guard.set_index((c10::DeviceIndex)dev);
        PyThreadState *save = PyEval_SaveThread();
        rc = (int)call();
        PyEval_RestoreThread(save);
    }
    return PyLong_FromLong(rc);
}

// Argument counts, and C++ exceptions as Python's.
template <typename F>
PyObject *guarded(Py_ssize_t have, Py_ssize_t want, F body) {
    if (have != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, have);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// x, y, freq, pos, pos0, layout, mscale, transpose, stream
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        const at::Tensor &x = tensor(a[0], "x");
        const int dt = dtype(x, "x");
        of_rank(x, 4, "x");
        const int dev = on_device(x, -1, "x");
        const auto s = x.sizes();
        const Rows xr(a[0], x.scalar_type(), s, dev, "x"), yr(a[1], x.scalar_type(), s, dev, "y");
        const Freq f(a[2], dev);
        const auto *pos = maybe<int64_t>(a[3], I64, {s[0], s[1]}, dev, "pos");
        const auto *pos0 = maybe<int64_t>(a[4], I64, {s[0]}, dev, "pos0");
        const int lay = layout(a[5]), tr = truth(a[7]);
        const float m = real(a[6]);
        void *st = stream_of(a[8], dev);
        return launch(dev, [&] {
            return qsa_rope(xr.p, xr.stride, yr.p, yr.stride, dt, (int)s[0], s[1], (int)s[2],
                            (int)s[3], f.p, f.rot, lay, m, tr, pos, pos0, st);
        });
    });
}

// q, k, q_out, k_out, freq, v, v_out, q_weight, k_weight, eps, pos, pos0, layout, mscale,
// slot, ws, stream
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 17, [&]() -> PyObject * {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
        of_type(q, BF, "q");
        of_rank(q, 4, "q");
        of_type(k, BF, "k");
        of_rank(k, 4, "k");
        const int dev = on_device(q, -1, "q");
        const auto s = q.sizes();
        const int64_t B = s[0], T = s[1], Hq = s[2], D = s[3], Hkv = k.size(2);
        const int64_t kv[4] = {B, T, Hkv, D};
        const Rows qr(a[0], BF, s, dev, "q"), kr(a[1], BF, kv, dev, "k");
        const Rows vr = a[5] == Py_None ? Rows() : Rows(a[5], BF, kv, dev, "v");
        if ((a[5] == Py_None) != (a[6] == Py_None)) {
            PyErr_SetString(PyExc_ValueError, "v and v_out go together");
            return nullptr;
        }
        const at::Tensor &ko = tensor(a[3], "k_out");
        of_rank(ko, 4, "k_out");
        const int64_t L = a[14] == Py_None ? T : ko.size(1);
        const int64_t out[4] = {B, L, Hkv, D};
        auto *q_out = need<qsa_bf16_t>(a[2], BF, s, dev, "q_out");
        auto *k_out = need<qsa_bf16_t>(a[3], BF, out, dev, "k_out");
        auto *v_out = maybe<qsa_bf16_t>(a[6], BF, out, dev, "v_out");
        const Freq f(a[4], dev);
        const auto *qw = maybe<float>(a[7], F32, {D}, dev, "q_weight");
        const auto *kw = maybe<float>(a[8], F32, {D}, dev, "k_weight");
        const float eps = real(a[9]), m = real(a[13]);
        const auto *pos = maybe<int64_t>(a[10], I64, {B, T}, dev, "pos");
        const auto *pos0 = maybe<int64_t>(a[11], I64, {B}, dev, "pos0");
        const int lay = layout(a[12]);
        const auto *slot = maybe<int64_t>(a[14], I64, {B, T}, dev, "slot");
        const Space ws(a[15], dev, "ws");
        if (ws.p && ws.n < 256) {
            PyErr_SetString(PyExc_ValueError, "ws must hold the 256-byte status header");
            return nullptr;
        }
        void *st = stream_of(a[16], dev);
        return launch(dev, [&] {
            return qsa_qk_norm_rope((const qsa_bf16_t *)qr.p, qr.stride, (const qsa_bf16_t *)kr.p,
                                    kr.stride, (const qsa_bf16_t *)vr.p, vr.stride, (int)B, T,
                                    (int)Hq, (int)Hkv, (int)D, qw, kw, eps, f.p, f.rot, lay, m,
                                    pos, pos0, q_out, k_out, v_out, slot, L, ws.p, st);
        });
    });
}

// d_q, d_k, q, k, dq, dk, freq, ws, q_weight, k_weight, dq_weight, dk_weight, eps, pos,
// pos0, layout, mscale, stream
PyObject *qk_norm_rope_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 18, [&] {
        const at::Tensor &dy = tensor(a[0], "d_q"), &dx = tensor(a[4], "dq");
        const int dt = dtype(dy, "d_q"), xt = dtype(dx, "dq");
        const at::Tensor &q = tensor(a[2], "q"), &k = tensor(a[3], "k");
        of_type(q, BF, "q");
        of_rank(q, 4, "q");
        of_type(k, BF, "k");
        of_rank(k, 4, "k");
        const int dev = on_device(q, -1, "q");
        const auto s = q.sizes();
        const int64_t B = s[0], T = s[1], Hq = s[2], D = s[3], Hkv = k.size(2);
        const int64_t kv[4] = {B, T, Hkv, D};
        const Rows qr(a[2], BF, s, dev, "q"), kr(a[3], BF, kv, dev, "k");
        const void *d_q = need<void>(a[0], dy.scalar_type(), s, dev, "d_q");
        const void *d_k = need<void>(a[1], dy.scalar_type(), kv, dev, "d_k");
        void *dq = need<void>(a[4], dx.scalar_type(), s, dev, "dq");
        void *dk = need<void>(a[5], dx.scalar_type(), kv, dev, "dk");
        const Freq f(a[6], dev);
        const Space ws(a[7], dev, "ws");
        const auto *qw = maybe<float>(a[8], F32, {D}, dev, "q_weight");
        const auto *kw = maybe<float>(a[9], F32, {D}, dev, "k_weight");
        auto *dqw = maybe<float>(a[10], F32, {D}, dev, "dq_weight");
        auto *dkw = maybe<float>(a[11], F32, {D}, dev, "dk_weight");
        const float eps = real(a[12]), m = real(a[16]);
        const auto *pos = maybe<int64_t>(a[13], I64, {B, T}, dev, "pos");
        const auto *pos0 = maybe<int64_t>(a[14], I64, {B}, dev, "pos0");
        const int lay = layout(a[15]);
        void *st = stream_of(a[17], dev);
        return launch(dev, [&] {
            return qsa_qk_norm_rope_backward(
                d_q, d_k, dt, (const qsa_bf16_t *)qr.p, qr.stride, (const qsa_bf16_t *)kr.p,
                kr.stride, (int)B, T, (int)Hq, (int)Hkv, (int)D, qw, kw, eps, f.p, f.rot, lay, m,
                pos, pos0, dq, dk, xt, dqw, dkw, ws.p, ws.n, st);
        });
    });
}

// What both tree calls pass.
struct Tree {
    int dev;
    int64_t B, N, Hq, Hkv, D, L;
    const qsa_bf16_t *q, *k, *v;
    const int32_t *seqlens, *parent, *n_draft;
    float scale;
    qsa_bf16_t *o;
    float *lse;
    Space ws;
    // q, k_cache, v_cache, seqlens, parent, o, ws, n_draft, scale, lse
    static int device(PyObject *q) {
        const at::Tensor &t = tensor(q, "q");
        of_type(t, BF, "q");
        of_rank(t, 4, "q");
        return on_device(t, -1, "q");
    }
    explicit Tree(PyObject *const *a) : dev(device(a[0])), ws(a[6], dev, "ws") {
        const auto s = tensor(a[0], "q").sizes();
        const at::Tensor &c = tensor(a[1], "k_cache");
        of_rank(c, 4, "k_cache");
        B = s[0]; N = s[1]; Hq = s[2]; D = s[3]; L = c.size(1); Hkv = c.size(2);
        const int64_t cache[4] = {B, L, Hkv, D};
        q = need<qsa_bf16_t>(a[0], BF, s, dev, "q");
        k = need<qsa_bf16_t>(a[1], BF, cache, dev, "k_cache");
        v = need<qsa_bf16_t>(a[2], BF, cache, dev, "v_cache");
        seqlens = need<int32_t>(a[3], I32, {B}, dev, "seqlens");
        parent = need<int32_t>(a[4], I32, {B, N}, dev, "parent");
        o = need<qsa_bf16_t>(a[5], BF, s, dev, "o");
        n_draft = maybe<int32_t>(a[7], I32, {B}, dev, "n_draft");
        scale = a[8] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : real(a[8]);
        lse = maybe<float>(a[9], F32, {B, N, Hq}, dev, "lse");
    }
};

// Tree's, stream
PyObject *dense_tree_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const Tree t(a);
        void *st = stream_of(a[10], t.dev);
        return launch(t.dev, [&] {
            return qsa_dense_tree_decode(t.q, t.k, t.v, t.seqlens, t.L, t.parent, t.n_draft,
                                         (int)t.B, (int)t.N, (int)t.Hq, (int)t.Hkv, (int)t.D,
                                         t.scale, t.o, t.lse, t.ws.p, t.ws.n, st);
        });
    });
}

// Tree's, sel, r, budget, stream
PyObject *sparse_tree_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> PyObject * {
        const Tree t(a);
        const int r = integer(a[11]), budget = integer(a[12]);
        const at::Tensor &sel = tensor(a[10], "sel");
        of_type(sel, I32, "sel");
        on_device(sel, t.dev, "sel");
        of_rank(sel, 3, "sel");
        of_shape(sel, {t.B, t.N, r > 0 ? budget / r : 0}, "sel");
        if (sel.size(2) > 1 && sel.stride(2) != 1) {
            PyErr_SetString(PyExc_ValueError, "sel's entries must be contiguous");
            return nullptr;
        }
        void *st = stream_of(a[13], t.dev);
        return launch(t.dev, [&] {
            return qsa_sparse_tree_decode(t.q, t.k, t.v, t.seqlens, t.L,
                                          static_cast<const int32_t *>(sel.data_ptr()),
                                          sel.stride(0), sel.stride(1), t.parent, t.n_draft,
                                          (int)t.B, (int)t.N, (int)t.Hq, (int)t.Hkv, (int)t.D, r,
                                          budget, t.scale, t.o, t.lse, t.ws.p, t.ws.n, st);
        });
    });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL,
            nullptr};
}

PyMethodDef methods[] = {method<rope>("rope"),
                         method<qk_norm_rope>("qk_norm_rope"),
                         method<qk_norm_rope_backward>("qk_norm_rope_backward"),
                         method<dense_tree_decode>("dense_tree_decode"),
                         method<sparse_tree_decode>("sparse_tree_decode"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
