// The layer operators' calls from Python without the interpreter in between:
// a call's checks, its output tensors and its argument structure cost ctypes
// and Python 10 to 30 us of host time, more than the smallest kernels run
// (a rotation of one token 15 us, here 4).
//
// Every function takes the usual call only: arguments of the documented types
// and shapes on the current device, outputs to allocate, the current stream, no
// status word. For anything else, and whenever the library refuses, it returns
// None, and the Python face handles the call (or names what is wrong with it).
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <vector>

#include "mlaq.h"

namespace {

decltype(&mla_rope_axes) rope_axes_fn;
decltype(&mla_rope_axes_table) rope_axes_table_fn;
decltype(&mla_gated_ffn_fwd) ffn_fwd_fn;
decltype(&mla_gated_ffn_bwd) ffn_bwd_fn;
decltype(&mla_adamw_step) adamw_step_fn;
decltype(&mla_rms_norm_fwd) norm_fwd_fn;
decltype(&mla_rms_norm_bwd) norm_bwd_fn;
decltype(&mla_rms_norm_bwd_workspace_size) norm_bwd_size_fn;
decltype(&mla_kv_cache_write) cache_write_fn;
decltype(&mla_kv_cache_read) cache_read_fn;
decltype(&mla_cache_attn) attn_fn;
decltype(&mla_cache_attn_workspace_size) attn_size_fn;

// load(path): the library whose entry points are called.
PyObject* load(PyObject*, PyObject* path) {
    const char* p = PyUnicode_AsUTF8(path);
    if (!p) return nullptr;
    void* lib = dlopen(p, RTLD_NOW | RTLD_LOCAL);
    if (!lib) return PyErr_Format(PyExc_RuntimeError, "%s", dlerror());
    auto get = [&](auto& fn, const char* name) {
        fn = reinterpret_cast<std::remove_reference_t<decltype(fn)>>(dlsym(lib, name));
        return fn != nullptr;
    };
    if (!get(rope_axes_fn, "mla_rope_axes") || !get(rope_axes_table_fn, "mla_rope_axes_table") ||
        !get(ffn_fwd_fn, "mla_gated_ffn_fwd") || !get(ffn_bwd_fn, "mla_gated_ffn_bwd") ||
        !get(adamw_step_fn, "mla_adamw_step") || !get(norm_fwd_fn, "mla_rms_norm_fwd") ||
        !get(norm_bwd_fn, "mla_rms_norm_bwd") || !get(norm_bwd_size_fn, "mla_rms_norm_bwd_workspace_size") ||
        !get(cache_write_fn, "mla_kv_cache_write") || !get(cache_read_fn, "mla_kv_cache_read") ||
        !get(attn_fn, "mla_cache_attn") || !get(attn_size_fn, "mla_cache_attn_workspace_size"))
        return PyErr_Format(PyExc_RuntimeError, "%s lacks an entry point", p);
    Py_RETURN_NONE;
}

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A dense tensor of this type and rank, on the device of `like` (or any CUDA device).
bool dense(const at::Tensor* t, at::ScalarType type, int64_t dim, const at::Tensor* like) {
    return t && t->scalar_type() == type && t->dim() == dim && t->is_cuda() && t->is_contiguous() &&
           (!like || t->device() == like->device());
}
bool shaped(const at::Tensor& t, int64_t rows, int64_t cols) { return t.size(0) == rows && t.size(1) == cols; }

// The library launches on the current device.
bool here(const at::Tensor& t) { return t.device().index() == c10::cuda::current_device(); }

void* stream_of(const at::Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

// The tables, positions and axes of a rotary call.
bool rotary_args(const at::Tensor* cos, const at::Tensor* sin, const at::Tensor* pos, PyObject* axes, int64_t Dr,
                 const at::Tensor* like) {
    return dense(cos, at::kFloat, 2, like) && dense(sin, at::kFloat, 2, cos) && sin->sizes() == cos->sizes() &&
           dense(pos, at::kInt, 2, cos) && PyBytes_Check(axes) && Dr > 0 && PyBytes_GET_SIZE(axes) == Dr / 2;
}

// rope_axes(x, cos, sin, pos, axes, Dr, mode)
PyObject* rope_axes(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7) Py_RETURN_NONE;
    const at::Tensor *x = tensor(a[0]), *cos = tensor(a[1]), *sin = tensor(a[2]), *pos = tensor(a[3]);
    const int64_t Dr = PyLong_AsLongLong(a[5]);
    const int mode = (int)PyLong_AsLong(a[6]);
    if (PyErr_Occurred()) return nullptr;
    if (!x || !x->is_cuda() || !here(*x) || x->dim() != 3 || !rotary_args(cos, sin, pos, a[4], Dr, x)) Py_RETURN_NONE;
    const bool bf = x->scalar_type() == at::kBFloat16;
    const int64_t T = x->size(0), H = x->size(1), D = x->size(2), Ho = mode == MLA_ROPE_INVERSE_SUM ? 1 : H;
    if ((!bf && x->scalar_type() != at::kFloat) || (D > 1 && x->stride(2) != 1) || Dr > D || pos->size(1) != T ||
        H > INT32_MAX || D > INT32_MAX || pos->size(0) > INT32_MAX)
        Py_RETURN_NONE;
    at::Tensor out = at::empty({T, Ho, D}, x->options());
    const mla_rope_axes_shape s{T,
                                (int32_t)H,
                                (int32_t)(D - Dr),
                                (int32_t)Dr,
                                (int32_t)pos->size(0),
                                cos->size(0),
                                cos->size(1),
                                T > 1 ? x->stride(0) : 0,
                                H > 1 ? x->stride(1) : 0,
                                T > 1 ? Ho * D : 0,
                                Ho > 1 ? D : 0,
                                0};
    const int st = rope_axes_fn(&s, bf ? MLA_IN_BF16 : MLA_IN_F32, mode, x->data_ptr(), cos->data_ptr<float>(),
                                sin->data_ptr<float>(), pos->data_ptr<int32_t>(),
                                reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(a[4])), out.data_ptr(), nullptr,
                                stream_of(*x));
    if (st != MLA_OK) Py_RETURN_NONE;
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// rope_axes_table(cos, sin, pos, axes, Dr)
PyObject* rope_axes_table(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 5) Py_RETURN_NONE;
    const at::Tensor *cos = tensor(a[0]), *sin = tensor(a[1]), *pos = tensor(a[2]);
    const int64_t Dr = PyLong_AsLongLong(a[4]);
    if (PyErr_Occurred()) return nullptr;
    if (!rotary_args(cos, sin, pos, a[3], Dr, nullptr) || !here(*cos) || Dr > INT32_MAX || pos->size(0) > INT32_MAX)
        Py_RETURN_NONE;
    const int64_t T = pos->size(1);
    at::Tensor c = at::empty({T, Dr}, cos->options()), s = at::empty({T, Dr}, cos->options());
    const mla_rope_axes_shape shape{T, 1, 0, (int32_t)Dr, (int32_t)pos->size(0), cos->size(0), cos->size(1), 0, 0, 0, 0, 0};
    const int st = rope_axes_table_fn(&shape, cos->data_ptr<float>(), sin->data_ptr<float>(), pos->data_ptr<int32_t>(),
                                      reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(a[3])), c.data_ptr<float>(),
                                      s.data_ptr<float>(), nullptr, stream_of(*pos));
    if (st != MLA_OK) Py_RETURN_NONE;
    PyObject *pc = THPVariable_Wrap(std::move(c)), *ps = THPVariable_Wrap(std::move(s));
    PyObject* r = pc && ps ? PyTuple_Pack(2, pc, ps) : nullptr;
    Py_XDECREF(pc);
    Py_XDECREF(ps);
    return r;
    END_HANDLE_TH_ERRORS
}

// x's row pitch when it is a bf16 matrix of contiguous rows like [T, K] that do not overlap, else -1. (A pitch of 0,
// one row for all tokens, would say dense to the library.)
int64_t row_pitch(const at::Tensor* x, int64_t T, int64_t K) {
    if (x->scalar_type() != at::kBFloat16 || x->dim() != 2 || !shaped(*x, T, K) || (K > 1 && x->stride(1) != 1)) return -1;
    if (T <= 1) return K;
    return x->stride(0) >= K ? x->stride(0) : -1;
}

// ffn_fwd(x, w_gate_up, w_down, act, save)
PyObject* ffn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 5) Py_RETURN_NONE;
    const at::Tensor *x = tensor(a[0]), *wgu = tensor(a[1]), *wd = tensor(a[2]);
    const int act = (int)PyLong_AsLong(a[3]), save = PyObject_IsTrue(a[4]);
    if (PyErr_Occurred()) return nullptr;
    if (!x || !x->is_cuda() || !here(*x) || x->dim() != 2 || !dense(wd, at::kBFloat16, 2, x) || !dense(wgu, at::kBFloat16, 2, x))
        Py_RETURN_NONE;
    const int64_t T = x->size(0), K = x->size(1), F = wd->size(1), ld = row_pitch(x, T, K);
    if (ld < 0 || wd->size(0) != K || !shaped(*wgu, 2 * F, K)) Py_RETURN_NONE;
    at::Tensor y = at::empty({T, K}, x->options()), h = at::empty({T, F}, x->options()), gu;
    if (save) gu = at::empty({T, 2 * F}, x->options());
    const mla_ffn_shape s{T, K, F, ld, act, 0};
    if (ffn_fwd_fn(&s, x->data_ptr(), wgu->data_ptr(), wd->data_ptr(), save ? gu.data_ptr() : nullptr, h.data_ptr(),
                   y.data_ptr(), nullptr, stream_of(*x)) != MLA_OK)
        Py_RETURN_NONE;
    if (!save) return THPVariable_Wrap(std::move(y));
    PyObject *py = THPVariable_Wrap(std::move(y)), *pg = THPVariable_Wrap(std::move(gu)),
             *ph = THPVariable_Wrap(std::move(h));
    PyObject* r = py && pg && ph ? PyTuple_Pack(3, py, pg, ph) : nullptr;
    Py_XDECREF(py);
    Py_XDECREF(pg);
    Py_XDECREF(ph);
    return r;
    END_HANDLE_TH_ERRORS
}

// ffn_bwd(dy, x, w_gate_up, w_down, gate_up, h, act): all three gradients
PyObject* ffn_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7) Py_RETURN_NONE;
    const at::Tensor *dy = tensor(a[0]), *x = tensor(a[1]), *wgu = tensor(a[2]), *wd = tensor(a[3]), *gu = tensor(a[4]),
                     *h = tensor(a[5]);
    const int act = (int)PyLong_AsLong(a[6]);
    if (PyErr_Occurred()) return nullptr;
    if (!dense(dy, at::kBFloat16, 2, nullptr) || !here(*dy) || !x || x->device() != dy->device() || !dense(wgu, at::kBFloat16, 2, dy) ||
        !dense(wd, at::kBFloat16, 2, dy) || !dense(gu, at::kBFloat16, 2, dy) || !dense(h, at::kBFloat16, 2, dy))
        Py_RETURN_NONE;
    const int64_t T = dy->size(0), K = dy->size(1), F = wd->size(1), ld = row_pitch(x, T, K);
    if (ld < 0 || wd->size(0) != K || !shaped(*wgu, 2 * F, K) || !shaped(*gu, T, 2 * F) || !shaped(*h, T, F))
        Py_RETURN_NONE;
    const auto o = dy->options();
    at::Tensor dgu = at::empty({T, 2 * F}, o), dx = at::empty({T, K}, o), dwgu = at::empty({2 * F, K}, o),
               dwd = at::empty({K, F}, o);
    const mla_ffn_shape s{T, K, F, ld, act, 0};
    if (ffn_bwd_fn(&s, dy->data_ptr(), x->data_ptr(), wgu->data_ptr(), wd->data_ptr(), gu->data_ptr(), h->data_ptr(),
                   dgu.data_ptr(), dx.data_ptr(), dwgu.data_ptr(), dwd.data_ptr(), nullptr, stream_of(*dy)) != MLA_OK)
        Py_RETURN_NONE;
    PyObject *p0 = THPVariable_Wrap(std::move(dx)), *p1 = THPVariable_Wrap(std::move(dwgu)),
             *p2 = THPVariable_Wrap(std::move(dwd));
    PyObject* r = p0 && p1 && p2 ? PyTuple_Pack(3, p0, p1, p2) : nullptr;
    Py_XDECREF(p0);
    Py_XDECREF(p1);
    Py_XDECREF(p2);
    return r;
    END_HANDLE_TH_ERRORS
}

// adamw_step(plan_host, plan_device, device index, plan's stream, step, lr, beta1, beta2, eps, weight_decay,
// grad_scale or None, seed or None): True, or None (also on another stream than the plan's)
PyObject* adamw_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 12) Py_RETURN_NONE;
    const uintptr_t host = (uintptr_t)PyLong_AsUnsignedLongLong(a[0]), dev = (uintptr_t)PyLong_AsUnsignedLongLong(a[1]);
    const int index = (int)PyLong_AsLong(a[2]);
    const uintptr_t on = (uintptr_t)PyLong_AsUnsignedLongLong(a[3]);
    mla_adamw_args q{};
    q.step = PyLong_AsLongLong(a[4]);
    q.lr = PyFloat_AsDouble(a[5]);
    q.beta1 = PyFloat_AsDouble(a[6]);
    q.beta2 = PyFloat_AsDouble(a[7]);
    q.eps = PyFloat_AsDouble(a[8]);
    q.weight_decay = PyFloat_AsDouble(a[9]);
    const float* scale = nullptr;
    if (a[10] != Py_None) {
        const at::Tensor* t = tensor(a[10]);
        if (!t || !t->is_cuda() || t->scalar_type() != at::kFloat || t->numel() != 1 || t->device().index() != index)
            Py_RETURN_NONE;
        scale = t->data_ptr<float>();
    }
    if (a[11] != Py_None) {
        q.stochastic = 1;
        q.seed = (uint32_t)PyLong_AsUnsignedLongMask(a[11]);
    }
    if (PyErr_Occurred()) return nullptr;
    if (index < 0 || index != c10::cuda::current_device()) Py_RETURN_NONE;
    void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
    if (reinterpret_cast<uintptr_t>(stream) != on) Py_RETURN_NONE;
    if (adamw_step_fn(reinterpret_cast<const void*>(host), reinterpret_cast<const void*>(dev), &q, scale, stream) != MLA_OK)
        Py_RETURN_NONE;
    Py_RETURN_TRUE;
    END_HANDLE_TH_ERRORS
}

// adamw_places(list or None, ...): the address, size, type and layout of every tensor of the lists, as bytes that are
// equal when all of these are. None when something else is listed.
PyObject* adamw_places(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    std::vector<int64_t> v;
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (a[i] == Py_None) {
            v.push_back(-1);
            continue;
        }
        if (!PyList_Check(a[i])) Py_RETURN_NONE;
        const Py_ssize_t count = PyList_GET_SIZE(a[i]);
        v.push_back(count);
        for (Py_ssize_t k = 0; k < count; ++k) {
            const at::Tensor* t = tensor(PyList_GET_ITEM(a[i], k));
            if (!t || t->layout() != at::kStrided) Py_RETURN_NONE;
            v.push_back((int64_t)reinterpret_cast<uintptr_t>(t->data_ptr()));
            v.push_back(t->numel());
            v.push_back((int64_t)t->scalar_type() * 2 + t->is_contiguous());
        }
    }
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(v.data()), (Py_ssize_t)(v.size() * sizeof(int64_t)));
    END_HANDLE_TH_ERRORS
}

// adamw_keep(list of gradients): their memory stays until the current stream has read them, whichever stream they are
// of (nothing to do where it is this one). True, or None when something else is listed.
PyObject* adamw_keep(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 1 || !PyList_Check(a[0])) Py_RETURN_NONE;
    for (Py_ssize_t k = 0; k < PyList_GET_SIZE(a[0]); ++k) {
        const at::Tensor* t = tensor(PyList_GET_ITEM(a[0], k));
        if (!t || !t->is_cuda()) Py_RETURN_NONE;
        c10::cuda::CUDACachingAllocator::recordStream(t->storage().data_ptr(),
                                                      c10::cuda::getCurrentCUDAStream(t->device().index()));
    }
    Py_RETURN_TRUE;
    END_HANDLE_TH_ERRORS
}

// The tensors as a tuple (one: itself); they are given up.
PyObject* wrapped(std::vector<at::Tensor> v) {
    if (v.size() == 1) return THPVariable_Wrap(std::move(v[0]));
    PyObject* r = PyTuple_New((Py_ssize_t)v.size());
    for (size_t i = 0; r && i < v.size(); ++i) {
        PyObject* o = nullptr;
        if (v[i].defined()) o = THPVariable_Wrap(std::move(v[i]));
        else Py_INCREF(o = Py_None);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, (Py_ssize_t)i, o);
    }
    return r;
}

// An optional tensor: false when o is neither one nor None.
bool optional(PyObject* o, const at::Tensor*& t) {
    t = o == Py_None ? nullptr : tensor(o);
    return t || o == Py_None;
}

bool float_type(const at::Tensor* t) { return t->scalar_type() == at::kFloat || t->scalar_type() == at::kBFloat16; }
int in_type(const at::Tensor* t) { return t->scalar_type() == at::kFloat ? MLA_IN_F32 : MLA_IN_BF16; }

// The row pitch of a matrix like `like` (itself: null) whose rows are contiguous and do not overlap, else -1.
int64_t norm_pitch(const at::Tensor* t, const at::Tensor* like) {
    if (!t || !t->is_cuda() || t->dim() != 2 || !float_type(t)) return -1;
    if (like && (t->scalar_type() != like->scalar_type() || t->sizes() != like->sizes() || t->device() != like->device()))
        return -1;
    const int64_t T = t->size(0), K = t->size(1);
    if (K > 1 && t->stride(1) != 1) return -1;
    if (T <= 1) return K;
    return t->stride(0) >= K ? t->stride(0) : -1;
}
bool norm_weight(const at::Tensor* w, const at::Tensor* x) {
    return w && float_type(w) && dense(w, w->scalar_type(), 1, x) && w->size(0) == x->size(1);
}

// rms_norm_fwd(x, weight, eps, residual, out mode, save): y, then scales, h and rstd where there are any
PyObject* rms_norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 6) Py_RETURN_NONE;
    const at::Tensor *x = tensor(a[0]), *w = tensor(a[1]), *res;
    const double eps = PyFloat_AsDouble(a[2]);
    const int mode = (int)PyLong_AsLong(a[4]), save = PyObject_IsTrue(a[5]);
    if (PyErr_Occurred()) return nullptr;
    const int64_t ld_x = norm_pitch(x, nullptr);
    if (ld_x < 0 || !here(*x) || !norm_weight(w, x) || !optional(a[3], res)) Py_RETURN_NONE;
    const int64_t T = x->size(0), K = x->size(1), ld_res = res ? norm_pitch(res, x) : 0;
    if (ld_res < 0) Py_RETURN_NONE;
    const bool mx = mode != MLA_NORM_OUT_SAME;
    if (mx && K % 32 != 0) Py_RETURN_NONE;
    std::vector<at::Tensor> v;
    const auto bytes = x->options().dtype(at::kByte);
    v.push_back(at::empty({T, K}, mx ? bytes : x->options()));
    if (mode == MLA_NORM_OUT_MXFP8) v.push_back(at::empty({T, K / 32}, bytes));
    if (mode == MLA_NORM_OUT_MXFP8_TILED) v.push_back(at::empty({(T + 127) / 128 * ((K / 32 + 3) / 4) * 512}, bytes));
    void *scales = mx ? v[1].data_ptr() : nullptr, *h = nullptr;
    float* rstd = nullptr;
    if (res) {
        v.push_back(at::empty({T, K}, x->options()));
        h = v.back().data_ptr();
    }
    if (save) {
        v.push_back(at::empty({T}, x->options().dtype(at::kFloat)));
        rstd = v.back().data_ptr<float>();
    }
    const mla_norm_shape s{T, K, ld_x, ld_res, 0, in_type(x), in_type(w), mode, (float)eps, 0};
    if (norm_fwd_fn(&s, x->data_ptr(), res ? res->data_ptr() : nullptr, w->data_ptr(), h, v[0].data_ptr(),
                    static_cast<uint8_t*>(scales), rstd, stream_of(*x)) != MLA_OK)
        Py_RETURN_NONE;
    return wrapped(std::move(v));
    END_HANDLE_TH_ERRORS
}

// rms_norm_bwd(dy, h, weight, rstd, dres): both gradients
PyObject* rms_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 5) Py_RETURN_NONE;
    const at::Tensor *dy = tensor(a[0]), *h = tensor(a[1]), *w = tensor(a[2]), *rstd = tensor(a[3]), *dres;
    const int64_t ld_x = norm_pitch(h, nullptr);
    if (ld_x < 0 || !here(*h) || !norm_weight(w, h) || !dense(rstd, at::kFloat, 1, h) || !optional(a[4], dres))
        Py_RETURN_NONE;
    const int64_t T = h->size(0), K = h->size(1), ld_dy = norm_pitch(dy, h), ld_res = dres ? norm_pitch(dres, h) : 0;
    if (ld_dy < 0 || ld_res < 0 || rstd->size(0) != T) Py_RETURN_NONE;
    const mla_norm_shape s{T, K, ld_x, ld_res, ld_dy, in_type(h), in_type(w), MLA_NORM_OUT_SAME, 0.f, 0};
    const int64_t size = (int64_t)norm_bwd_size_fn(&s);
    at::Tensor dx = at::empty({T, K}, h->options()), dw = at::empty({K}, w->options()),
               ws = at::empty({size}, h->options().dtype(at::kByte));
    if (norm_bwd_fn(&s, dy->data_ptr(), h->data_ptr(), w->data_ptr(), rstd->data_ptr<float>(),
                    dres ? dres->data_ptr() : nullptr, dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), (size_t)size,
                    stream_of(*h)) != MLA_OK)
        Py_RETURN_NONE;
    return wrapped({dx, dw});
    END_HANDLE_TH_ERRORS
}

// The cache of a[0..4]: k, k_scales, v, v_scales, Dv. False when it is not one on the current device.
bool cache_args(PyObject* const* a, mla_kv_cache& c, const at::Tensor*& k) {
    const at::Tensor *ks = tensor(a[1]), *v, *vs;
    k = tensor(a[0]);
    if (!dense(k, at::kByte, 4, nullptr) || !here(*k) || !dense(ks, at::kByte, 3, k) || !optional(a[2], v) ||
        !optional(a[3], vs) || !v != !vs)
        return false;
    const int64_t pages = k->size(0), H = k->size(1), page = k->size(2), Dk = k->size(3), per = ks->size(2);
    const int64_t Dv = PyLong_AsLongLong(a[4]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    if (ks->size(0) != pages || ks->size(1) != H || per < 1 || page < 16 || page > 1024 || page % per != 0 || H > 65535 ||
        Dk > 4096 || Dv < 1 || Dv > 4096)
        return false;
    if (v && (!dense(v, at::kByte, 4, k) || v->size(0) != pages || v->size(1) != H || v->size(2) != page ||
              v->size(3) != Dv || !dense(vs, at::kByte, 3, k) || vs->sizes() != ks->sizes()))
        return false;
    c = {pages, (int32_t)page, (int32_t)(page / per), (int32_t)H, (int32_t)Dk, (int32_t)Dv, 0,
         static_cast<uint8_t*>(k->data_ptr()), static_cast<uint8_t*>(ks->data_ptr()),
         v ? static_cast<uint8_t*>(v->data_ptr()) : nullptr, vs ? static_cast<uint8_t*>(vs->data_ptr()) : nullptr};
    return true;
}

// table [B, width], positions [B], cu [B + 1] or None, for T rows.
bool sequence_args(const at::Tensor* table, const at::Tensor* at, const at::Tensor* cu, int64_t T, const at::Tensor* like) {
    return dense(table, at::kInt, 2, like) && dense(at, at::kInt, 1, like) && at->size(0) == table->size(0) &&
           (cu ? dense(cu, at::kInt, 1, like) && cu->size(0) == table->size(0) + 1 : T == table->size(0));
}

// bf16 rows [T, H, D] with unit inner stride
bool rows3(const at::Tensor* t, int64_t H, int64_t D, const at::Tensor* like) {
    return t && t->scalar_type() == at::kBFloat16 && t->dim() == 3 && t->size(1) == H && t->size(2) == D && t->is_cuda() &&
           t->device() == like->device() && (D <= 1 || t->stride(2) == 1);
}
int64_t token_stride(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : 0; }
int64_t head_stride(const at::Tensor& t) { return t.size(1) > 1 ? t.stride(1) : 0; }
const int32_t* ints(const at::Tensor* t) { return t ? t->data_ptr<int32_t>() : nullptr; }

// kv_cache_write(the cache's five, k, v, table, start, cu): True
PyObject* kv_cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 10) Py_RETURN_NONE;
    mla_kv_cache c;
    const at::Tensor *ck, *k = tensor(a[5]), *v, *table = tensor(a[7]), *start = tensor(a[8]), *cu;
    if (!cache_args(a, c, ck) || !rows3(k, c.H, c.Dk, ck) || !optional(a[6], v) || !optional(a[9], cu) || !v != !c.v)
        Py_RETURN_NONE;
    const int64_t T = k->size(0);
    if ((v && (!rows3(v, c.H, c.Dv, ck) || v->size(0) != T)) || !sequence_args(table, start, cu, T, ck)) Py_RETURN_NONE;
    if (cache_write_fn(&c, k->data_ptr(), token_stride(*k), head_stride(*k), v ? v->data_ptr() : nullptr,
                       v ? token_stride(*v) : 0, v ? head_stride(*v) : 0, T, table->size(0), ints(table), table->size(1),
                       ints(start), ints(cu), nullptr, stream_of(*ck)) != MLA_OK)
        Py_RETURN_NONE;
    Py_RETURN_TRUE;
    END_HANDLE_TH_ERRORS
}

// kv_cache_read(the cache's five, table, start, tokens, cu, dtype): (k, v or None)
PyObject* kv_cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 10) Py_RETURN_NONE;
    mla_kv_cache c;
    const at::Tensor *ck, *table = tensor(a[5]), *start = tensor(a[6]), *cu;
    const int64_t T = PyLong_AsLongLong(a[7]);
    const int dtype = (int)PyLong_AsLong(a[9]);
    if (PyErr_Occurred()) return nullptr;
    if (!cache_args(a, c, ck) || !optional(a[8], cu) || T < 0 || !sequence_args(table, start, cu, T, ck)) Py_RETURN_NONE;
    const auto o = ck->options().dtype(dtype == MLA_IN_F32 ? at::kFloat : at::kBFloat16);
    at::Tensor k = at::empty({T, c.H, c.Dk}, o), v;
    if (c.v) v = at::empty({T, c.H, c.Dv}, o);
    if (cache_read_fn(&c, k.data_ptr(), c.v ? v.data_ptr() : nullptr, dtype, T, table->size(0), ints(table),
                      table->size(1), ints(start), ints(cu), nullptr, stream_of(*ck)) != MLA_OK)
        Py_RETURN_NONE;
    return wrapped({k, v});
    END_HANDLE_TH_ERRORS
}

// cache_attn(q, the cache's five, table, length, cu, scale (NaN: Dk^-1/2), lse): out or (out, lse)
PyObject* cache_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 11) Py_RETURN_NONE;
    mla_kv_cache c;
    const at::Tensor *q = tensor(a[0]), *ck, *table = tensor(a[6]), *length = tensor(a[7]), *cu;
    double scale = PyFloat_AsDouble(a[9]);
    const int want = PyObject_IsTrue(a[10]);
    if (PyErr_Occurred()) return nullptr;
    if (!cache_args(a + 1, c, ck) || !optional(a[8], cu) || !q || q->dim() != 3 || !rows3(q, q->size(1), c.Dk, ck) ||
        q->size(1) < 1 || q->size(1) > INT32_MAX || !sequence_args(table, length, cu, q->size(0), ck))
        Py_RETURN_NONE;
    if (scale != scale) scale = 1.0 / std::sqrt((double)c.Dk);
    const int64_t T = q->size(0), Hq = q->size(1);
    const mla_attn_shape s{T, table->size(0), token_stride(*q), head_stride(*q), table->size(1), (int32_t)Hq, (float)scale, 0};
    const int64_t size = (int64_t)attn_size_fn(&s, &c);
    at::Tensor out = at::empty({T, Hq, c.Dv}, q->options()), lse, ws = at::empty({size}, ck->options());
    if (want) lse = at::empty({T, Hq}, q->options().dtype(at::kFloat));
    if (attn_fn(&s, &c, q->data_ptr(), ints(table), ints(length), ints(cu), out.data_ptr(),
                want ? lse.data_ptr<float>() : nullptr, ws.data_ptr(), (size_t)size, nullptr, stream_of(*ck)) != MLA_OK)
        Py_RETURN_NONE;
    if (!want) return wrapped({out});
    return wrapped({out, lse});
    END_HANDLE_TH_ERRORS
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"load", load, METH_O, "Use the entry points of the library at this path."},
    {"rope_axes", fast(rope_axes), METH_FASTCALL, nullptr},
    {"rope_axes_table", fast(rope_axes_table), METH_FASTCALL, nullptr},
    {"ffn_fwd", fast(ffn_fwd), METH_FASTCALL, nullptr},
    {"ffn_bwd", fast(ffn_bwd), METH_FASTCALL, nullptr},
    {"adamw_step", fast(adamw_step), METH_FASTCALL, nullptr},
    {"adamw_places", fast(adamw_places), METH_FASTCALL, nullptr},
    {"adamw_keep", fast(adamw_keep), METH_FASTCALL, nullptr},
    {"rms_norm_fwd", fast(rms_norm_fwd), METH_FASTCALL, nullptr},
    {"rms_norm_bwd", fast(rms_norm_bwd), METH_FASTCALL, nullptr},
    {"kv_cache_write", fast(kv_cache_write), METH_FASTCALL, nullptr},
    {"kv_cache_read", fast(kv_cache_read), METH_FASTCALL, nullptr},
    {"cache_attn", fast(cache_attn), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
