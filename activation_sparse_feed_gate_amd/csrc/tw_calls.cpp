// tw_calls.cpp -- the allocating calls of the Python binding (layer and RMS norm,
// int8 products, gated FFN, cross entropy, gradient clipping) in native code: checks
// of the tensors, allocation of the outputs and the call of the C ABI.  A decoded
// token's norm runs 4 us on the GPU; the same steps in interpreted Python took 20 us of
// host time, which then set the pace of a loop of small calls (here 6 us, of which 2.6
// are the launch and 0.7 each of the four outputs).
//
// Each function returns its tensor or a dict of them, or None when anything
// about its arguments is not as the library needs it or the library refuses
// the call: tw.py then makes the call through its checked low-level function,
// which raises the error with its message.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <vector>

#include "tw.h"

namespace {

using at::Tensor;

// One call's arguments: what is wrong with any of them ends in !ok.
struct Call {
    bool ok = true;
    at::Device device = at::kCPU;

    const Tensor *tensor(PyObject *o) {
        if (!THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(o);
    }
    // A two-dimensional device tensor with contiguous rows; it sets the device.
    const Tensor *rows(PyObject *o, bool int8, int *type, int64_t *stride) {
        const Tensor *t = tensor(o);
        if (!t || t->dim() != 2 || !t->is_cuda() || !kind(t->scalar_type(), int8, type)) {
            ok = false;
            return nullptr;
        }
        const int64_t M = t->size(0), K = t->size(1);
        if (M > INT32_MAX || K > INT32_MAX || (K > 1 && M > 0 && t->stride(1) != 1)) ok = false;
        *stride = M > 1 ? t->stride(0) : K;
        device = t->device();
        return t;
    }
    bool kind(at::ScalarType s, bool int8, int *type) {
        if (s == at::kBFloat16) *type = TW_BF16;
        else if (s == at::kFloat) *type = TW_F32;
        else if (int8 && s == at::kChar) *type = TW_INT8;
        else return ok = false;
        return true;
    }
    // Address of a contiguous tensor of this type and shape (cols < 0: one
    // dimension); null for None where that is allowed.
    void *need(PyObject *o, at::ScalarType s, int64_t n, int64_t cols = -1) {
        const Tensor *t = tensor(o);
        if (!t) return nullptr;
        const bool shape = cols < 0 ? t->dim() == 1 && t->size(0) == n
                                    : t->dim() == 2 && t->size(0) == n && t->size(1) == cols;
        if (!shape || t->scalar_type() != s || t->device() != device || !t->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        return t->data_ptr();
    }
    void *opt(PyObject *o, at::ScalarType s, int64_t n, int64_t cols = -1) {
        return o == Py_None ? nullptr : need(o, s, n, cols);
    }
    // The same for a matrix of either floating type.
    void *matrix(PyObject *o, int *type, int64_t m, int64_t n) {
        const Tensor *t = tensor(o);
        if (!t || !kind(t->scalar_type(), false, type)) return nullptr;
        return need(o, t->scalar_type(), m, n);
    }
    void *opt_matrix(PyObject *o, int *type, int64_t m, int64_t n) {
        *type = 0;
        return o == Py_None ? nullptr : matrix(o, type, m, n);
    }
    at::ScalarType dtype(PyObject *o, int *type) {
        if (!THPDtype_Check(o)) {
            ok = false;
            return at::kFloat;
        }
        const at::ScalarType s = reinterpret_cast<THPDtype *>(o)->scalar_type;
        kind(s, false, type);
        return s;
    }
    float real(PyObject *o) {
        const double v = PyFloat_AsDouble(o);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return (float)v;
    }
    Tensor empty(at::IntArrayRef size, at::ScalarType s) const {
        return Tensor(at::detail::empty_cuda(size, s, device, std::nullopt));
    }
    // The current stream of the tensors' device.
    void *stream() const {
        return c10::hip::getCurrentHIPStreamMasqueradingAsCUDA(device.index()).stream();
    }
};

PyObject *none() { Py_RETURN_NONE; }

PyObject *wrapped(const Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    return none();
}

// {name: tensor, ...}, with None for tensors that the call has not.
struct Named {
    const char *name;
    const Tensor &t;
};
template <size_t N>
PyObject *dict_of(const Named (&items)[N]) {
    PyObject *d = PyDict_New();
    if (!d) return nullptr;
    for (const Named &i : items) {
        PyObject *v = wrapped(i.t);
        const int bad = v ? PyDict_SetItemString(d, i.name, v) : -1;
        Py_XDECREF(v);
        if (bad) {
            Py_DECREF(d);
            return nullptr;
        }
    }
    return d;
}

// C++ exceptions (an allocation that fails) end in None too: the Python path
// meets the same condition and raises torch's own error.
template <typename F>
PyObject *guarded(F f) {
    try {
        return f();
    } catch (...) {
        return none();
    }
}

// layernorm(x, gamma, beta, eps, add, out_dtype) -> {y, sum, mean, rstd}
PyObject *layernorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 6) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        int xt, at_, yt;
        int64_t stride;
        const Tensor *x = c.rows(a[0], false, &xt, &stride);
        if (!x) return none();
        const int64_t M = x->size(0), K = x->size(1);
        auto gamma = (const float *)c.need(a[1], at::kFloat, K);
        auto beta = (const float *)c.opt(a[2], at::kFloat, K);
        const float eps = c.real(a[3]);
        const void *add = c.opt_matrix(a[4], &at_, M, K);
        const at::ScalarType os = c.dtype(a[5], &yt);
        if (!c.ok) return none();
        const c10::DeviceGuard guard(c.device);
        Tensor y = c.empty({M, K}, os), sum, mean = c.empty({M}, at::kFloat),
               rstd = c.empty({M}, at::kFloat);
        if (a[4] != Py_None) sum = c.empty({M, K}, x->scalar_type());
        if (tw_layernorm_fwd(x->data_ptr(), xt, stride, add, at_, gamma, beta, eps, (int)M, (int)K,
                             sum.defined() ? sum.data_ptr() : nullptr, y.data_ptr(), yt,
                             mean.data_ptr<float>(), rstd.data_ptr<float>(), c.stream(),
                             nullptr) != TW_OK)
            return none();
        return dict_of({{"y", y}, {"sum", sum}, {"mean", mean}, {"rstd", rstd}});
    });
}

// layernorm_backward(dy, x, gamma, mean, rstd, dres, dx_dtype) -> {dx, dgamma, dbeta}
PyObject *layernorm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 7) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        int xt, dt, ot;
        int64_t stride;
        const Tensor *x = c.rows(a[1], false, &xt, &stride);
        if (!x) return none();
        const int64_t M = x->size(0), K = x->size(1);
        const void *dy = c.matrix(a[0], &dt, M, K);
        auto gamma = (const float *)c.need(a[2], at::kFloat, K);
        auto mean = (const float *)c.need(a[3], at::kFloat, M);
        auto rstd = (const float *)c.need(a[4], at::kFloat, M);
        const at::ScalarType os = c.dtype(a[6], &ot);
        const void *dres = c.opt(a[5], os, M, K);
        if (!c.ok) return none();
        const c10::DeviceGuard guard(c.device);
        const size_t nws = tw_layernorm_bwd_workspace_bytes((int)M, (int)K);
        Tensor dx = c.empty({M, K}, os), dg = c.empty({K}, at::kFloat),
               db = c.empty({K}, at::kFloat), ws = c.empty({(int64_t)nws}, at::kByte);
        if (tw_layernorm_bwd(dy, dt, x->data_ptr(), xt, stride, gamma, mean, rstd, dres, (int)M,
                             (int)K, dx.data_ptr(), ot, dg.data_ptr<float>(),
                             db.data_ptr<float>(), ws.data_ptr(), nws, c.stream(),
                             nullptr) != TW_OK)
            return none();
        return dict_of({{"dx", dx}, {"dgamma", dg}, {"dbeta", db}});
    });
}

// Input of a product: float rows and a workspace, or int8 rows with scales.
struct ProductIn {
    const Tensor *x = nullptr;
    int type = 0;
    int64_t stride = 0, M = 0, K = 0;
    const float *scale = nullptr;
    ProductIn(Call &c, PyObject *xo, PyObject *so) {
        x = c.rows(xo, true, &type, &stride);
        if (!x) return;
        M = x->size(0);
        K = x->size(1);
        if (type == TW_INT8) scale = (const float *)c.need(so, at::kFloat, M);
        else if (so != Py_None) c.ok = false;
    }
    size_t bytes() const {
        return type == TW_INT8 ? 0 : tw_quant_workspace_bytes((int)M, (int)K);
    }
};

// The workspace of a call: the caller's, or one for this call.
struct Workspace {
    Tensor own;
    void *p = nullptr;
    size_t bytes = 0;
    Workspace(Call &c, PyObject *o, size_t need) {
        if (o != Py_None) {
            const Tensor *t = c.tensor(o);
            if (!t || t->device() != c.device || !t->is_contiguous()) {
                c.ok = false;
                return;
            }
            p = t->data_ptr();
            bytes = t->nbytes();
        } else if (c.ok && need) {
            own = c.empty({(int64_t)need}, at::kByte);
            p = own.data_ptr();
            bytes = need;
        }
    }
};

// Address of a row's values at 16 bytes, as the library takes it: a contiguous tensor
// that begins elsewhere (tokens[1:]) is copied, on the current stream of its device.
struct Aligned {
    Tensor own;
    const void *p;
    Aligned(PyObject *o, const void *at) : p(at) {
        if (reinterpret_cast<uintptr_t>(at) % 16 == 0) return;
        own = THPVariable_Unpack(o).clone();
        p = own.data_ptr();
    }
};

// Rows of a weight matrix (its first dimension).
int64_t rows_of(Call &c, PyObject *o) {
    const Tensor *t = c.tensor(o);
    if (!t || t->dim() != 2 || t->size(0) > INT32_MAX) {
        c.ok = false;
        return 0;
    }
    return t->size(0);
}

// quant_linear(x, w, w_scale, bias, x_scale, out_dtype, ws) -> y
PyObject *quant_linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 7) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        const ProductIn in(c, a[0], a[4]);
        if (!in.x) return none();
        const int64_t N = rows_of(c, a[1]);
        auto w = (const int8_t *)c.need(a[1], at::kChar, N, in.K);
        auto w_scale = (const float *)c.need(a[2], at::kFloat, N);
        auto bias = (const float *)c.opt(a[3], at::kFloat, N);
        int yt;
        const at::ScalarType os = c.dtype(a[5], &yt);
        if (!c.ok) return none();
        const c10::DeviceGuard guard(c.device);
        Tensor y = c.empty({in.M, N}, os);
        const Workspace ws(c, a[6], in.bytes());
        if (!c.ok || tw_quant_linear(in.x->data_ptr(), in.type, in.stride, in.scale, w, w_scale,
                                     bias, (int)in.M, (int)in.K, (int)N, y.data_ptr(), yt, ws.p,
                                     ws.bytes, c.stream(), nullptr) != TW_OK)
            return none();
        return wrapped(y);
    });
}

// quant_gateup(x, wg, g_scale, wu, u_scale, gamma, beta, eps, x_scale, out_dtype, ws) -> h
PyObject *quant_gateup(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 11) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        const ProductIn in(c, a[0], a[8]);
        if (!in.x) return none();
        const int64_t N = rows_of(c, a[1]);
        auto wg = (const int8_t *)c.need(a[1], at::kChar, N, in.K);
        auto gs = (const float *)c.need(a[2], at::kFloat, N);
        auto wu = (const int8_t *)c.need(a[3], at::kChar, N, in.K);
        auto us = (const float *)c.need(a[4], at::kFloat, N);
        auto gamma = (const float *)c.opt(a[5], at::kFloat, in.K);
        auto beta = (const float *)c.opt(a[6], at::kFloat, in.K);
        const float eps = c.real(a[7]);
        int ht;
        const at::ScalarType os = c.dtype(a[9], &ht);
        if (!c.ok) return none();
        const c10::DeviceGuard guard(c.device);
        Tensor h = c.empty({in.M, N}, os);
        const Workspace ws(c, a[10], in.bytes());
        if (!c.ok || tw_quant_gateup(in.x->data_ptr(), in.type, in.stride, in.scale, gamma, beta,
                                     eps, wg, gs, wu, us, (int)in.M, (int)in.K, (int)N,
                                     h.data_ptr(), ht, ws.p, ws.bytes, c.stream(),
                                     nullptr) != TW_OK)
            return none();
        return wrapped(h);
    });
}

// rmsnorm(x, gamma, eps, add, out_dtype) -> {y, sum, rstd}
PyObject *rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 5) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        int xt, at_, yt;
        int64_t stride;
        const Tensor *x = c.rows(a[0], false, &xt, &stride);
        if (!x) return none();
        const int64_t M = x->size(0), K = x->size(1);
        auto gamma = (const float *)c.need(a[1], at::kFloat, K);
        const float eps = c.real(a[2]);
        const void *add = c.opt_matrix(a[3], &at_, M, K);
        const at::ScalarType os = c.dtype(a[4], &yt);
        if (!c.ok) return none();
        const c10::DeviceGuard guard(c.device);
        Tensor y = c.empty({M, K}, os), sum, rstd = c.empty({M}, at::kFloat);
        if (a[3] != Py_None) sum = c.empty({M, K}, x->scalar_type());
        if (tw_rmsnorm_fwd(x->data_ptr(), xt, stride, add, at_, gamma, eps, (int)M, (int)K,
                           sum.defined() ? sum.data_ptr() : nullptr, y.data_ptr(), yt,
                           rstd.data_ptr<float>(), c.stream(), nullptr) != TW_OK)
            return none();
        return dict_of({{"y", y}, {"sum", sum}, {"rstd", rstd}});
    });
}

// rmsnorm_quantize(x, gamma, eps, add) -> {q, scale, sum}
PyObject *rmsnorm_quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 4) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        int xt, at_;
        int64_t stride;
        const Tensor *x = c.rows(a[0], false, &xt, &stride);
        if (!x) return none();
        const int64_t M = x->size(0), K = x->size(1);
        auto gamma = (const float *)c.need(a[1], at::kFloat, K);
        const float eps = c.real(a[2]);
        const void *add = c.opt_matrix(a[3], &at_, M, K);
        if (!c.ok) return none();
        const c10::DeviceGuard guard(c.device);
        Tensor q = c.empty({M, K}, at::kChar), scale = c.empty({M}, at::kFloat), sum;
        if (a[3] != Py_None) sum = c.empty({M, K}, x->scalar_type());
        if (tw_rmsnorm_quant(x->data_ptr(), xt, stride, add, at_, gamma, eps, (int)M, (int)K,
                             sum.defined() ? sum.data_ptr() : nullptr, q.data_ptr<int8_t>(),
                             scale.data_ptr<float>(), c.stream(), nullptr) != TW_OK)
            return none();
        return dict_of({{"q", q}, {"scale", scale}, {"sum", sum}});
    });
}

// rmsnorm_backward(dy, x, gamma, rstd, dres, dx_dtype) -> {dx, dgamma}
PyObject *rmsnorm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 6) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        int xt, dt, ot;
        int64_t stride;
        const Tensor *x = c.rows(a[1], false, &xt, &stride);
        if (!x) return none();
        const int64_t M = x->size(0), K = x->size(1);
        const void *dy = c.matrix(a[0], &dt, M, K);
        auto gamma = (const float *)c.need(a[2], at::kFloat, K);
        const void *rstd = c.need(a[3], at::kFloat, M);
        const at::ScalarType os = c.dtype(a[5], &ot);
        const void *dres = c.opt(a[4], os, M, K);
        if (!c.ok) return none();
        const c10::DeviceGuard guard(c.device);
        const size_t nws = tw_rmsnorm_bwd_workspace_bytes((int)M, (int)K);
        Tensor dx = c.empty({M, K}, os), dg = c.empty({K}, at::kFloat),
               ws = c.empty({(int64_t)nws}, at::kByte);
        const Aligned ra(a[3], rstd);
        if (tw_rmsnorm_bwd(dy, dt, x->data_ptr(), xt, stride, gamma, (const float *)ra.p, dres,
                           (int)M, (int)K, dx.data_ptr(), ot, dg.data_ptr<float>(), ws.data_ptr(),
                           nws, c.stream(), nullptr) != TW_OK)
            return none();
        return dict_of({{"dx", dx}, {"dgamma", dg}});
    });
}

// bf16 rows of the tile kernels.
const Tensor *bf16_rows(Call &c, PyObject *o, int64_t *stride) {
    int type;
    const Tensor *x = c.rows(o, false, &type, stride);
    if (x && type != TW_BF16) c.ok = false;
    return c.ok ? x : nullptr;
}

int act_of(Call &c, PyObject *o) {
    static const char *const names[] = {"relu", "silu", "gelu"};  // tw_act's order
    const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    for (int i = 0; s && i < 3; ++i)
        if (!std::strcmp(s, names[i])) return i;
    PyErr_Clear();
    c.ok = false;
    return 0;
}

// gated_ffn(x, wg_t, wu_t, wd, act, keep, out_dtype, ws) -> {y, g, u}
PyObject *gated_ffn(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 8) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        int64_t stride;
        const Tensor *x = bf16_rows(c, a[0], &stride);
        if (!x) return none();
        const int64_t M = x->size(0), K = x->size(1), N = rows_of(c, a[1]);
        auto wg = (const uint16_t *)c.need(a[1], at::kBFloat16, N, K);
        auto wu = (const uint16_t *)c.need(a[2], at::kBFloat16, N, K);
        auto wd = (const uint16_t *)c.need(a[3], at::kBFloat16, N, K);
        const int act = act_of(c, a[4]);
        const int keep = PyObject_IsTrue(a[5]);
        int yt;
        const at::ScalarType os = c.dtype(a[6], &yt);
        if (keep < 0) PyErr_Clear();
        if (!c.ok || keep < 0) return none();
        const c10::DeviceGuard guard(c.device);
        Tensor y = c.empty({M, K}, os), g, u;
        if (keep) {
            g = c.empty({M, N}, at::kBFloat16);
            u = c.empty({M, N}, at::kBFloat16);
        }
        const Workspace ws(c, a[7], tw_gated_ffn_workspace_bytes((int)M, (int)K, (int)N));
        if (!c.ok || tw_gated_ffn_fwd((const uint16_t *)x->data_ptr(), stride, wg, wu, wd, act,
                                      (int)M, (int)K, (int)N,
                                      keep ? (uint16_t *)g.data_ptr() : nullptr,
                                      keep ? (uint16_t *)u.data_ptr() : nullptr, y.data_ptr(), yt,
                                      ws.p, ws.bytes, c.stream(), nullptr) != TW_OK)
            return none();
        return dict_of({{"y", y}, {"g", g}, {"u", u}});
    });
}

// gated_ffn_backward(dy, x, wg_t, wu_t, wd, g, u, act, dx_dtype, dw_dtype, ws) ->
// {dx, dwg_t, dwu_t, dwd}
PyObject *gated_ffn_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 11) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        int64_t stride;
        const Tensor *x = bf16_rows(c, a[1], &stride);
        if (!x) return none();
        const int64_t M = x->size(0), K = x->size(1), N = rows_of(c, a[2]);
        auto dy = (const uint16_t *)c.need(a[0], at::kBFloat16, M, K);
        auto wg = (const uint16_t *)c.need(a[2], at::kBFloat16, N, K);
        auto wu = (const uint16_t *)c.need(a[3], at::kBFloat16, N, K);
        auto wd = (const uint16_t *)c.need(a[4], at::kBFloat16, N, K);
        auto g = (const uint16_t *)c.need(a[5], at::kBFloat16, M, N);
        auto u = (const uint16_t *)c.need(a[6], at::kBFloat16, M, N);
        const int act = act_of(c, a[7]);
        int xt, wt;
        const at::ScalarType xs = c.dtype(a[8], &xt), wts = c.dtype(a[9], &wt);
        if (!c.ok) return none();
        const c10::DeviceGuard guard(c.device);
        Tensor dx = c.empty({M, K}, xs), dwg = c.empty({N, K}, wts), dwu = c.empty({N, K}, wts),
               dwd = c.empty({N, K}, wts);
        const Workspace ws(c, a[10], tw_gated_ffn_bwd_workspace_bytes((int)M, (int)K, (int)N));
        if (!c.ok || tw_gated_ffn_bwd(dy, (const uint16_t *)x->data_ptr(), stride, wg, wu, wd, act,
                                      g, u, (int)M, (int)K, (int)N, dx.data_ptr(), xt,
                                      dwg.data_ptr(), dwu.data_ptr(), dwd.data_ptr(), wt, ws.p,
                                      ws.bytes, c.stream(), nullptr) != TW_OK)
            return none();
        return dict_of({{"dx", dx}, {"dwg_t", dwg}, {"dwu_t", dwu}, {"dwd", dwd}});
    });
}

// A row's targets: 32- or 64-bit integers.
const void *targets(Call &c, PyObject *o, int64_t M, int *type) {
    const Tensor *t = c.tensor(o);
    if (!t) return nullptr;
    *type = t->scalar_type() == at::kInt ? TW_INT32 : TW_INT64;
    return c.need(o, *type == TW_INT32 ? at::kInt : at::kLong, M);
}

// linear_ce(x, w, target, ws) -> {loss, lse}
PyObject *linear_ce(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 4) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        int64_t stride;
        const Tensor *x = bf16_rows(c, a[0], &stride);
        if (!x) return none();
        const int64_t M = x->size(0), K = x->size(1), V = rows_of(c, a[1]);
        auto w = (const uint16_t *)c.need(a[1], at::kBFloat16, V, K);
        int tt;
        const void *t = targets(c, a[2], M, &tt);
        if (!c.ok) return none();
        const c10::DeviceGuard guard(c.device);
        Tensor loss = c.empty({M}, at::kFloat), lse = c.empty({M}, at::kFloat);
        const Workspace ws(c, a[3], tw_linear_ce_workspace_bytes((int)M, (int)K, (int)V));
        if (!c.ok) return none();
        const Aligned ta(a[2], t);
        if (tw_linear_ce_fwd((const uint16_t *)x->data_ptr(), stride, w, ta.p, tt, (int)M, (int)K,
                             (int)V, loss.data_ptr<float>(), lse.data_ptr<float>(), ws.p, ws.bytes,
                             c.stream(), nullptr) != TW_OK)
            return none();
        return dict_of({{"loss", loss}, {"lse", lse}});
    });
}

// linear_ce_backward(dloss, x, w, target, lse, dx_dtype, dw_dtype, ws) -> {dx, dw}
PyObject *linear_ce_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 8) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        int64_t stride;
        const Tensor *x = bf16_rows(c, a[1], &stride);
        if (!x) return none();
        const int64_t M = x->size(0), K = x->size(1), V = rows_of(c, a[2]);
        const void *dloss = c.need(a[0], at::kFloat, M);
        auto w = (const uint16_t *)c.need(a[2], at::kBFloat16, V, K);
        int tt, xt, wt;
        const void *t = targets(c, a[3], M, &tt);
        const void *lse = c.need(a[4], at::kFloat, M);
        const at::ScalarType xs = c.dtype(a[5], &xt), wts = c.dtype(a[6], &wt);
        if (!c.ok) return none();
        const c10::DeviceGuard guard(c.device);
        Tensor dx = c.empty({M, K}, xs), dw = c.empty({V, K}, wts);
        const Workspace ws(c, a[7], tw_linear_ce_bwd_workspace_bytes((int)M, (int)K, (int)V));
        if (!c.ok) return none();
        const Aligned da(a[0], dloss), ta(a[3], t), la(a[4], lse);
        if (tw_linear_ce_bwd((const float *)da.p, (const uint16_t *)x->data_ptr(), stride, w, ta.p,
                             tt, (const float *)la.p, (int)M, (int)K, (int)V, dx.data_ptr(), xt,
                             dw.data_ptr(), wt, ws.p, ws.bytes, c.stream(), nullptr) != TW_OK)
            return none();
        return dict_of({{"dx", dx}, {"dw", dw}});
    });
}

// Tensors of a list or tuple: contiguous, of either floating type, on one device.
struct Buffers {
    std::vector<void *> p;
    std::vector<int64_t> n;
    std::vector<int> type;
    std::vector<const Tensor *> t;
    Buffers(Call &c, PyObject *o, bool first) {
        if (!PyList_Check(o) && !PyTuple_Check(o)) {
            c.ok = false;
            return;
        }
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(o);
        p.reserve(count);
        n.reserve(count);
        type.reserve(count);
        t.reserve(count);
        for (Py_ssize_t i = 0; i < count; ++i) {
            const Tensor *x = c.tensor(PySequence_Fast_GET_ITEM(o, i));
            int k;
            if (!x || !c.kind(x->scalar_type(), false, &k)) return;
            if (first && i == 0) c.device = x->device();
            if (x->device() != c.device || !x->is_cuda() || !x->is_contiguous()) {
                c.ok = false;
                return;
            }
            p.push_back(x->data_ptr());
            n.push_back(x->numel());
            type.push_back(k);
            t.push_back(x);
        }
        if (first && count == 0) c.ok = false;
    }
};

// clip_grads(grads, max_norm, eps, out or None) -> norm
PyObject *clip_grads(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 4) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        const Buffers g(c, a[0], true);
        if (!c.ok || g.t.size() > (1u << 20)) return none();
        const float most = c.real(a[1]), eps = c.real(a[2]);
        const Buffers o(c, a[3] == Py_None ? a[0] : a[3], false);
        if (!c.ok || o.t.size() != g.t.size()) return none();
        for (size_t i = 0; i < g.t.size(); ++i)
            if (g.t[i] != o.t[i] && g.t[i]->sizes() != o.t[i]->sizes()) return none();
        const c10::DeviceGuard guard(c.device);
        const int count = (int)g.t.size();
        const size_t nws = tw_grad_norm_workspace_bytes(count, g.n.data());
        Tensor norm = c.empty({}, at::kFloat), ws = c.empty({(int64_t)nws}, at::kByte);
        if (tw_grad_clip(count, g.p.data(), g.n.data(), g.type.data(), o.p.data(), o.type.data(),
                         most, eps, norm.data_ptr<float>(), ws.data_ptr(), nws, c.stream(),
                         nullptr) != TW_OK)
            return none();
        return wrapped(norm);
    });
}

#define TW_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TW_METHOD(layernorm), TW_METHOD(layernorm_backward),
                         TW_METHOD(quant_linear), TW_METHOD(quant_gateup),
                         TW_METHOD(rmsnorm), TW_METHOD(rmsnorm_quantize),
                         TW_METHOD(rmsnorm_backward), TW_METHOD(gated_ffn),
                         TW_METHOD(gated_ffn_backward), TW_METHOD(linear_ce),
                         TW_METHOD(linear_ce_backward), TW_METHOD(clip_grads),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_tw_calls", nullptr, -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tw_calls(void) { return PyModule_Create(&module_def); }
