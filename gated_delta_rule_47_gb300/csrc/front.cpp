// front.cpp -- the short way from Python into the layer operators.
//
// The smallest calls are bound by the host: checking, allocating and marshalling
// in Python took 7 to 10 us of a call whose kernel runs 2.4 (one token of one
// user, a norm of 8 rows).  Here the same is done on the tensors' C++ side, for
// calls in which all is well.  Whatever is not (a wrong type or shape, a call on
// another stream, workspaces or outputs of the caller's) gives NotImplemented,
// and binding.py takes the call the long way, with its checks and messages.
#include <Python.h>

#include <limits.h>

#include <algorithm>
#include <utility>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <ATen/ops/empty_strided.h>
#include <c10/core/impl/DeviceGuardImplInterface.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gdn.h"

namespace {

using at::IntArrayRef;
using at::Tensor;

// The library's entry points, by address: this module links none of it.
struct Api {
    decltype(&linattn_chunk_fwd_workspace_bytes) fwd_bytes;
    decltype(&linattn_chunk_fwd) fwd;
    decltype(&linattn_chunk_bwd_workspace_bytes) bwd_bytes;
    decltype(&linattn_chunk_bwd) bwd;
    decltype(&linattn_step) step;
    decltype(&gdn_step) delta;
    decltype(&rms_norm_fwd) norm;
    decltype(&rms_norm_bwd_workspace_bytes) norm_bytes;
    decltype(&rms_norm_bwd) norm_back;
    decltype(&state_pool_fork_workspace_bytes) fork_bytes;
    decltype(&state_pool_fork) fork;
    decltype(&state_pool_compact_workspace_bytes) compact_bytes;
    decltype(&state_pool_compact) compact;
    decltype(&causal_conv_fwd) conv;
    decltype(&causal_conv_bwd_workspace_bytes) conv_bytes;
    decltype(&causal_conv_bwd) conv_back;
    decltype(&causal_conv_step) conv_step;
    decltype(&ssm_scan_fwd_workspace_bytes) scan_bytes;
    decltype(&ssm_scan_fwd) scan;
    decltype(&ssm_scan_bwd_workspace_bytes) scan_back_bytes;
    decltype(&ssm_scan_bwd) scan_back;
    decltype(&ssm_step) scan_step;
    decltype(&gated_norm_fwd) gated;
    decltype(&gated_norm_bwd_workspace_bytes) gated_bytes;
    decltype(&gated_norm_bwd) gated_back;
    decltype(&block_norm_fwd) block;
    decltype(&block_norm_bwd_workspace_bytes) block_bytes;
    decltype(&block_norm_bwd) block_back;
} api;
PyObject *current_stream, *fail;  // torch's query, and binding.py's function that raises

struct Odd {};  // the call is for the long way

void need(bool ok) {
    if (!ok) throw Odd{};
}

const Tensor &tensor(PyObject *o) {
    need(THPVariable_Check(o));
    const Tensor &t = THPVariable_Unpack(o);
    need(t.is_cuda());
    return t;
}

// A tensor or None.
struct Maybe {
    const Tensor *t;
    explicit Maybe(PyObject *o) : t(o == Py_None ? nullptr : &tensor(o)) {}
    explicit operator bool() const { return t != nullptr; }
    template <typename T = void>
    T *ptr() const {
        return t ? static_cast<T *>(t->data_ptr()) : nullptr;
    }
};

// Sizes that the C interface takes as int.
void ints(IntArrayRef sizes) {
    for (int64_t n : sizes) need(n <= INT_MAX);
}

void dense(const Tensor &t, IntArrayRef shape, at::ScalarType type) {
    need(t.scalar_type() == type && t.sizes() == shape && t.is_contiguous());
}
void dense(const Maybe &m, IntArrayRef shape, at::ScalarType type) {
    if (m) dense(*m.t, shape, type);
}

int code(const Tensor &t) {
    need(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat);
    return t.scalar_type() == at::kBFloat16 ? GDN_BF16 : GDN_F32;
}

void *stream_of(const Tensor &t) {
    PyObject *index = PyLong_FromLong(t.device().index());
    PyObject *s = index ? PyObject_CallOneArg(current_stream, index) : nullptr;
    Py_XDECREF(index);
    void *p = s ? PyLong_AsVoidPtr(s) : nullptr;
    Py_XDECREF(s);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        throw Odd{};
    }
    return p;
}

double number(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        throw Odd{};
    }
    return x;
}

// A flag, by its truth as Python has it.
bool truth(PyObject *o) {
    const int yes = PyObject_IsTrue(o);
    if (yes < 0) {
        PyErr_Clear();
        throw Odd{};
    }
    return yes;
}

Tensor scratch(size_t bytes, const Tensor &like) {
    need(bytes != (size_t)-1);
    return bytes ? at::empty({(int64_t)bytes}, like.options().dtype(at::kByte)) : Tensor();
}
void *ptr(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

// A tensor for an answer, None for an undefined one.
PyObject *wrap(const Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject *pack(std::initializer_list<Tensor> ts) {
    PyObject *r = PyTuple_New(ts.size());
    Py_ssize_t i = 0;
    for (const Tensor &t : ts) {
        PyObject *x = r ? wrap(t) : nullptr;
        if (!x) {
            Py_XDECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, x);
    }
    return r;
}

// Runs f, which gives the answer; what binding.py reports or takes is left to it.
// An allocation that failed is torch's own error, as on the long way.
template <typename F>
PyObject *guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
    HANDLE_TH_ERRORS
    try {
        need(given == wanted);
        return f();
    } catch (const Odd &) {
        Py_RETURN_NOTIMPLEMENTED;
    }
    END_HANDLE_TH_ERRORS
}
bool good(const char *name, int status) {
    if (status == GDN_OK) return true;
    Py_XDECREF(PyObject_CallFunction(fail, "si", name, status));
    return false;
}

// step(q, k, v, beta, g, state, slots, state_out, scale, l2norm)
PyObject *step(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        const Tensor &q = tensor(x[0]), &k = tensor(x[1]), &v = tensor(x[2]), &g = tensor(x[4]), &s = tensor(x[5]);
        const Maybe beta(x[3]), slots(x[6]), to(x[7]);
        need(q.dim() == 3 && v.dim() == 3 && s.dim() == 4);
        const int64_t B = q.size(0), Hk = q.size(1), Dk = q.size(2), H = v.size(1), Dv = v.size(2), pages = s.size(0);
        const auto type = q.scalar_type();
        const int dt = code(q);
        dense(q, {B, Hk, Dk}, type);
        dense(k, {B, Hk, Dk}, type);
        dense(v, {B, H, Dv}, type);
        need(Hk > 0 && H % Hk == 0);
        ints({B, H, pages});
        const bool per_head = g.dim() == 1;
        if (per_head) dense(g, {H}, at::kFloat);
        else dense(g, {B, H}, at::kFloat);
        dense(s, {pages, H, Dk, Dv}, at::kFloat);
        dense(to, {pages, H, Dk, Dv}, at::kFloat);
        dense(slots, {B}, at::kInt);
        dense(beta, {B, H}, type);
        need(slots || B <= pages);
        const float scale = (float)number(x[8]);
        const unsigned flags = (per_head ? GDN_G_PER_HEAD : 0) | (truth(x[9]) ? GDN_QK_L2NORM : 0);
        Tensor o = at::empty_like(v);
        float *out = to ? to.ptr<float>() : s.data_ptr<float>();
        void *stream = stream_of(q);
        const int st =
            beta ? api.delta(q.data_ptr(), k.data_ptr(), v.data_ptr(), beta.ptr(), g.data_ptr<float>(), s.data_ptr<float>(),
                             out, slots.ptr<int>(), o.data_ptr(), B, H, Hk, Dk, Dv, pages, scale, flags, dt, stream)
                 : api.step(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr<float>(), s.data_ptr<float>(), out,
                            slots.ptr<int>(), o.data_ptr(), B, H, Hk, Dk, Dv, pages, scale, flags, dt, stream);
        return good(beta ? "gdn_step" : "linattn_step", st) ? wrap(o) : nullptr;
    });
}

// norm(x, weight, residual, eps, e4m3, group): (y, scales, h)
PyObject *norm(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject * {
        const Tensor &in = tensor(x[0]);
        const Maybe w(x[1]), res(x[2]);
        need(in.dim() > 0);
        const int64_t C = in.size(-1), group = (int64_t)number(x[5]), rows = C ? in.numel() / C : 0;
        const int dt = code(in);
        const bool e4m3 = truth(x[4]);
        ints({C});
        dense(in, in.sizes(), in.scalar_type());
        dense(res, in.sizes(), in.scalar_type());
        dense(w, {C}, at::kFloat);
        need(group == 0 || (e4m3 && (group == 32 || group == 64 || group == 128) && C % group == 0));
        Tensor y = e4m3 ? at::empty(in.sizes(), in.options().dtype(at::kFloat8_e4m3fn)) : at::empty_like(in), scales;
        if (e4m3) {
            c10::SmallVector<int64_t, 6> shape(in.sizes().begin(), in.sizes().end());
            shape.back() = group ? C / group : 1;
            scales = at::empty(shape, in.options().dtype(at::kFloat));
        }
        Tensor h = res ? at::empty_like(in) : in;
        const int st = api.norm(in.data_ptr(), res.ptr(), w.ptr<float>(), y.data_ptr(), static_cast<float *>(ptr(scales)),
                                res ? h.data_ptr() : nullptr, rows, C, group, (float)number(x[3]), e4m3, dt, stream_of(in));
        return good("rms_norm_fwd", st) ? pack({y, scales, h}) : nullptr;
    });
}

// norm_back(dy, h, weight, dresidual, eps): (dx, dw)
PyObject *norm_back(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject * {
        const Tensor &dy = tensor(x[0]), &h = tensor(x[1]);
        const Maybe w(x[2]), res(x[3]);
        need(h.dim() > 0);
        const int64_t C = h.size(-1), rows = C ? h.numel() / C : 0;
        const int dt = code(h);
        ints({C});
        dense(h, h.sizes(), h.scalar_type());
        dense(dy, h.sizes(), h.scalar_type());
        dense(res, h.sizes(), h.scalar_type());
        dense(w, {C}, at::kFloat);
        const size_t bytes = api.norm_bytes(rows, C);
        Tensor dx = at::empty_like(h), dw = at::empty({C}, h.options().dtype(at::kFloat)), ws = scratch(bytes, h);
        const int st = api.norm_back(dy.data_ptr(), h.data_ptr(), w.ptr<float>(), res.ptr(), dx.data_ptr(),
                                     dw.data_ptr<float>(), rows, C, (float)number(x[4]), dt, ptr(ws), bytes, stream_of(h));
        return good("rms_norm_bwd", st) ? pack({dx, dw}) : nullptr;
    });
}

struct Pool {
    int64_t layers, slots;
    size_t page;
    explicit Pool(const Tensor &t) {
        need(t.dim() >= 2 && t.is_contiguous() && t.numel() > 0);
        layers = t.size(0), slots = t.size(1), page = (size_t)t.stride(1) * t.element_size();
        need(page % 16 == 0);
        ints({layers, slots});
    }
};

// fork(pool, live, parents): children
PyObject *fork_(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject * {
        const Tensor &pool = tensor(x[0]), &live = tensor(x[1]), &parents = tensor(x[2]);
        const Pool p(pool);
        dense(live, {p.slots}, at::kByte);
        need(parents.dim() == 1);
        dense(parents, parents.sizes(), at::kInt);
        const size_t bytes = api.fork_bytes(p.slots, parents.numel());
        Tensor children = at::empty_like(parents), ws = scratch(bytes, pool);
        const int st = api.fork(pool.data_ptr(), p.layers, p.slots, p.page, live.data_ptr<uint8_t>(), parents.data_ptr<int>(),
                                children.data_ptr<int>(), parents.numel(), ptr(ws), bytes, stream_of(pool));
        return good("state_pool_fork", st) ? wrap(children) : nullptr;
    });
}

// compact(pool, live): (remap, n_live)
PyObject *compact(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 2, [&]() -> PyObject * {
        const Tensor &pool = tensor(x[0]), &live = tensor(x[1]);
        const Pool p(pool);
        dense(live, {p.slots}, at::kByte);
        const size_t bytes = api.compact_bytes(p.slots);
        const auto ints = pool.options().dtype(at::kInt);
        Tensor remap = at::empty({p.slots}, ints), count = at::empty({1}, ints), ws = scratch(bytes, pool);
        const int st = api.compact(pool.data_ptr(), p.layers, p.slots, p.page, live.data_ptr<uint8_t>(),
                                   remap.data_ptr<int>(), count.data_ptr<int>(), ptr(ws), bytes, stream_of(pool));
        return good("state_pool_compact", st) ? pack({remap, count}) : nullptr;
    });
}

// What linear attention's two directions share.
struct Prompt {
    int64_t B, Hk, T, Dk, H, Dv, seqs;
    int dt;
    unsigned flags;
    bool plain = true;  // everything contiguous
    Prompt(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &g, const Maybe &s0, const Maybe &cu, PyObject *simt) {
        need(q.dim() == 4 && v.dim() == 4);
        B = q.size(0), Hk = q.size(1), T = q.size(2), Dk = q.size(3), H = v.size(1), Dv = v.size(3), dt = code(q);
        strided(q, {B, Hk, T, Dk}, q.scalar_type());
        strided(k, {B, Hk, T, Dk}, q.scalar_type());
        strided(v, {B, H, T, Dv}, q.scalar_type());
        need(Hk > 0 && H % Hk == 0);
        ints({B, H, T});
        const bool per_head = g.dim() == 1;
        if (per_head) {
            dense(g, {H}, at::kFloat);
        } else {
            need(g.scalar_type() == at::kFloat && g.sizes() == IntArrayRef({B, H, T}));
            plain = plain && g.is_contiguous();
        }
        seqs = B;
        if (cu) {
            need(cu.t->dim() == 1 && cu.t->numel() >= 2 && B == 1);
            dense(cu, cu.t->sizes(), at::kInt);
            seqs = cu.t->numel() - 1;
        }
        dense(s0, {seqs, H, Dk, Dv}, at::kFloat);
        flags = (per_head ? GDN_G_PER_HEAD : 0) | (truth(simt) ? GDN_PATH_SIMT : 0);
    }
    // [..,D] with D contiguous, other strides multiples of 16 bytes and none of 0 over several elements
    void strided(const Tensor &t, IntArrayRef shape, at::ScalarType type) {
        need(t.scalar_type() == type && t.sizes() == shape);
        if (t.is_contiguous()) return;
        plain = false;
        need(t.stride(3) == 1);
        for (int i = 0; i < 3; ++i)
            need(t.size(i) <= 1 || (t.stride(i) > 0 && t.stride(i) * t.element_size() % 16 == 0));
    }
};
// No two elements in one place, as far as strides tell: each dimension steps by
// at least what those of smaller steps span.
void apart(const Tensor &t) {
    std::pair<int64_t, int64_t> by[4];  // step, elements
    int n = 0;
    for (int i = 0; i < t.dim(); ++i)
        if (t.size(i) > 1) by[n++] = {t.stride(i), t.size(i)};
    std::sort(by, by + n);
    int64_t span = 1;
    for (int i = 0; i < n; ++i) {
        need(by[i].first >= span);
        span += by[i].first * (by[i].second - 1);
    }
}
void steps(const Tensor &t, long long *out) {
    for (int i = 0; i < 3; ++i) out[i] = t.dim() > 1 && t.size(i) > 1 ? t.stride(i) : 0;
}

// fwd(q, k, v, g, initial_state, output_final_state, cu_seqlens, scale, simt): (o, final_state)
PyObject *fwd(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject * {
        const Tensor &q = tensor(x[0]), &k = tensor(x[1]), &v = tensor(x[2]), &g = tensor(x[3]);
        const Maybe s0(x[4]), cu(x[6]);
        const Prompt p(q, k, v, g, s0, cu, x[8]);
        const bool final_state = truth(x[5]);
        const size_t bytes = api.fwd_bytes(p.B, p.H, p.Hk, p.T, p.Dk, p.Dv, p.seqs, cu ? 1 : 0, p.flags, p.dt);
        Tensor o = at::empty_like(v), sf, ws = scratch(bytes, q);
        if (final_state) sf = at::empty({p.seqs, p.H, p.Dk, p.Dv}, g.options());
        long long st[15];
        const bool plain = p.plain && o.is_contiguous();
        if (!plain) steps(q, st), steps(k, st + 3), steps(v, st + 6), steps(o, st + 9), steps(g, st + 12);
        const int status = api.fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr<float>(), s0.ptr<float>(), o.data_ptr(),
                                   static_cast<float *>(ptr(sf)), cu.ptr<int>(), plain ? nullptr : st, p.seqs, p.B, p.H, p.Hk,
                                   p.T, p.Dk, p.Dv, (float)number(x[7]), p.flags, p.dt, ptr(ws), bytes, stream_of(q));
        return good("linattn_chunk_fwd", status) ? pack({o, sf}) : nullptr;
    });
}

// bwd(q, k, v, g, dout, initial_state, dfinal_state, cu_seqlens, scale, simt): (dq, dk, dv, dg, dinitial_state)
PyObject *bwd(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        const Tensor &q = tensor(x[0]), &k = tensor(x[1]), &v = tensor(x[2]), &g = tensor(x[3]), &go = tensor(x[4]);
        const Maybe s0(x[5]), dsf(x[6]), cu(x[7]);
        Prompt p(q, k, v, g, s0, cu, x[9]);
        p.strided(go, {p.B, p.H, p.T, p.Dv}, q.scalar_type());
        dense(dsf, {p.seqs, p.H, p.Dk, p.Dv}, at::kFloat);
        // gradients take their tensors' strides
        if (!p.plain) apart(q), apart(k), apart(v), apart(g);
        const size_t bytes = api.bwd_bytes(p.B, p.H, p.Hk, p.T, p.Dk, p.Dv, p.seqs, cu ? 1 : 0, p.flags, p.dt);
        auto like = [](const Tensor &t) { return at::empty_strided(t.sizes(), t.strides(), t.options()); };
        Tensor dq = like(q), dk = like(k), dv = like(v), dg = like(g), ds0, ws = scratch(bytes, q);
        if (s0) ds0 = at::empty_like(*s0.t);
        long long st[15];
        if (!p.plain) steps(q, st), steps(k, st + 3), steps(v, st + 6), steps(go, st + 9), steps(g, st + 12);
        const int status =
            api.bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr<float>(), s0.ptr<float>(), go.data_ptr(),
                    dsf.ptr<float>(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dg.data_ptr<float>(),
                    static_cast<float *>(ptr(ds0)), cu.ptr<int>(), p.plain ? nullptr : st, p.seqs, p.B, p.H, p.Hk, p.T, p.Dk,
                    p.Dv, (float)number(x[8]), p.flags, p.dt, ptr(ws), bytes, stream_of(q));
        return good("linattn_chunk_bwd", status) ? pack({dq, dk, dv, dg, ds0}) : nullptr;
    });
}

// ---- next to a mixer

// The tensors of a call lie on the current device.
void here(const Tensor &like, std::initializer_list<const Tensor *> others) {
    need(c10::impl::getDeviceGuardImpl(c10::DeviceType::CUDA)->getDevice() == like.device());
    for (const Tensor *t : others) need(!t || t->device() == like.device());
}

// [..,C] with C contiguous and other strides, as the C interface takes them.
void pitched(const Tensor &t, IntArrayRef shape, at::ScalarType type, long long *out) {
    need(t.scalar_type() == type && t.sizes() == shape && (t.numel() == 0 || t.stride(-1) == 1 || t.size(-1) == 1));
    for (int i = 0; i + 1 < t.dim(); ++i) {
        out[i] = t.size(i) > 1 ? t.stride(i) : 0;
        need(out[i] >= 0 && out[i] * t.element_size() % 16 == 0);
    }
}

struct Rows {
    int64_t B, T, C, seqs;
    Rows(const Tensor &x, const Maybe &cu) {
        need(x.dim() == 3);
        B = x.size(0), T = x.size(1), C = x.size(2), seqs = B;
        ints({B, T, C});
        if (cu) {
            need(cu.t->dim() == 1 && cu.t->numel() >= 2 && B == 1);
            dense(cu, cu.t->sizes(), at::kInt);
            seqs = cu.t->numel() - 1;
        }
    }
};
int64_t taps(const Tensor &w, const Maybe &bias, int64_t C) {
    need(w.dim() == 2);
    dense(w, {C, w.size(1)}, at::kFloat);
    dense(bias, {C}, at::kFloat);
    ints({w.size(1)});
    need(w.size(1) >= 2);
    return w.size(1);
}
Tensor fp32(const Maybe &like) { return like ? at::empty_like(*like.t) : Tensor(); }

// conv(x, weight, bias, initial_window, output_final_window, cu_seqlens, silu): (y, final_window)
PyObject *conv(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject * {
        const Tensor &in = tensor(x[0]), &w = tensor(x[1]);
        const Maybe bias(x[2]), win(x[3]), cu(x[5]);
        const Rows r(in, cu);
        const auto type = in.scalar_type();
        const int dt = code(in);
        const int64_t W = taps(w, bias, r.C);
        long long st[4];
        pitched(in, in.sizes(), type, st);
        dense(win, {r.seqs, W - 1, r.C}, type);
        here(in, {&w, bias.t, win.t, cu.t});
        const bool last = truth(x[4]);
        Tensor y = at::empty(in.sizes(), in.options()), out;
        if (last) out = at::empty({r.seqs, W - 1, r.C}, in.options());
        st[2] = r.T * r.C, st[3] = r.C;
        const int status = api.conv(in.data_ptr(), w.data_ptr<float>(), bias.ptr<float>(), win.ptr(), y.data_ptr(), ptr(out),
                                    cu.ptr<int>(), st, r.seqs, r.B, r.T, r.C, W, truth(x[6]) ? GDN_SILU : 0, dt, stream_of(in));
        return good("causal_conv_fwd", status) ? pack({y, out}) : nullptr;
    });
}

// conv_back(x, weight, dy, bias, initial_window, dfinal_window, cu_seqlens, silu): (dx, dweight, dbias, dinitial_window)
PyObject *conv_back(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject * {
        const Tensor &in = tensor(x[0]), &w = tensor(x[1]), &dy = tensor(x[2]);
        const Maybe bias(x[3]), win(x[4]), dlast(x[5]), cu(x[6]);
        const Rows r(in, cu);
        const auto type = in.scalar_type();
        const int dt = code(in);
        const int64_t W = taps(w, bias, r.C);
        long long st[4];
        pitched(in, in.sizes(), type, st);
        pitched(dy, in.sizes(), type, st + 2);
        dense(win, {r.seqs, W - 1, r.C}, type);
        dense(dlast, {r.seqs, W - 1, r.C}, type);
        here(in, {&w, &dy, bias.t, win.t, dlast.t, cu.t});
        const size_t bytes = api.conv_bytes(r.B, r.T, r.C, W);
        Tensor ws = scratch(bytes, in), dx = at::empty(in.sizes(), in.options()), dw = at::empty_like(w), db = fp32(bias), dwin = fp32(win);
        const int status = api.conv_back(in.data_ptr(), w.data_ptr<float>(), bias.ptr<float>(), dy.data_ptr(), win.ptr(), dlast.ptr(),
                                         dx.data_ptr(), dw.data_ptr<float>(), static_cast<float *>(ptr(db)), ptr(dwin), cu.ptr<int>(),
                                         st, r.seqs, r.B, r.T, r.C, W, truth(x[7]) ? GDN_SILU : 0, dt, ptr(ws), bytes, stream_of(in));
        return good("causal_conv_bwd", status) ? pack({dx, dw, db, dwin}) : nullptr;
    });
}

// A pool's pages of `shape`, and the rows' slots.
int64_t pages(const Tensor &pool, const Maybe &out, IntArrayRef shape, at::ScalarType type, const Maybe &slots, int64_t B) {
    need(pool.dim() == 3);
    const int64_t count = pool.size(0);
    dense(pool, {count, shape[0], shape[1]}, type);
    dense(out, pool.sizes(), type);
    if (out && out.ptr() != pool.data_ptr()) {  // in place, or apart
        const char *p = static_cast<const char *>(pool.data_ptr()), *q = static_cast<const char *>(out.ptr());
        const int64_t bytes = pool.numel() * pool.element_size();
        need(p + bytes <= q || q + bytes <= p);
    }
    dense(slots, {B}, at::kInt);
    need(slots || B <= count);
    ints({B, count});
    return count;
}

// conv_step(x, weight, window, bias, slots, window_out, silu): y
PyObject *conv_step(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject * {
        const Tensor &in = tensor(x[0]), &w = tensor(x[1]), &pool = tensor(x[2]);
        const Maybe bias(x[3]), slots(x[4]), out(x[5]);
        need(in.dim() == 2);
        const int64_t B = in.size(0), C = in.size(1), W = taps(w, bias, C);
        ints({B, C});
        const int dt = code(in);
        long long step;
        pitched(in, in.sizes(), in.scalar_type(), &step);
        const int64_t count = pages(pool, out, {W - 1, C}, in.scalar_type(), slots, B);
        here(in, {&w, &pool, bias.t, slots.t, out.t});
        Tensor y = at::empty(in.sizes(), in.options());
        const int status = api.conv_step(in.data_ptr(), w.data_ptr<float>(), bias.ptr<float>(), pool.data_ptr(),
                                         out ? out.ptr() : pool.data_ptr(), slots.ptr<int>(), y.data_ptr(), step, B, C, W, count,
                                         truth(x[6]) ? GDN_SILU : 0, dt, stream_of(in));
        return good("causal_conv_step", status) ? wrap(y) : nullptr;
    });
}

// What the scan's two directions share.
struct Scan : Rows {
    int64_t N;
    int dt;
    unsigned flags;
    long long st[12];
    Scan(const Tensor &x, const Tensor &d, const Tensor &A, const Tensor &Bt, const Tensor &Ct, const Maybe &skip, const Maybe &z,
         const Maybe &bias, const Maybe &s0, const Maybe &cu, PyObject *soft)
        : Rows(x, cu) {
        need(A.dim() == 2);
        N = A.size(1), dt = code(x);
        ints({N});
        const auto type = x.scalar_type();
        dense(A, {C, N}, at::kFloat);
        pitched(x, {B, T, C}, type, st);
        pitched(d, {B, T, C}, type, st + 2);
        pitched(Bt, {B, T, N}, type, st + 4);
        pitched(Ct, {B, T, N}, type, st + 6);
        pitched(z ? *z.t : x, {B, T, C}, type, st + 8);
        dense(skip, {C}, at::kFloat);
        dense(bias, {C}, at::kFloat);
        dense(s0, {seqs, C, N}, at::kFloat);
        here(x, {&d, &A, &Bt, &Ct, skip.t, z.t, bias.t, s0.t, cu.t});
        flags = truth(soft) ? GDN_DT_SOFTPLUS : 0;
    }
};

// scan(x, dt, A, B, C, D, z, dt_bias, initial_state, output_final_state, cu_seqlens, softplus): (y, final_state)
PyObject *scan(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject * {
        const Tensor &in = tensor(x[0]), &d = tensor(x[1]), &A = tensor(x[2]), &Bt = tensor(x[3]), &Ct = tensor(x[4]);
        const Maybe skip(x[5]), z(x[6]), bias(x[7]), s0(x[8]), cu(x[10]);
        Scan p(in, d, A, Bt, Ct, skip, z, bias, s0, cu, x[11]);
        const bool last = truth(x[9]);
        const size_t bytes = api.scan_bytes(p.B, p.T, p.C, p.N, p.dt);
        Tensor ws = scratch(bytes, in), y = at::empty(in.sizes(), in.options()), sf;
        if (last) sf = at::empty({p.seqs, p.C, p.N}, A.options());
        p.st[10] = p.T * p.C, p.st[11] = p.C;
        const int status = api.scan(in.data_ptr(), d.data_ptr(), A.data_ptr<float>(), Bt.data_ptr(), Ct.data_ptr(), skip.ptr<float>(),
                                    z.ptr(), bias.ptr<float>(), s0.ptr<float>(), y.data_ptr(), static_cast<float *>(ptr(sf)),
                                    cu.ptr<int>(), p.st, p.seqs, p.B, p.T, p.C, p.N, p.flags, p.dt, ptr(ws), bytes, stream_of(in));
        return good("ssm_scan_fwd", status) ? pack({y, sf}) : nullptr;
    });
}

// scan_back(x, dt, A, B, C, dy, D, z, dt_bias, initial_state, dfinal_state, cu_seqlens, softplus):
// (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dinitial_state)
PyObject *scan_back(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject * {
        const Tensor &in = tensor(x[0]), &d = tensor(x[1]), &A = tensor(x[2]), &Bt = tensor(x[3]), &Ct = tensor(x[4]), &dy = tensor(x[5]);
        const Maybe skip(x[6]), z(x[7]), bias(x[8]), s0(x[9]), dsf(x[10]), cu(x[11]);
        Scan p(in, d, A, Bt, Ct, skip, z, bias, s0, cu, x[12]);
        pitched(dy, in.sizes(), in.scalar_type(), p.st + 10);
        dense(dsf, {p.seqs, p.C, p.N}, at::kFloat);
        here(in, {&dy, dsf.t});
        const size_t bytes = api.scan_back_bytes(p.B, p.T, p.C, p.N, p.dt);
        auto rows = [&](int64_t width) { return at::empty({p.B, p.T, width}, in.options()); };
        Tensor ws = scratch(bytes, in), dx = rows(p.C), dd = rows(p.C), dB = rows(p.N), dC = rows(p.N), dz, dA = at::empty_like(A);
        Tensor dskip = fp32(skip), dbias = fp32(bias), ds0 = fp32(s0);
        if (z) dz = rows(p.C);
        auto f = [](const Tensor &t) { return static_cast<float *>(ptr(t)); };
        const int status = api.scan_back(in.data_ptr(), d.data_ptr(), A.data_ptr<float>(), Bt.data_ptr(), Ct.data_ptr(),
                                         skip.ptr<float>(), z.ptr(), bias.ptr<float>(), s0.ptr<float>(), dy.data_ptr(),
                                         dsf.ptr<float>(), dx.data_ptr(), dd.data_ptr(), f(dA), dB.data_ptr(), dC.data_ptr(), f(dskip),
                                         ptr(dz), f(dbias), f(ds0), cu.ptr<int>(), p.st, p.seqs, p.B, p.T, p.C, p.N, p.flags, p.dt,
                                         ptr(ws), bytes, stream_of(in));
        return good("ssm_scan_bwd", status) ? pack({dx, dd, dA, dB, dC, dskip, dz, dbias, ds0}) : nullptr;
    });
}

// scan_step(x, dt, A, B, C, state, D, z, dt_bias, slots, state_out, softplus): y
PyObject *scan_step(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject * {
        const Tensor &in = tensor(x[0]), &d = tensor(x[1]), &A = tensor(x[2]), &Bt = tensor(x[3]), &Ct = tensor(x[4]), &pool = tensor(x[5]);
        const Maybe skip(x[6]), z(x[7]), bias(x[8]), slots(x[9]), out(x[10]);
        need(in.dim() == 2 && A.dim() == 2);
        const int64_t B = in.size(0), C = in.size(1), N = A.size(1);
        ints({B, C, N});
        const auto type = in.scalar_type();
        const int dt = code(in);
        dense(A, {C, N}, at::kFloat);
        long long st[5];
        pitched(in, {B, C}, type, st);
        pitched(d, {B, C}, type, st + 1);
        pitched(Bt, {B, N}, type, st + 2);
        pitched(Ct, {B, N}, type, st + 3);
        pitched(z ? *z.t : in, {B, C}, type, st + 4);
        dense(skip, {C}, at::kFloat);
        dense(bias, {C}, at::kFloat);
        const int64_t count = pages(pool, out, {C, N}, at::kFloat, slots, B);
        here(in, {&d, &A, &Bt, &Ct, &pool, skip.t, z.t, bias.t, slots.t, out.t});
        Tensor y = at::empty(in.sizes(), in.options());
        const int status = api.scan_step(in.data_ptr(), d.data_ptr(), A.data_ptr<float>(), Bt.data_ptr(), Ct.data_ptr(),
                                         skip.ptr<float>(), z.ptr(), bias.ptr<float>(), pool.data_ptr<float>(),
                                         out ? out.ptr<float>() : pool.data_ptr<float>(), slots.ptr<int>(), y.data_ptr(), st, B, C, N,
                                         count, truth(x[11]) ? GDN_DT_SOFTPLUS : 0, dt, stream_of(in));
        return good("ssm_step", status) ? wrap(y) : nullptr;
    });
}

// What the gated norm's two directions share.
struct Gated {
    int64_t B, T, H, D;
    int dt;
    unsigned flags;
    long long st[12];
    Gated(const Tensor &x, const Tensor &gate, const Maybe &w, PyObject *first, PyObject *sigmoid) {
        need(x.dim() == 4);
        B = x.size(0), T = x.size(1), H = x.size(2), D = x.size(3), dt = code(x);
        ints({B, T, H, D});
        pitched(x, x.sizes(), x.scalar_type(), st);
        pitched(gate, x.sizes(), x.scalar_type(), st + 3);
        const bool shared = !w || w.t->dim() == 1;
        if (shared) dense(w, {D}, at::kFloat);
        else dense(w, {H, D}, at::kFloat);
        flags = (truth(first) ? GDN_GATE_FIRST : 0) | (truth(sigmoid) ? GDN_GATE_SIGMOID : 0) | (shared ? GDN_W_SHARED : 0);
    }
};

// gated(x, gate, weight, eps, gate_first, sigmoid): y
PyObject *gated(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject * {
        const Tensor &in = tensor(x[0]), &gate = tensor(x[1]);
        const Maybe w(x[2]);
        const Gated p(in, gate, w, x[4], x[5]);
        here(in, {&gate, w.t});
        Tensor y = at::empty(in.sizes(), in.options());
        const int status = api.gated(in.data_ptr(), gate.data_ptr(), w.ptr<float>(), y.data_ptr(), p.st, p.B, p.T, p.H, p.D,
                                     (float)number(x[3]), p.flags, p.dt, stream_of(in));
        return good("gated_norm_fwd", status) ? wrap(y) : nullptr;
    });
}

// gated_back(dy, x, gate, weight, eps, gate_first, sigmoid): (dx, dgate, dweight)
PyObject *gated_back(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject * {
        const Tensor &dy = tensor(x[0]), &in = tensor(x[1]), &gate = tensor(x[2]);
        const Maybe w(x[3]);
        Gated p(in, gate, w, x[5], x[6]);
        pitched(dy, in.sizes(), in.scalar_type(), p.st + 6);
        here(in, {&dy, &gate, w.t});
        apart(in);  // dx takes its strides
        const size_t bytes = api.gated_bytes(p.B, p.T, p.H, p.D, p.flags);
        Tensor ws = scratch(bytes, in), dx = at::empty_like(in), dg = at::empty(in.sizes(), in.options());
        Tensor dw = p.flags & GDN_W_SHARED ? at::empty({p.D}, in.options().dtype(at::kFloat))
                                           : at::empty({p.H, p.D}, in.options().dtype(at::kFloat));
        pitched(dx, in.sizes(), in.scalar_type(), p.st + 9);
        const int status = api.gated_back(dy.data_ptr(), in.data_ptr(), gate.data_ptr(), w.ptr<float>(), dx.data_ptr(), dg.data_ptr(),
                                          dw.data_ptr<float>(), p.st, p.B, p.T, p.H, p.D, (float)number(x[4]), p.flags, p.dt, ptr(ws),
                                          bytes, stream_of(in));
        return good("gated_norm_bwd", status) ? pack({dx, dg, dw}) : nullptr;
    });
}

// What the block norm's two directions share.
struct Block {
    int64_t C, rows, groups = 0;
    int dt;
    Block(const Tensor &x, const Maybe &w1, const Maybe &s, const Maybe &w2) {
        need(x.dim() > 0);
        C = x.size(-1), rows = C ? x.numel() / C : 0, dt = code(x);
        ints({C});
        dense(x, x.sizes(), x.scalar_type());
        dense(w1, {C}, at::kFloat);
        dense(w2, {C}, at::kFloat);
        if (s) {
            need(s.t->dim() == 1 || s.t->dim() == 2);
            groups = s.t->dim() == 1 ? 1 : s.t->size(0);
            if (s.t->dim() == 1) dense(s, {C}, at::kFloat);
            else dense(s, {groups, C}, at::kFloat);
            ints({groups});
            need(groups > 0 && rows % groups == 0);
        }
    }
};

// block(x, residual, post_weight, scale, weight, eps): (y, h)
PyObject *block(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject * {
        const Tensor &in = tensor(x[0]), &res = tensor(x[1]);
        const Maybe w1(x[2]), s(x[3]), w2(x[4]);
        const Block p(in, w1, s, w2);
        dense(res, in.sizes(), in.scalar_type());
        here(in, {&res, w1.t, s.t, w2.t});
        Tensor y = at::empty_like(in), h = at::empty_like(in);
        const int status = api.block(in.data_ptr(), res.data_ptr(), w1.ptr<float>(), s.ptr<float>(), w2.ptr<float>(), y.data_ptr(),
                                     h.data_ptr(), p.rows, p.C, p.groups, (float)number(x[5]), p.dt, stream_of(in));
        return good("block_norm_fwd", status) ? pack({y, h}) : nullptr;
    });
}

// block_back(dy, dh, x, h, post_weight, scale, weight, eps): (dx, dresidual, dpost_weight, dscale, dweight)
PyObject *block_back(PyObject *, PyObject *const *x, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject * {
        const Tensor &dy = tensor(x[0]), &in = tensor(x[2]), &h = tensor(x[3]);
        const Maybe dh(x[1]), w1(x[4]), s(x[5]), w2(x[6]);
        const Block p(in, w1, s, w2);
        dense(dy, in.sizes(), in.scalar_type());
        dense(h, in.sizes(), in.scalar_type());
        dense(dh, in.sizes(), in.scalar_type());
        here(in, {&dy, &h, dh.t, w1.t, s.t, w2.t});
        const size_t bytes = api.block_bytes(p.rows, p.C, p.groups);
        Tensor ws = scratch(bytes, in), dx = at::empty_like(in), dres = at::empty_like(in), dw1 = fp32(w1), ds = fp32(s), dw2 = fp32(w2);
        auto f = [](const Tensor &t) { return static_cast<float *>(ptr(t)); };
        const int status = api.block_back(dy.data_ptr(), dh.ptr(), in.data_ptr(), h.data_ptr(), w1.ptr<float>(), s.ptr<float>(),
                                          w2.ptr<float>(), dx.data_ptr(), dres.data_ptr(), f(dw1), f(ds), f(dw2), p.rows, p.C, p.groups,
                                          (float)number(x[7]), p.dt, ptr(ws), bytes, stream_of(in));
        return good("block_norm_bwd", status) ? pack({dx, dres, dw1, ds, dw2}) : nullptr;
    });
}

// init(addresses of the entry points in Api's order, current stream's query, raise)
PyObject *init(PyObject *, PyObject *args) {
    PyObject *at_;
    if (!PyArg_ParseTuple(args, "O!OO", &PyTuple_Type, &at_, &current_stream, &fail)) return nullptr;
    constexpr Py_ssize_t count = sizeof(Api) / sizeof(void *);
    if (PyTuple_GET_SIZE(at_) != count) {
        PyErr_SetString(PyExc_ValueError, "not as many entry points as there are places");
        return nullptr;
    }
    void **to = reinterpret_cast<void **>(&api);
    for (Py_ssize_t i = 0; i < count; ++i)
        if (!(to[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(at_, i)))) return nullptr;
    Py_INCREF(current_stream);
    Py_INCREF(fail);
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f));
}

PyMethodDef methods[] = {{"init", init, METH_VARARGS, nullptr},
                         {"step", fast(step), METH_FASTCALL, nullptr},
                         {"norm", fast(norm), METH_FASTCALL, nullptr},
                         {"norm_back", fast(norm_back), METH_FASTCALL, nullptr},
                         {"fork", fast(fork_), METH_FASTCALL, nullptr},
                         {"compact", fast(compact), METH_FASTCALL, nullptr},
                         {"fwd", fast(fwd), METH_FASTCALL, nullptr},
                         {"bwd", fast(bwd), METH_FASTCALL, nullptr},
                         {"conv", fast(conv), METH_FASTCALL, nullptr},
                         {"conv_back", fast(conv_back), METH_FASTCALL, nullptr},
                         {"conv_step", fast(conv_step), METH_FASTCALL, nullptr},
                         {"scan", fast(scan), METH_FASTCALL, nullptr},
                         {"scan_back", fast(scan_back), METH_FASTCALL, nullptr},
                         {"scan_step", fast(scan_step), METH_FASTCALL, nullptr},
                         {"gated", fast(gated), METH_FASTCALL, nullptr},
                         {"gated_back", fast(gated_back), METH_FASTCALL, nullptr},
                         {"block", fast(block), METH_FASTCALL, nullptr},
                         {"block_back", fast(block_back), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_front", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__front() { return PyModule_Create(&module); }
