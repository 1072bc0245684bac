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
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_front", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__front() { return PyModule_Create(&module); }
