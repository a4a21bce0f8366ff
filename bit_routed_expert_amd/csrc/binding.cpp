// The tensor side of ops.py: a CPython module whose functions check the
// tensors of a call and hand their addresses to libstrata_moe.so.
//
// A small call is bound by the host.  A launch takes 3.3 us of it; the same
// checks through the tensors' Python methods took another 2.5 to 5 us (combine
// of one token 6.8 us a call, a norm 8.5 us), here they take under 0.5.
//
// The library's functions are reached by address (bind), so nothing is linked
// but libtorch; the module's only state are those addresses and ops.py's
// helpers: what raises, what runs a call on another device, and what gives the
// current device and stream.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include "strata_train.h"

namespace {

enum Fn {
    SORT, DISPATCH, DISPATCH_BACK, COMBINE, COMBINE_BACK, PRODUCT, DGRAD, WGRAD, NORM, NORM_BACK,
    BALANCE, BALANCE_BACK, EMBED, EMBED_BACK, VOCAB, VOCAB_BACK, ORTH, FNS
};
void *g_fn[FNS];         // the library's functions
PyObject *g_self[FNS];   // this module's, for a call that has to move to another device
PyObject *g_raise, *g_elsewhere, *g_device, *g_first_device, *g_stream;

constexpr auto BF16 = at::ScalarType::BFloat16, F32 = at::ScalarType::Float, I32 = at::ScalarType::Int;

// a*b*c elements; -1 (no tensor has that many) past 63 bits.
int64_t count(int64_t a, int64_t b, int64_t c = 1) {
    const __int128 n = (__int128)a * b * c;
    return n > INT64_MAX ? -1 : (int64_t)n;
}

// One call: its arguments (the last is the stream), the device of its tensors,
// and whether a check has failed (the Python error is set then, and later
// checks do nothing).
struct Call {
    Fn fn;
    PyObject *const *a;
    const char *const *names;
    Py_ssize_t n;
    int64_t dev = -2;   // -2: no tensor among the arguments
    bool ok = true;

    void bad(const char *format, ...) {
        if (!ok) return;
        ok = false;
        va_list v;
        va_start(v, format);
        PyObject *m = PyUnicode_FromFormatV(format, v);
        va_end(v);
        if (!m) return;
        Py_XDECREF(PyObject_CallOneArg(g_raise, m));   // raises
        Py_DECREF(m);
    }
    const at::Tensor *tensor(Py_ssize_t i) const {
        PyObject *o = a[i];
        if (o == Py_None || PyLong_CheckExact(o) || !THPVariable_Check(o)) return nullptr;
        return &THPVariable_Unpack(o);
    }
    // The first tensor's device; every tensor of the call has to be on it.
    void device() {
        for (Py_ssize_t i = 0; i + 1 < n && dev < 0; ++i)
            if (const at::Tensor *t = tensor(i)) {
                if (!t->is_cuda()) return bad("%s is not in device memory", names[i]);
                dev = t->get_device();
            }
    }
    long long integer(int i) {
        if (!ok) return 0;
        const long long v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) ok = false;
        return v;
    }
    int32_t size(int i) {   // what a C int32 holds, and no less than 0
        const long long v = integer(i);
        if (v < 0 || v > INT32_MAX) bad("%s is negative or does not fit 32 bits", names[i]);
        return (int32_t)v;
    }
    int64_t bytes(int i) {
        const long long v = integer(i);
        if (v < 0) bad("%s is negative", names[i]);
        return v;
    }
    float number(int i) {
        if (!ok) return 0.f;
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) ok = false;
        return (float)v;
    }
    strata_xdtype code(long long c, const char *name) {
        if (c != STRATA_X_BF16 && c != STRATA_X_F32) bad("%s is not X_BF16 or X_F32", name);
        return (strata_xdtype)c;
    }
    strata_xdtype code(int i) {
        const long long c = integer(i);
        return code(c, names[i]);
    }
    // The address that stands for a tensor (None: null).
    void *address(int i) {
        if (a[i] == Py_None) return nullptr;
        if (!PyLong_Check(a[i])) {
            bad("%s is neither a tensor nor an address", names[i]);
            return nullptr;
        }
        void *p = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(a[i]);
        if (PyErr_Occurred()) ok = false;
        return p;
    }
    bool here(const at::Tensor *t, int i) {
        if (!t->is_cuda()) bad("%s is not in device memory", names[i]);
        else if (t->get_device() != dev) bad("%s is on device %d, not %d", names[i], (int)t->get_device(), (int)dev);
        return ok;
    }
    // Address of a contiguous tensor of `want` elements; None and addresses pass.
    template <typename T = void> T *ptr(int i, at::ScalarType type, int64_t want) {
        if (!ok) return nullptr;
        const at::Tensor *t = tensor(i);
        if (!t) return (T *)address(i);
        if (!here(t, i)) return nullptr;
        if (t->scalar_type() != type)
            bad("%s holds %s, not %s", names[i], c10::toString(t->scalar_type()), c10::toString(type));
        else if (t->numel() != want)
            bad("%s has %lld elements, not %lld", names[i], (long long)t->numel(), (long long)want);
        else if (!t->is_contiguous()) bad("%s is not contiguous", names[i]);
        return ok ? (T *)t->data_ptr() : nullptr;
    }
    // The same of truth values or bytes.
    uint8_t *truths(int i, int64_t want) {
        const at::Tensor *t = ok ? tensor(i) : nullptr;
        return ptr<uint8_t>(i, t && t->scalar_type() == at::ScalarType::Byte ? at::ScalarType::Byte : at::ScalarType::Bool, want);
    }
    void *rows(int i, strata_xdtype c, int64_t want) { return ptr(i, c == STRATA_X_BF16 ? BF16 : F32, want); }
    // Address of a workspace said to hold `need` bytes.
    void *workspace(int i, int64_t need) {
        if (!ok) return nullptr;
        const at::Tensor *t = tensor(i);
        if (!t) return address(i);
        if (!here(t, i)) return nullptr;
        if ((int64_t)t->nbytes() < need || !t->is_contiguous()) bad("%s is smaller than ws_bytes", names[i]);
        return ok ? t->data_ptr() : nullptr;
    }

    // f(function, stream) with the tensors' device current, on its current
    // stream unless one is given; a status that is not OK raises.
    template <typename F> PyObject *run(F f) {
        if (!ok) return nullptr;
        PyObject *d = PyObject_CallNoArgs(dev >= 0 ? g_device : g_first_device);
        if (!d) return nullptr;
        const long long current = PyLong_AsLongLong(d);
        if (dev >= 0 && dev != current) {
            Py_DECREF(d);
            return elsewhere();
        }
        PyObject *s = a[n - 1], *own = nullptr;
        if (s == Py_None) own = s = PyObject_CallOneArg(g_stream, d);
        else if (!PyLong_Check(s)) own = s = stream_on(s, current);
        Py_DECREF(d);
        if (!s) return nullptr;
        void *stream = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(s);
        Py_XDECREF(own);
        if (PyErr_Occurred()) return nullptr;
        strata_status st;
        Py_BEGIN_ALLOW_THREADS;
        st = f(g_fn[fn], stream);
        Py_END_ALLOW_THREADS;
        if (st == STRATA_OK) Py_RETURN_NONE;
        PyObject *c = PyLong_FromLong(st);
        if (!c) return nullptr;
        PyObject *r = PyObject_CallOneArg(g_raise, c);
        Py_DECREF(c);
        return r;
    }
    // A stream object's address; one of another device would run the kernels there, on memory of this one.
    PyObject *stream_on(PyObject *s, long long current) {
        PyObject *d = PyObject_GetAttrString(s, "device_index");
        if (!d) {
            if (!PyErr_ExceptionMatches(PyExc_AttributeError)) return nullptr;
            PyErr_Clear();   // not torch's: its address is all there is to know
        } else {
            const long long on = PyLong_AsLongLong(d);
            Py_DECREF(d);
            if (PyErr_Occurred()) return nullptr;
            if (on != current) {
                bad("stream is on device %lld, not %lld", on, current);
                return nullptr;
            }
        }
        return PyObject_GetAttrString(s, "cuda_stream");
    }
    // The same call once more with the tensors' device current.
    PyObject *elsewhere() {
        PyObject *args = PyTuple_New(n + 2), *d = PyLong_FromLongLong(dev);
        if (!args || !d) {
            Py_XDECREF(args);
            Py_XDECREF(d);
            return nullptr;
        }
        PyTuple_SET_ITEM(args, 0, d);
        Py_INCREF(g_self[fn]);
        PyTuple_SET_ITEM(args, 1, g_self[fn]);
        for (Py_ssize_t i = 0; i < n; ++i) {
            Py_INCREF(a[i]);
            PyTuple_SET_ITEM(args, i + 2, a[i]);
        }
        PyObject *r = PyObject_CallObject(g_elsewhere, args);
        Py_DECREF(args);
        return r;
    }
};

// A function of the module: as many arguments as names, and no C++ exception
// past this point.
template <size_t N, typename Body>
PyObject *entry(Fn fn, PyObject *const *a, Py_ssize_t n, const char *const (&names)[N], Body body) {
    if (n != (Py_ssize_t)N || !g_fn[fn]) {
        PyErr_SetString(PyExc_TypeError, g_fn[fn] ? "wrong number of arguments" : "the library is not bound");
        return nullptr;
    }
    try {
        Call c{fn, a, names, n};
        c.device();
        return body(c);
    } catch (const std::exception &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

#define ARGS PyObject *, PyObject *const *args, Py_ssize_t nargs
// f as the library's function of that type
#define AS(FUNCTION) ((decltype(&FUNCTION))f)

PyObject *sort_picks(ARGS) {
    static const char *const names[] = {"idx",  "T",   "k",  "n_experts", "counts", "offsets",
                                        "perm", "pos", "ws", "ws_bytes",  "stream"};
    return entry(SORT, args, nargs, names, [](Call &c) {
        const int32_t T = c.size(1), k = c.size(2), E = c.size(3);
        const int64_t wb = c.bytes(9), picks = count(T, k);
        const auto idx = c.ptr<int32_t>(0, I32, picks), counts = c.ptr<int32_t>(4, I32, E);
        const auto offsets = c.ptr<int32_t>(5, I32, (int64_t)E + 1), perm = c.ptr<int32_t>(6, I32, picks);
        const auto pos = c.ptr<int32_t>(7, I32, picks);
        void *const ws = c.workspace(8, wb);
        return c.run([=](void *f, void *stream) {
            return AS(strata_moe_sort)(idx, T, k, E, counts, offsets, perm, pos, ws, (size_t)wb, stream);
        });
    });
}

PyObject *dispatch(ARGS) {
    static const char *const names[] = {"x", "xdtype", "T", "k", "d", "pos", "xs", "rows", "stream"};
    return entry(DISPATCH, args, nargs, names, [](Call &c) {
        const auto xt = c.code(1);
        const int32_t T = c.size(2), k = c.size(3), d = c.size(4), rows = c.size(7);
        const void *const x = c.rows(0, xt, count(T, d));
        const auto pos = c.ptr<int32_t>(5, I32, count(T, k));
        void *const xs = c.rows(6, xt, count(rows, d));
        return c.run([=](void *f, void *stream) {
            return AS(strata_moe_dispatch)(x, xt, T, k, d, pos, xs, rows, stream);
        });
    });
}

PyObject *dispatch_backward(ARGS) {
    static const char *const names[] = {"dxs", "xdtype", "rows", "pos", "T", "k", "d", "dx", "stream"};
    return entry(DISPATCH_BACK, args, nargs, names, [](Call &c) {
        const auto xt = c.code(1);
        const int32_t rows = c.size(2), T = c.size(4), k = c.size(5), d = c.size(6);
        const void *const dxs = c.rows(0, xt, count(rows, d));
        const auto pos = c.ptr<int32_t>(3, I32, count(T, k));
        void *const dx = c.rows(7, xt, count(T, d));
        return c.run([=](void *f, void *stream) {
            return AS(strata_moe_dispatch_backward)(dxs, xt, rows, pos, T, k, d, dx, stream);
        });
    });
}

PyObject *combine(ARGS) {
    static const char *const names[] = {"ys", "ydtype", "rows", "pos",    "w",    "T",
                                        "k",  "d",      "out",  "odtype", "base", "stream"};
    return entry(COMBINE, args, nargs, names, [](Call &c) {
        const auto yt = c.code(1), ot = c.code(9);
        const int32_t rows = c.size(2), T = c.size(5), k = c.size(6), d = c.size(7);
        const void *const ys = c.rows(0, yt, count(rows, d));
        const auto pos = c.ptr<int32_t>(3, I32, count(T, k));
        const auto w = c.ptr<float>(4, F32, count(T, k));
        void *const out = c.rows(8, ot, count(T, d));
        const void *const base = c.rows(10, ot, count(T, d));
        return c.run([=](void *f, void *stream) {
            return AS(strata_moe_combine)(ys, yt, rows, pos, w, T, k, d, base, out, ot, stream);
        });
    });
}

PyObject *combine_backward(ARGS) {
    static const char *const names[] = {"dout", "odtype", "ys", "ydtype", "rows", "pos", "w",
                                        "T",    "k",      "d",  "dys",    "dw",   "dz",  "stream"};
    return entry(COMBINE_BACK, args, nargs, names, [](Call &c) {
        const auto ot = c.code(1), yt = c.code(3);
        const int32_t rows = c.size(4), T = c.size(7), k = c.size(8), d = c.size(9);
        const int64_t picks = count(T, k);
        const void *const dout = c.rows(0, ot, count(T, d)), *const ys = c.rows(2, yt, count(rows, d));
        const auto pos = c.ptr<int32_t>(5, I32, picks);
        const auto w = c.ptr<float>(6, F32, picks);
        void *const dys = c.rows(10, yt, count(rows, d));
        const auto dw = c.ptr<float>(11, F32, picks), dz = c.ptr<float>(12, F32, picks);
        return c.run([=](void *f, void *stream) {
            return AS(strata_moe_combine_backward)(dout, ot, ys, yt, rows, pos, w, T, k, d, dys, dw, dz, stream);
        });
    });
}

// The three products: rows of A and B, the experts' row offsets, and the
// output, of which elements each has (0: rows of N, 1: rows of K, 2: matrices).
PyObject *grouped(Fn fn, PyObject *const *args, Py_ssize_t nargs, const char *const (&names)[12], int A, int B, int out) {
    return entry(fn, args, nargs, names, [=](Call &c) {
        const int32_t rows = c.size(3), E = c.size(4), N = c.size(5), K = c.size(6);
        const int64_t n[3] = {count(rows, N), count(rows, K), count(E, N, K)};
        const auto t = c.code(8);
        const int64_t wb = c.bytes(10);
        const void *const a = c.ptr(0, BF16, n[A]), *const b = c.ptr(1, BF16, n[B]);
        const auto offsets = c.ptr<int32_t>(2, I32, (int64_t)E + 1);
        void *const o = c.rows(7, t, n[out]), *const ws = c.workspace(9, wb);
        return c.run([=](void *f, void *stream) {
            return AS(strata_moe_grouped_product)(a, b, offsets, rows, E, N, K, o, t, ws, (size_t)wb, stream);
        });
    });
}

PyObject *grouped_product(ARGS) {
    static const char *const names[] = {"x", "W", "offsets", "rows",   "n_experts", "N",
                                        "K", "y", "ydtype",  "ws", "ws_bytes",  "stream"};
    return grouped(PRODUCT, args, nargs, names, 1, 2, 0);
}

PyObject *grouped_dgrad(ARGS) {
    static const char *const names[] = {"dy", "W",  "offsets", "rows", "n_experts", "N",
                                        "K",  "dx", "xdtype",  "ws",   "ws_bytes",  "stream"};
    return grouped(DGRAD, args, nargs, names, 0, 2, 1);
}

PyObject *grouped_wgrad(ARGS) {
    static const char *const names[] = {"dy", "x",  "offsets", "rows", "n_experts", "N",
                                        "K",  "dW", "wdtype",  "ws",   "ws_bytes",  "stream"};
    return grouped(WGRAD, args, nargs, names, 0, 1, 2);
}

// A block norm's description: the bytes of a BlockNormArgs.
struct NormCall {
    strata_block_norm_args p{};
    int64_t n = 0;
    strata_xdtype x, y, u;
    explicit NormCall(Call &c) {
        Py_buffer v;
        if (!c.ok) return;
        if (PyObject_GetBuffer(c.a[0], &v, PyBUF_SIMPLE) != 0) {
            c.ok = false;
            return;
        }
        if (v.len == (Py_ssize_t)sizeof(p)) memcpy(&p, v.buf, sizeof(p));
        else c.bad("args is not a BlockNormArgs");
        PyBuffer_Release(&v);
        n = count(p.T, p.d);
        x = c.code(p.x_dtype, "x_dtype");
        y = c.code(p.y_dtype, "y_dtype");
        u = c.code(p.u_dtype, "u_dtype");
    }
    void *gate(Call &c, int i) const {
        return p.flags & STRATA_GATE_TOKEN ? c.ptr(i, F32, p.T) : c.rows(i, y, n);
    }
};

PyObject *block_norm(ARGS) {
    static const char *const names[] = {"args", "x", "y",      "gate",   "g_post", "g_pre",
                                        "r",    "u", "rstd_y", "rstd_r", "stream"};
    return entry(NORM, args, nargs, names, [](Call &c) {
        const NormCall q(c);
        const void *const x = c.rows(1, q.x, q.n), *const y = c.rows(2, q.y, q.n), *const gate = q.gate(c, 3);
        const auto g_post = c.ptr<float>(4, F32, q.p.d), g_pre = c.ptr<float>(5, F32, q.p.d);
        void *const r = c.rows(6, q.x, q.n), *const u = c.rows(7, q.u, q.n);
        const auto rstd_y = c.ptr<float>(8, F32, q.p.T), rstd_r = c.ptr<float>(9, F32, q.p.T);
        return c.run([=](void *f, void *stream) {
            return AS(strata_block_norm)(&q.p, x, y, gate, g_post, g_pre, r, u, rstd_y, rstd_r, stream);
        });
    });
}

PyObject *block_norm_backward(ARGS) {
    static const char *const names[] = {"args",   "dr",     "du", "r",  "y",     "gate",    "g_post", "g_pre",    "rstd_y",
                                        "rstd_r", "dx",     "dy", "dgate", "dg_post", "dg_pre", "ws",    "ws_bytes", "stream"};
    return entry(NORM_BACK, args, nargs, names, [](Call &c) {
        const NormCall q(c);
        const int64_t wb = c.bytes(16);
        const void *const dr = c.rows(1, q.x, q.n), *const du = c.rows(2, q.u, q.n), *const r = c.rows(3, q.x, q.n);
        const void *const y = c.rows(4, q.y, q.n), *const gate = q.gate(c, 5);
        const auto g_post = c.ptr<float>(6, F32, q.p.d), g_pre = c.ptr<float>(7, F32, q.p.d);
        const auto rstd_y = c.ptr<float>(8, F32, q.p.T), rstd_r = c.ptr<float>(9, F32, q.p.T);
        void *const dx = c.rows(10, q.x, q.n), *const dy = c.rows(11, q.y, q.n), *const dgate = q.gate(c, 12);
        const auto dg_post = c.ptr<float>(13, F32, q.p.d), dg_pre = c.ptr<float>(14, F32, q.p.d);
        void *const ws = c.workspace(15, wb);
        return c.run([=](void *f, void *stream) {
            return AS(strata_block_norm_backward)(&q.p, dr, du, r, y, gate, g_post, g_pre, rstd_y, rstd_r, dx, dy, dgate,
                                                  dg_post, dg_pre, ws, (size_t)wb, stream);
        });
    });
}

PyObject *balance_loss(ARGS) {
    static const char *const names[] = {"z",   "zdtype", "idx",    "T",  "k",        "n_experts", "losses", "counts",
                                        "lse", "tokens", "ws", "ws_bytes", "prob",      "keep",   "stream"};
    return entry(BALANCE, args, nargs, names, [](Call &c) {
        const auto zt = c.code(1);
        const int32_t T = c.size(3), k = c.size(4), E = c.size(5);
        const int64_t wb = c.bytes(11);
        const void *const z = c.rows(0, zt, count(T, E));
        const auto idx = c.ptr<int32_t>(2, I32, count(T, k));
        const auto losses = c.ptr<float>(6, F32, 2);
        const auto counts = c.ptr<int32_t>(7, I32, E);
        const auto lse = c.ptr<float>(8, F32, T);
        const auto tokens = c.ptr<int32_t>(9, I32, 1);
        void *const ws = c.workspace(10, wb);
        const auto prob = c.ptr<float>(12, F32, E);
        const auto keep = c.truths(13, T);
        return c.run([=](void *f, void *stream) {
            return AS(strata_moe_balance)(z, zt, idx, keep, T, k, E, losses, counts, prob, lse, tokens, ws, (size_t)wb, stream);
        });
    });
}

PyObject *balance_loss_backward(ARGS) {
    static const char *const names[] = {"z",      "zdtype", "idx",     "T",  "k",    "n_experts", "lse",
                                        "counts", "tokens", "dlosses", "dz", "keep", "dpicks",    "stream"};
    return entry(BALANCE_BACK, args, nargs, names, [](Call &c) {
        const auto zt = c.code(1);
        const int32_t T = c.size(3), k = c.size(4), E = c.size(5);
        const void *const z = c.rows(0, zt, count(T, E));
        const auto idx = c.ptr<int32_t>(2, I32, count(T, k));
        const auto lse = c.ptr<float>(6, F32, T);
        const auto counts = c.ptr<int32_t>(7, I32, E), tokens = c.ptr<int32_t>(8, I32, 1);
        const auto dlosses = c.ptr<float>(9, F32, 2);
        void *const dz = c.rows(10, zt, count(T, E));
        const auto keep = c.truths(11, T);
        const auto dpicks = c.ptr<float>(12, F32, count(T, k));
        return c.run([=](void *f, void *stream) {
            return AS(strata_moe_balance_backward)(z, zt, idx, keep, T, k, E, lse, counts, tokens, dlosses, dpicks, dz, stream);
        });
    });
}

PyObject *embed(ARGS) {
    static const char *const names[] = {"W", "wdtype", "V", "d", "ids", "T", "scale", "out", "odtype", "stream"};
    return entry(EMBED, args, nargs, names, [](Call &c) {
        const auto wt = c.code(1), ot = c.code(8);
        const int32_t V = c.size(2), d = c.size(3), T = c.size(5);
        const float scale = c.number(6);
        const void *const W = c.rows(0, wt, count(V, d));
        const auto ids = c.ptr<int32_t>(4, I32, T);
        void *const out = c.rows(7, ot, count(T, d));
        return c.run([=](void *f, void *stream) { return AS(strata_embed)(W, wt, V, d, ids, T, scale, out, ot, stream); });
    });
}

PyObject *embed_backward(ARGS) {
    static const char *const names[] = {"dout", "odtype", "ids", "T",        "V",     "d",     "scale",
                                        "dW",   "wdtype", "ws",  "ws_bytes", "flags", "stream"};
    return entry(EMBED_BACK, args, nargs, names, [](Call &c) {
        const auto ot = c.code(1), wt = c.code(8);
        const int32_t T = c.size(3), V = c.size(4), d = c.size(5), flags = c.size(11);
        const float scale = c.number(6);
        const int64_t wb = c.bytes(10);
        const void *const dout = c.rows(0, ot, count(T, d));
        const auto ids = c.ptr<int32_t>(2, I32, T);
        void *const dW = c.rows(7, wt, count(V, d)), *const ws = c.workspace(9, wb);
        return c.run([=](void *f, void *stream) {
            return AS(strata_embed_backward)(dout, ot, ids, T, V, d, scale, dW, wt, (uint32_t)flags, ws, (size_t)wb, stream);
        });
    });
}

PyObject *vocab_loss(ARGS) {
    static const char *const names[] = {"h", "W", "targets", "T", "V", "d", "loss", "lse", "ws", "ws_bytes", "stream"};
    return entry(VOCAB, args, nargs, names, [](Call &c) {
        const int32_t T = c.size(3), V = c.size(4), d = c.size(5);
        const int64_t wb = c.bytes(9);
        const void *const h = c.ptr(0, BF16, count(T, d)), *const W = c.ptr(1, BF16, count(V, d));
        const auto targets = c.ptr<int32_t>(2, I32, T);
        const auto loss = c.ptr<float>(6, F32, T), lse = c.ptr<float>(7, F32, T);
        void *const ws = c.workspace(8, wb);
        return c.run([=](void *f, void *stream) {
            return AS(strata_vocab_loss)(h, W, targets, T, V, d, loss, lse, ws, (size_t)wb, stream);
        });
    });
}

PyObject *vocab_loss_backward(ARGS) {
    static const char *const names[] = {"h",        "W",    "targets", "T",       "V",  "d",       "lse",   "dloss", "ws",
                                        "ws_bytes", "dlse", "dh",      "dhdtype", "dW", "dwdtype", "flags", "stream"};
    return entry(VOCAB_BACK, args, nargs, names, [](Call &c) {
        const int32_t T = c.size(3), V = c.size(4), d = c.size(5), flags = c.size(15);
        const auto ht = c.code(12), wt = c.code(14);
        const int64_t wb = c.bytes(9);
        const void *const h = c.ptr(0, BF16, count(T, d)), *const W = c.ptr(1, BF16, count(V, d));
        const auto targets = c.ptr<int32_t>(2, I32, T);
        const auto lse = c.ptr<float>(6, F32, T), dloss = c.ptr<float>(7, F32, T), dlse = c.ptr<float>(10, F32, T);
        void *const ws = c.workspace(8, wb), *const dh = c.rows(11, ht, count(T, d)), *const dW = c.rows(13, wt, count(V, d));
        return c.run([=](void *f, void *stream) {
            return AS(strata_vocab_loss_backward)(h, W, targets, T, V, d, lse, dloss, dlse, dh, ht, dW, wt, (uint32_t)flags, ws,
                                                  (size_t)wb, stream);
        });
    });
}

PyObject *orthogonalise(ARGS) {
    static const char *const names[] = {"G",     "gdtype", "n", "N", "K", "out",   "ws", "ws_bytes",
                                        "steps", "a",      "b", "c", "scale", "eps", "stream"};
    return entry(ORTH, args, nargs, names, [](Call &c) {
        const auto gt = c.code(1);
        const int32_t n = c.size(2), N = c.size(3), K = c.size(4), steps = c.size(8);
        const int64_t wb = c.bytes(7);
        const float p[3] = {c.number(9), c.number(10), c.number(11)}, scale = c.number(12), eps = c.number(13);
        const void *const G = c.rows(0, gt, count(n, N, K));
        void *const out = c.ptr(5, BF16, count(n, N, K)), *const ws = c.workspace(6, wb);
        return c.run([=](void *f, void *stream) {
            return AS(strata_orthogonalise)(G, gt, n, N, K, steps, p, scale, eps, out, ws, (size_t)wb, stream);
        });
    });
}

#define METHOD(NAME) {#NAME, (PyCFunction)(void (*)())NAME, METH_FASTCALL, nullptr}
PyObject *bind(PyObject *, PyObject *);
PyMethodDef g_methods[] = {   // in the order of Fn
    METHOD(sort_picks),      METHOD(dispatch),      METHOD(dispatch_backward), METHOD(combine),
    METHOD(combine_backward), METHOD(grouped_product), METHOD(grouped_dgrad),     METHOD(grouped_wgrad),
    METHOD(block_norm),      METHOD(block_norm_backward), METHOD(balance_loss),   METHOD(balance_loss_backward),
    METHOD(embed),           METHOD(embed_backward),  METHOD(vocab_loss),         METHOD(vocab_loss_backward),
    METHOD(orthogonalise),   {"bind", bind, METH_VARARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};

// bind(addresses of the library's functions, raise, elsewhere, device, first device, stream)
PyObject *bind(PyObject *module, PyObject *args) {
    PyObject *fns, *o[5];
    if (!PyArg_ParseTuple(args, "O!OOOOO", &PyTuple_Type, &fns, o, o + 1, o + 2, o + 3, o + 4)) return nullptr;
    if (PyTuple_GET_SIZE(fns) != FNS) {
        PyErr_SetString(PyExc_TypeError, "an address for every function");
        return nullptr;
    }
    PyObject **const to[5] = {&g_raise, &g_elsewhere, &g_device, &g_first_device, &g_stream};
    for (int i = 0; i < 5; ++i) {
        Py_INCREF(o[i]);
        Py_XSETREF(*to[i], o[i]);
    }
    for (int i = 0; i < FNS; ++i) {
        PyObject *self = PyObject_GetAttrString(module, g_methods[i].ml_name);
        if (!self) return nullptr;
        Py_XSETREF(g_self[i], self);
        g_fn[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(fns, i));
        if (PyErr_Occurred()) return nullptr;
    }
    Py_RETURN_NONE;
}

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
