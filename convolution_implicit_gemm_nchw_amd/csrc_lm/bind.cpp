// bind.cpp -- Python binding of the state-space operators (module _miconv_bind):
// checks the operands, allocates the outputs that were not given, fills the C
// structures and calls libmiconv.so on the current stream.  A token's calls take a few
// microseconds on the GPU, and as much Python as these checks need took longer.
//
// Every function takes all its arguments by position; None stands for an absent one.
// A misfit raises ValueError; for a status the function given to errors() raises.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/miconv.h"

namespace {

typedef std::initializer_list<int64_t> Shape;

struct Raised {};                          // a Python error is set

PyObject *on_status_fn = nullptr, *out_of_memory = nullptr;

[[noreturn]] void refuse(const std::string &what) { throw std::invalid_argument(what); }

std::string text(at::IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + ")";
}

const at::Tensor &tensor(const char *name, PyObject *o) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

int code_of(at::ScalarType t) {
    if (t == at::kFloat) return MICONV_F32;
    if (t == at::kBFloat16) return MICONV_BF16;
    refuse(std::string("unsupported dtype ") + c10::toString(t) + "; expected float32 or bfloat16");
}

// What the leading operand fixes for the others.
struct Lead {
    const at::Tensor &t;
    at::ScalarType dt;
    int code, dev;
    Lead(const char *name, PyObject *o, int64_t dims) : t(tensor(name, o)) {
        if (!t.is_cuda() || t.dim() != dims)
            refuse(std::string(name) + " must be a " + std::to_string(dims) + "-dimensional device tensor");
        dt = t.scalar_type();
        code = code_of(dt);
        dev = t.get_device();
    }
};

const at::Tensor &fits(const char *name, PyObject *o, at::IntArrayRef shape, at::ScalarType dt, int dev) {
    const at::Tensor &t = tensor(name, o);
    if (t.scalar_type() != dt || t.sizes() != shape || !t.is_cuda() || t.get_device() != dev)
        refuse(std::string(name) + " must be a " + c10::toString(dt) + " tensor of shape " + text(shape) + " on device " +
               std::to_string(dev) + ", not " + c10::toString(t.scalar_type()) + " of " + text(t.sizes()) + " on " +
               t.device().str());
    return t;
}

void *packed(const char *name, PyObject *o, Shape shape, at::ScalarType dt, int dev) {
    const at::Tensor &t = fits(name, o, shape, dt, dev);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    return t.data_ptr();
}

void *optional(const char *name, PyObject *o, Shape shape, at::ScalarType dt, int dev) {
    return o == Py_None ? nullptr : packed(name, o, shape, dt, dev);
}

miconv_rows_t rows_of(const char *name, const at::Tensor &t) {
    if (t.dim() == 3 && t.size(2) > 1 && t.stride(2) != 1)
        refuse(std::string(name) + " must have contiguous time steps (stride 1 along the last axis)");
    return {t.data_ptr(), t.stride(0), t.stride(1)};
}

// A [B, D, L] or [B, D] operand shaped like the leading one; zeros for None.
miconv_rows_t rows(const char *name, PyObject *o, const Lead &x) {
    if (o == Py_None) return {nullptr, 0, 0};
    return rows_of(name, fits(name, o, x.t.sizes(), x.dt, x.dev));
}

// An output: the caller's tensor, or a new one.
struct Out {
    at::Tensor t;
    Out(const char *name, PyObject *o, at::IntArrayRef shape, at::ScalarType dt, const Lead &x, bool views = false) {
        if (o == Py_None) {
            t = at::empty(shape, x.t.options().dtype(dt));
        } else {
            t = fits(name, o, shape, dt, x.dev);
            if (!views && !t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
        }
    }
    Out() {}
    void *data() const { return t.defined() ? t.data_ptr() : nullptr; }
    PyObject *wrap() const {
        if (t.defined()) return THPVariable_Wrap(t);
        Py_RETURN_NONE;
    }
};

struct Scratch {
    at::Tensor t;
    void *p = nullptr;
    size_t n = 0;
    Scratch(PyObject *given, size_t need, const Lead &x) {
        if (given != Py_None) {
            const at::Tensor &w = tensor("workspace", given);
            if (!w.is_cuda() || w.get_device() != x.dev || !w.is_contiguous())
                refuse("workspace must be a contiguous tensor on the operands' device");
            p = w.data_ptr();
            n = w.nbytes();
        } else if (need) {
            t = at::empty({(int64_t)need}, x.t.options().dtype(at::kByte));
            p = t.data_ptr();
            n = need;
        }
    }
};

void check(int status, const char *where) {
    if (status == MICONV_OK) return;
    PyObject *r = PyObject_CallFunction(on_status_fn, "is", status, where);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: status %d", where, status);
    throw Raised();
}

// Calls fn(..., stream) with the operands' device current, on its current stream.  fn throws nothing:
// the device that was current before would not be set again.
template <typename F>
void run(const char *where, int dev, F fn) {
    const int now = c10::hip::current_device();
    if (now != dev) c10::hip::set_device(dev);
    const int status = fn((void *)c10::hip::getCurrentHIPStream(dev).stream());
    if (now != dev) c10::hip::set_device(now);
    check(status, where);
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised();
    return v != 0;
}

int dim(int64_t v) {
    if (v > 0x7fffffff) refuse("a size is too large");
    return (int)v;
}

PyObject *tuple(std::initializer_list<const Out *> outs) {
    PyObject *t = PyTuple_New((Py_ssize_t)outs.size());
    if (!t) throw Raised();
    Py_ssize_t i = 0;
    for (const Out *o : outs) {
        PyObject *w = o->wrap();
        if (!w) {
            Py_DECREF(t);
            throw Raised();
        }
        PyTuple_SET_ITEM(t, i++, w);
    }
    return t;
}

typedef PyObject *const *Args;

// ------------------------------------------------------------------ causal convolution

int taps(PyObject *w) {
    const at::Tensor &t = tensor("w", w);
    if (t.dim() != 2) refuse("w must be [D, K]");
    return dim(t.size(1));
}

// x, w, bias, silu, initial_state, lengths: the first six arguments of both passes.
miconv_causal_conv_t conv_common(const Lead &x, Args a) {
    miconv_causal_conv_t c = {};
    c.B = dim(x.t.size(0));
    c.D = dim(x.t.size(1));
    c.L = dim(x.t.size(2));
    c.K = taps(a[1]);
    c.silu = truth(a[3]);
    c.x = rows_of("x", x.t);
    c.w = packed("w", a[1], {c.D, c.K}, x.dt, x.dev);
    c.bias = (const float *)optional("bias", a[2], {c.D}, at::kFloat, x.dev);
    c.initial_state = optional("initial_state", a[4], {c.B, c.D, c.K - 1}, x.dt, x.dev);
    c.lengths = (const int *)optional("lengths", a[5], {c.B}, at::kInt, x.dev);
    return c;
}

// (x, w, bias, silu, initial_state, lengths, y, final_state) -> y
PyObject *conv_fwd(Args a) {
    const Lead x("x", a[0], 3);
    miconv_causal_conv_t c = conv_common(x, a);
    const Out y("y", a[6], x.t.sizes(), x.dt, x, true);
    c.y = rows_of("y", y.t);
    c.final_state = optional("final_state", a[7], {c.B, c.D, c.K - 1}, x.dt, x.dev);
    run("causal_conv1d_fwd", x.dev, [&](void *st) { return causal_conv1d_fwd(&c, x.code, st); });
    return y.wrap();
}

// (x, w, bias, silu, initial_state, lengths, dy, d_final_state, dx, dw, dbias, d_initial_state, workspace)
// -> (dx, dw, dbias)
PyObject *conv_bwd(Args a) {
    const Lead x("x", a[0], 3);
    miconv_causal_conv_t c = conv_common(x, a);
    if (a[6] == Py_None) refuse("dy must be a tensor");
    c.dy = rows("dy", a[6], x);
    c.d_final_state = optional("d_final_state", a[7], {c.B, c.D, c.K - 1}, x.dt, x.dev);
    const Out dx("dx", a[8], x.t.sizes(), x.dt, x, true), dw("dw", a[9], {c.D, c.K}, at::kFloat, x);
    const Out db = a[2] == Py_None && a[10] == Py_None ? Out() : Out("dbias", a[10], {c.D}, at::kFloat, x);
    c.dx = rows_of("dx", dx.t);
    c.dw = (float *)dw.data();
    c.dbias = (float *)db.data();
    c.d_initial_state = optional("d_initial_state", a[11], {c.B, c.D, c.K - 1}, x.dt, x.dev);
    size_t need = 0;
    if (a[12] == Py_None)
        check(causal_conv1d_bwd_workspace_size(&c, x.code, MICONV_MAX_WORKSPACE_BYTES, &need),
              "causal_conv1d_bwd_workspace_size");
    const Scratch ws(a[12], need, x);
    run("causal_conv1d_bwd", x.dev, [&](void *st) { return causal_conv1d_bwd(&c, x.code, ws.p, ws.n, st); });
    return tuple({&dx, &dw, &db});
}

// The states of a step: how many, and which slot each sequence has.
struct States {
    int slots;
    const int *slot_of;
    States(PyObject *state, PyObject *slots_arg, int B, int dev) {
        const at::Tensor &t = tensor("state", state);
        if (t.dim() != 3) refuse("state must have 3 dimensions");
        slots = dim(t.size(0));
        if (slots_arg == Py_None && slots != B) refuse("without slots, state must hold one state for each sequence");
        slot_of = (const int *)optional("slots", slots_arg, {B}, at::kInt, dev);
    }
};

// (x, state, w, bias, silu, state_out, slots, y) -> y
PyObject *conv_step(Args a) {
    const Lead x("x", a[0], 2);
    const int B = dim(x.t.size(0)), D = dim(x.t.size(1)), K = taps(a[2]);
    const States s(a[1], a[6], B, x.dev);
    const void *in = packed("state", a[1], {s.slots, D, K - 1}, x.dt, x.dev);
    void *out = a[5] == Py_None ? (void *)in : packed("state_out", a[5], {s.slots, D, K - 1}, x.dt, x.dev);
    const void *w = packed("w", a[2], {D, K}, x.dt, x.dev);
    const float *bias = (const float *)optional("bias", a[3], {D}, at::kFloat, x.dev);
    const int silu = truth(a[4]);
    const Out y("y", a[7], x.t.sizes(), x.dt, x, true);
    const miconv_rows_t xr = rows_of("x", x.t), yr = rows_of("y", y.t);
    run("causal_conv1d_step", x.dev, [&](void *st) {
        return causal_conv1d_step(B, D, K, silu, x.code, xr, in, s.slots, s.slot_of, w, bias, out, yr, st);
    });
    return y.wrap();
}

// ------------------------------------------------------------------ selective scan

miconv_scan_in_t scan_in(const char *name, PyObject *o, at::IntArrayRef shape, const Lead &x) {
    const at::Tensor &t = fits(name, o, shape, x.dt, x.dev);
    if (t.dim() == 4 && t.size(3) > 1 && t.stride(3) != 1)
        refuse(std::string(name) + " must have contiguous time steps (stride 1 along the last axis)");
    return {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}

// x, delta, A, B, C, D, z, delta_bias, softplus, lengths: the first ten arguments of all.
miconv_scan_t scan_common(const Lead &x, Args a, bool step) {
    miconv_scan_t s = {};
    const at::Tensor &A = tensor("A", a[2]), &Bm = tensor("B", a[3]);
    if (A.dim() != 2 || Bm.dim() != (step ? 3 : 4))
        refuse("A must be [D, N], B and C [B, G, N, L] ([B, G, N] for one step)");
    s.B = dim(x.t.size(0));
    s.D = dim(x.t.size(1));
    s.L = step ? 1 : dim(x.t.size(2));
    s.N = dim(A.size(1));
    s.G = dim(Bm.size(1));
    s.softplus = truth(a[8]);
    s.x = rows_of("x", x.t);
    if (a[1] == Py_None) refuse("delta must be a tensor");
    s.delta = rows("delta", a[1], x);
    s.z = rows("z", a[6], x);
    s.A = (const float *)packed("A", a[2], {s.D, s.N}, at::kFloat, x.dev);
    const int64_t shape[4] = {s.B, s.G, s.N, s.L};
    s.Bm = scan_in("B", a[3], at::IntArrayRef(shape, step ? 3 : 4), x);
    s.Cm = scan_in("C", a[4], at::IntArrayRef(shape, step ? 3 : 4), x);
    s.D_skip = (const float *)optional("D", a[5], {s.D}, at::kFloat, x.dev);
    s.delta_bias = (const float *)optional("delta_bias", a[7], {s.D}, at::kFloat, x.dev);
    s.lengths = (const int *)optional("lengths", a[9], {s.B}, at::kInt, x.dev);
    return s;
}

int64_t states_count(int B, int D, int L, int N) {
    size_t bytes = 0;
    check(selective_scan_states_size(B, D, L, N, &bytes), "selective_scan_states_size");
    return (int64_t)(bytes / 4);
}

// (x, A) -> states
PyObject *scan_states(Args a) {
    const Lead x("x", a[0], 3);
    const at::Tensor &A = tensor("A", a[1]);
    if (A.dim() != 2) refuse("A must be [D, N]");
    const int64_t n = states_count(dim(x.t.size(0)), dim(x.t.size(1)), dim(x.t.size(2)), dim(A.size(1)));
    return THPVariable_Wrap(at::empty({n}, x.t.options().dtype(at::kFloat)));
}

// (..., initial_state, y, final_state, states, workspace) -> y
PyObject *scan_fwd(Args a) {
    const Lead x("x", a[0], 3);
    miconv_scan_t s = scan_common(x, a, false);
    s.initial_state = (const float *)optional("initial_state", a[10], {s.B, s.D, s.N}, at::kFloat, x.dev);
    const Out y("y", a[11], x.t.sizes(), x.dt, x, true);
    s.y = rows_of("y", y.t);
    s.final_state = (float *)optional("final_state", a[12], {s.B, s.D, s.N}, at::kFloat, x.dev);
    if (a[13] != Py_None)
        s.states = (float *)packed("states", a[13], {states_count(s.B, s.D, s.L, s.N)}, at::kFloat, x.dev);
    size_t need = 0;
    if (a[14] == Py_None)
        check(selective_scan_fwd_workspace_size(&s, x.code, MICONV_MAX_WORKSPACE_BYTES, &need),
              "selective_scan_fwd_workspace_size");
    const Scratch ws(a[14], need, x);
    run("selective_scan_fwd", x.dev, [&](void *st) { return selective_scan_fwd(&s, x.code, ws.p, ws.n, st); });
    return y.wrap();
}

// (..., dy, states, d_final_state, d_initial_state, dx, ddelta, dz, workspace)
// -> (dx, ddelta, dz, dA, dB, dC, dD, ddelta_bias)
PyObject *scan_bwd(Args a) {
    const Lead x("x", a[0], 3);
    miconv_scan_t s = scan_common(x, a, false);
    if (a[10] == Py_None) refuse("dy must be a tensor");
    if (a[11] == Py_None) refuse("states of the forward pass are needed");
    s.dy = rows("dy", a[10], x);
    s.states = (float *)packed("states", a[11], {states_count(s.B, s.D, s.L, s.N)}, at::kFloat, x.dev);
    s.d_final_state = (const float *)optional("d_final_state", a[12], {s.B, s.D, s.N}, at::kFloat, x.dev);
    s.d_initial_state = (float *)optional("d_initial_state", a[13], {s.B, s.D, s.N}, at::kFloat, x.dev);
    const Out dx("dx", a[14], x.t.sizes(), x.dt, x, true), dd("ddelta", a[15], x.t.sizes(), x.dt, x, true);
    const Out dz = a[6] == Py_None ? Out() : Out("dz", a[16], x.t.sizes(), x.dt, x, true);
    const at::ScalarType f = at::kFloat;
    const Out dA("dA", Py_None, {s.D, s.N}, f, x), dB("dB", Py_None, {s.B, s.G, s.N, s.L}, f, x),
        dC("dC", Py_None, {s.B, s.G, s.N, s.L}, f, x);
    const Out dD = a[5] == Py_None ? Out() : Out("dD", Py_None, {s.D}, f, x);
    const Out db = a[7] == Py_None ? Out() : Out("ddelta_bias", Py_None, {s.D}, f, x);
    s.dx = rows_of("dx", dx.t);
    s.ddelta = rows_of("ddelta", dd.t);
    if (dz.t.defined()) s.dz = rows_of("dz", dz.t);
    s.dA = (float *)dA.data();
    s.dB = (float *)dB.data();
    s.dC = (float *)dC.data();
    s.dD = (float *)dD.data();
    s.ddelta_bias = (float *)db.data();
    size_t need = 0;
    if (a[17] == Py_None)
        check(selective_scan_bwd_workspace_size(&s, x.code, &need), "selective_scan_bwd_workspace_size");
    const Scratch ws(a[17], need, x);
    run("selective_scan_bwd", x.dev, [&](void *st) { return selective_scan_bwd(&s, x.code, ws.p, ws.n, st); });
    return tuple({&dx, &dd, &dz, &dA, &dB, &dC, &dD, &db});
}

// (..., state, state_out, slots, y) -> y
PyObject *scan_step(Args a) {
    const Lead x("x", a[0], 2);
    miconv_scan_t s = scan_common(x, a, true);
    const States t(a[10], a[12], s.B, x.dev);
    const float *in = (const float *)packed("state", a[10], {t.slots, s.D, s.N}, at::kFloat, x.dev);
    float *out = a[11] == Py_None ? (float *)in : (float *)packed("state_out", a[11], {t.slots, s.D, s.N}, at::kFloat, x.dev);
    const Out y("y", a[13], x.t.sizes(), x.dt, x, true);
    s.y = rows_of("y", y.t);
    run("selective_scan_step", x.dev,
        [&](void *st) { return selective_scan_step(&s, x.code, in, t.slots, t.slot_of, out, st); });
    return y.wrap();
}

// ------------------------------------------------------------------ 8-bit products

// (x, channel_major, q, scale) -> (q, scale)
PyObject *quantize(Args a) {
    const bool cm = truth(a[1]);
    const int64_t dims = THPVariable_Check(a[0]) && !cm && THPVariable_Unpack(a[0]).dim() == 2 ? 2 : 3;
    const Lead x("x", a[0], dims);
    int64_t nb = 1, L, C, sb = 0, sl, sc = 1;
    if (cm) {
        nb = x.t.size(0), C = x.t.size(1), L = x.t.size(2);
        sb = x.t.stride(0), sc = x.t.stride(1), sl = 1;
        if (L > 1 && x.t.stride(2) != 1) refuse("x must have contiguous time steps (stride 1 along the last axis)");
    } else {
        if (dims == 3) nb = x.t.size(0), sb = x.t.stride(0);
        L = x.t.size(dims - 2), sl = x.t.stride(dims - 2), C = x.t.size(dims - 1);
        if (C > 1 && x.t.stride(dims - 1) != 1) refuse("x must have contiguous channels (stride 1 along the last axis)");
    }
    const int64_t pad = (C + MICONV_I8_PAD - 1) / MICONV_I8_PAD * MICONV_I8_PAD;
    const int B = dim(nb), tokens = dim(L), channels = dim(C);
    const Out q("q", a[2], {nb * L, pad}, at::kChar, x), scale("scale", a[3], {nb * L}, at::kFloat, x);
    const void *data = x.t.data_ptr();
    run("quantize_tokens", x.dev, [&](void *st) {
        return quantize_tokens(B, tokens, channels, x.code, data, sb, sl, sc, (signed char *)q.data(),
                               (float *)scale.data(), st);
    });
    return tuple({&q, &scale});
}

// (q, scale, wq, wscale, bias, bf16, length, y, workspace) -> y
PyObject *matmul(Args a) {
    const at::Tensor &q = tensor("q", a[0]), &w = tensor("wq", a[2]);
    if (!q.is_cuda() || q.dim() != 2 || w.dim() != 2) refuse("q and wq must be 2-dimensional device tensors");
    const int dev = q.get_device();
    const int T = dim(q.size(0)), K = dim(q.size(1)), O = dim(w.size(0));
    int B = 1, L = T;
    const bool cm = a[6] != Py_None;
    if (cm) {
        const long length = PyLong_AsLong(a[6]);
        if (length == -1 && PyErr_Occurred()) throw Raised();
        if (length < 1 || T % length) refuse("length must divide the number of tokens");
        L = dim(length);
        B = T / L;
    }
    const signed char *qp = (const signed char *)packed("q", a[0], {T, K}, at::kChar, dev);
    const float *qs = (const float *)packed("scale", a[1], {T}, at::kFloat, dev);
    const signed char *wp = (const signed char *)packed("wq", a[2], {O, K}, at::kChar, dev);
    const float *ws = (const float *)packed("wscale", a[3], {O}, at::kFloat, dev);
    const float *bias = (const float *)optional("bias", a[4], {O}, at::kFloat, dev);
    at::Tensor y;
    if (a[7] == Py_None) {
        const auto opt = q.options().dtype(truth(a[5]) ? at::kBFloat16 : at::kFloat);
        y = cm ? at::empty({B, O, L}, opt) : at::empty({T, O}, opt);
    } else {
        const at::ScalarType dt = tensor("y", a[7]).scalar_type();
        code_of(dt);
        y = fits("y", a[7], cm ? at::IntArrayRef({B, O, L}) : at::IntArrayRef({T, O}), dt, dev);
        if (!y.is_contiguous()) refuse("y must be contiguous");
    }
    size_t need = 0;
    if (a[8] == Py_None)
        check(matmul_i8_workspace_size(B, L, O, K, MICONV_MAX_WORKSPACE_BYTES, &need), "matmul_i8_workspace_size");
    at::Tensor held;
    void *work = nullptr;
    if (a[8] != Py_None) {
        held = tensor("workspace", a[8]);
        if (!held.is_cuda() || held.get_device() != dev || !held.is_contiguous())
            refuse("workspace must be a contiguous tensor on the operands' device");
        need = held.nbytes();
    } else if (need) {
        held = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
    }
    if (held.defined()) work = held.data_ptr();
    const int code = code_of(y.scalar_type());
    void *out = y.data_ptr();
    run("matmul_i8", dev, [&](void *st) {
        return matmul_i8(B, L, O, K, qp, qs, wp, ws, bias, cm, code, out, work, work ? need : 0, st);
    });
    return THPVariable_Wrap(y);
}

// ------------------------------------------------------------------ module

// fn with N arguments; no C++ exception leaves it.
template <PyObject *(*FN)(Args), int N>
PyObject *entry(PyObject *, Args args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return FN(args);
    } catch (const Raised &) {
    } catch (const std::invalid_argument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(out_of_memory ? out_of_memory : PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// errors(on_status, OutOfMemoryError): what raises for a status, and torch's class.
PyObject *errors(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "expected 2 arguments");
        return nullptr;
    }
    Py_INCREF(args[0]);
    Py_INCREF(args[1]);
    Py_XDECREF(on_status_fn);
    Py_XDECREF(out_of_memory);
    on_status_fn = args[0];
    out_of_memory = args[1];
    Py_RETURN_NONE;
}

#define ENTRY(name, fn, n) {name, (PyCFunction)(void *)entry<fn, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY("causal_conv1d_fwd", conv_fwd, 8),
                         ENTRY("causal_conv1d_bwd", conv_bwd, 13),
                         ENTRY("causal_conv1d_step", conv_step, 8),
                         ENTRY("selective_scan_states", scan_states, 2),
                         ENTRY("selective_scan_fwd", scan_fwd, 15),
                         ENTRY("selective_scan_bwd", scan_bwd, 18),
                         ENTRY("selective_scan_step", scan_step, 14),
                         ENTRY("quantize_tokens", quantize, 4),
                         ENTRY("matmul_i8", matmul, 9),
                         {"errors", (PyCFunction)(void *)errors, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_miconv_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__miconv_bind(void) { return PyModule_Create(&module); }
