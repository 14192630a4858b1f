// Short way through the Python binding for calls that fit as they are.
//
// A single token's operator takes 3-11 us on the GPU; the Python checks,
// allocations and ctypes conversions around it took 10-16 us.  Each function
// here takes the binding's arguments, makes the same checks and allocations in
// C++ and calls the C entry point.  It knows no errors: whatever does not fit
// (another type, shape, layout or device, a CPU tensor) returns None, and the
// binding's own code then refuses the call or makes it.  A status other than
// SSD_OK comes back as an int.
//
// Built against a ROCm build of torch (libtorch_hip): allocations go straight to
// its allocator of GPU memory.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>

#include "ssd.h"

namespace {

decltype(&ssd_causal_conv_fwd) g_conv;
decltype(&ssd_selective_scan_fwd) g_scan;
decltype(&ssd_selective_scan_workspace_bytes) g_scan_bytes;
decltype(&ssd_gated_norm_fwd) g_norm;
decltype(&ssd_verify_drafts) g_verify;
decltype(&ssd_verify_workspace_bytes) g_verify_bytes;
decltype(&ssd_gated_delta_fwd) g_delta;
decltype(&ssd_gated_delta_workspace_bytes) g_delta_bytes;
decltype(&ssd_residual_norm_fwd) g_residual_norm;

// An argument that is a tensor or None (anything else does not fit).
struct Arg {
    at::Tensor t;
    bool ok;
    explicit Arg(PyObject *o) : ok(o == Py_None || THPVariable_Check(o)) {
        if (ok && o != Py_None) t = THPVariable_Unpack(o);
    }
    void *ptr() const { return t.defined() ? t.data_ptr() : nullptr; }
};

bool sized(const at::Tensor &t, std::initializer_list<int64_t> sizes) {
    return t.sizes() == at::IntArrayRef(sizes.begin(), sizes.size());
}
// A dense tensor of these sizes, or absent where it may be.
bool dense(const Arg &a, std::initializer_list<int64_t> sizes, at::ScalarType type, at::Device dev,
           bool required = false) {
    if (!a.ok) return false;
    if (!a.t.defined()) return !required;
    return sized(a.t, sizes) && a.t.scalar_type() == type && a.t.device() == dev && a.t.is_contiguous();
}
// The same, but with free strides before the last `inner` dimensions.
bool strided(const Arg &a, std::initializer_list<int64_t> sizes, at::ScalarType type, at::Device dev, bool required,
             int inner = 1) {
    if (!a.ok) return false;
    if (!a.t.defined()) return !required;
    if (!sized(a.t, sizes) || a.t.scalar_type() != type || a.t.device() != dev || a.t.stride(-1) != 1) return false;
    return inner == 1 || a.t.stride(-2) == a.t.size(-1);
}

// The type code of a first argument on the current GPU, -1 where it does not fit.
int code_of(const Arg &a) {
    if (!a.ok || !a.t.defined() || !a.t.is_cuda()) return -1;
    if (a.t.device() != c10::impl::VirtualGuardImpl(at::kCUDA).getDevice()) return -1;
    return a.t.scalar_type() == at::kBFloat16 ? SSD_DTYPE_BF16 : a.t.scalar_type() == at::kFloat ? SSD_DTYPE_F32 : -1;
}

// A new dense tensor on the GPU: what at::empty makes behind the dispatcher, which
// costs as much host time again.
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, at::Device dev) {
    return at::Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
}

PyObject *none() { Py_RETURN_NONE; }
PyObject *wrap(const at::Tensor &t) { return t.defined() ? THPVariable_Wrap(t) : none(); }
PyObject *three(PyObject *a, PyObject *b, PyObject *c) {
    PyObject *r = a && b && c ? PyTuple_Pack(3, a, b, c) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    Py_XDECREF(c);
    return r;
}
void *stream_of(PyObject *o) { return PyLong_AsVoidPtr(o); }

// Gives the interpreter lock away, as ctypes does around a foreign function: a
// launch waits where the stream's queue is full and an allocation may wait for
// the GPU, and other Python threads (one that the queue itself waits for among
// them, in a host callback) run meanwhile.  Nothing of Python is touched while
// it lives; it takes the lock back before an exception passes.
class Unlocked {
    PyThreadState *state_ = PyEval_SaveThread();

public:
    Unlocked() = default;
    Unlocked(const Unlocked &) = delete;
    Unlocked &operator=(const Unlocked &) = delete;
    ~Unlocked() { PyEval_RestoreThread(state_); }
};

// No C++ exception leaves a function called from Python: torch's macros turn
// it into the Python error it stands for (out of memory among them).
template <typename F>
PyObject *guarded(F &&f) {
    HANDLE_TH_ERRORS
    return f();
    END_HANDLE_TH_ERRORS
}

// x, weight, bias, init_state, state_out_idx, split, silu, final_state, return_final_state, stream
PyObject *conv(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 10 || !PyBool_Check(a[6]) || !PyBool_Check(a[8])) return none();
        const Arg x(a[0]), w(a[1]), bias(a[2]), init(a[3]), idx(a[4]);
        Arg fin(a[7]);
        const int code = code_of(x);
        if (code < 0 || x.t.dim() != 3 || !w.ok || !w.t.defined() || w.t.dim() != 2) return none();
        const int64_t b = x.t.size(0), T = x.t.size(1), ch = x.t.size(2), W = w.t.size(1);
        const auto type = x.t.scalar_type();
        const auto dev = x.t.device();
        int64_t sizes[3] = {ch, 0, 0};
        int outs = 1;
        if (a[5] != Py_None) {
            const bool list = PyList_CheckExact(a[5]);
            if (!list && !PyTuple_CheckExact(a[5])) return none();
            outs = (int)PySequence_Fast_GET_SIZE(a[5]);
            if (outs < 1 || outs > 3) return none();
            int64_t sum = 0;
            for (int i = 0; i < outs; ++i) {
                PyObject *o = PySequence_Fast_GET_ITEM(a[5], i);
                if (!PyLong_CheckExact(o)) return none();
                sizes[i] = PyLong_AsLongLong(o);
                if (sizes[i] <= 0 || sizes[i] > ch) {
                    PyErr_Clear();
                    return none();
                }
                sum += sizes[i];
            }
            if (sum != ch) return none();
        }
        if (b == 0 || T == 0 || ch == 0 || W < 2 || !strided(x, {b, T, ch}, type, dev, true) ||
            !dense(w, {ch, W}, at::kFloat, dev, true) || !dense(bias, {ch}, at::kFloat, dev) ||
            !dense(init, {b, W - 1, ch}, type, dev) || !dense(idx, {b}, at::kInt, dev) ||
            !dense(fin, {b, W - 1, ch}, type, dev))
            return none();
        const bool want_final = a[8] == Py_True, silu = a[6] == Py_True;
        void *const stream = stream_of(a[9]);
        at::Tensor out[3], at_j;
        ssd_status st;
        {
            const Unlocked unlocked;
            const auto opt = x.t.options();
            for (int i = 0; i < outs; ++i) out[i] = at::empty({b, T, sizes[i]}, opt);
            if (!fin.t.defined() && want_final) fin.t = at::empty({b, W - 1, ch}, opt);
            if (idx.t.defined()) at_j = at::empty({b, W - 1, ch}, opt);
            ssd_conv_shape s = {b, T, {sizes[0], sizes[1], sizes[2]}, W, x.t.stride(0), x.t.stride(1)};
            auto p = [](const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; };
            st = g_conv(x.ptr(), (const float *)w.ptr(), (const float *)bias.ptr(), init.ptr(),
                        silu ? SSD_ACT_SILU : SSD_ACT_NONE, p(out[0]), p(out[1]), p(out[2]), fin.ptr(),
                        (const int32_t *)idx.ptr(), p(at_j), &s, (ssd_dtype)code, stream);
        }
        if (st != SSD_OK) return PyLong_FromLong(st);
        PyObject *o;
        if (a[5] == Py_None) {
            o = wrap(out[0]);
        } else {
            o = PyTuple_New(outs);
            for (int i = 0; o && i < outs; ++i) PyTuple_SET_ITEM(o, i, wrap(out[i]));
        }
        return three(o, wrap(fin.t), wrap(at_j));
    });
}

// u, delta, A, B, C, D, z, delta_bias, init_state, state_out_idx, softplus, final_state, return_final_state, stream
PyObject *scan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 14 || !PyBool_Check(a[10]) || !PyBool_Check(a[12])) return none();
        const Arg u(a[0]), dl(a[1]), A(a[2]), B(a[3]), C(a[4]), D(a[5]), z(a[6]), bias(a[7]), init(a[8]), idx(a[9]);
        Arg fin(a[11]);
        const int code = code_of(u);
        if (code < 0 || u.t.dim() != 3 || !A.ok || !A.t.defined() || A.t.dim() != 2 || !B.ok || !B.t.defined() ||
            B.t.dim() != 4)
            return none();
        const int64_t b = u.t.size(0), T = u.t.size(1), ch = u.t.size(2), G = B.t.size(2), N = B.t.size(3);
        const auto type = u.t.scalar_type();
        const auto dev = u.t.device();
        if (b == 0 || T == 0 || ch == 0 || !strided(u, {b, T, ch}, type, dev, true) ||
            !strided(dl, {b, T, ch}, type, dev, true) || !strided(z, {b, T, ch}, type, dev, false) ||
            !strided(B, {b, T, G, N}, type, dev, true, 2) || !strided(C, {b, T, G, N}, type, dev, true, 2) ||
            !dense(A, {ch, N}, at::kFloat, dev, true) || !dense(D, {ch}, at::kFloat, dev) ||
            !dense(bias, {ch}, at::kFloat, dev) || !dense(init, {b, ch, N}, at::kFloat, dev) ||
            !dense(idx, {b}, at::kInt, dev) || !dense(fin, {b, ch, N}, at::kFloat, dev))
            return none();
        const bool want_final = a[12] == Py_True, softplus = a[10] == Py_True;
        void *const stream = stream_of(a[13]);
        at::Tensor y, at_j, ws;
        ssd_status r;
        {
            const Unlocked unlocked;
            auto st = [](const Arg &t, int d) { return t.t.defined() ? t.t.stride(d) : 0; };
            ssd_selective_shape s = {b,        T,        ch,       N,        G,        st(u, 0), st(u, 1), st(dl, 0),
                                     st(dl, 1), st(z, 0), st(z, 1), st(B, 0), st(B, 1), st(C, 0), st(C, 1)};
            const size_t bytes = g_scan_bytes(&s, (ssd_dtype)code);
            y = at::empty({b, T, ch}, u.t.options());
            if (!fin.t.defined() && want_final) fin.t = at::empty({b, ch, N}, A.t.options());
            if (idx.t.defined()) at_j = at::empty({b, ch, N}, A.t.options());
            if (bytes > 0) ws = at::empty({(int64_t)bytes}, A.t.options().dtype(at::kByte));
            auto p = [](const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; };
            r = g_scan(u.ptr(), dl.ptr(), (const float *)A.ptr(), B.ptr(), C.ptr(), (const float *)D.ptr(), z.ptr(),
                       (const float *)bias.ptr(), softplus, (const float *)init.ptr(), y.data_ptr(), (float *)fin.ptr(),
                       (const int32_t *)idx.ptr(), (float *)p(at_j), &s, (ssd_dtype)code, p(ws), bytes, stream);
        }
        if (r != SSD_OK) return PyLong_FromLong(r);
        return three(wrap(y), wrap(fin.t), wrap(at_j));
    });
}

// x, z, weight, ngroups, eps, norm_before_gate, stream; x of two or three dimensions
PyObject *norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 7 || !PyLong_CheckExact(a[3]) || !PyFloat_CheckExact(a[4]) || !PyBool_Check(a[5])) return none();
        const Arg x(a[0]), z(a[1]), w(a[2]);
        const int code = code_of(x);
        if (code < 0 || (x.t.dim() != 2 && x.t.dim() != 3) || x.t.numel() == 0 || !z.ok) return none();
        const bool two = x.t.dim() == 2;
        const int64_t b = two ? 1 : x.t.size(0), T = x.t.size(-2), dim = x.t.size(-1);
        if (x.t.stride(-1) != 1 || !dense(w, {dim}, at::kFloat, x.t.device())) return none();
        if (z.t.defined() && (z.t.sizes() != x.t.sizes() || z.t.scalar_type() != x.t.scalar_type() ||
                              z.t.device() != x.t.device() || z.t.stride(-1) != 1))
            return none();
        const int64_t groups = PyLong_AsLongLong(a[3]);
        if (groups == -1) {
            PyErr_Clear();
            return none();
        }
        const float eps = (float)PyFloat_AS_DOUBLE(a[4]);
        const bool norm_first = a[5] == Py_True;
        void *const stream = stream_of(a[6]);
        at::Tensor out;
        ssd_status st;
        {
            const Unlocked unlocked;
            out = at::empty(x.t.sizes(), x.t.options());
            auto bs = [&](const at::Tensor &t) { return !t.defined() || two ? 0 : t.stride(0); };
            ssd_norm_shape s = {b,           T,       dim, groups, bs(x.t), x.t.stride(-2),
                                bs(z.t), z.t.defined() ? z.t.stride(-2) : 0};
            st = g_norm(x.ptr(), z.ptr(), (const float *)w.ptr(), out.data_ptr(), eps, norm_first, &s, (ssd_dtype)code,
                        stream);
        }
        return st != SSD_OK ? PyLong_FromLong(st) : wrap(out);
    });
}

// target_probs, draft_tokens, uniforms, draft_probs, draft_lens, stream
PyObject *verify(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 6) return none();
        const Arg p(a[0]), tok(a[1]), u(a[2]), q(a[3]), lens(a[4]);
        const int code = code_of(p);
        if (code < 0 || p.t.dim() != 3 || p.t.numel() == 0) return none();
        const int64_t b = p.t.size(0), K = p.t.size(1) - 1, V = p.t.size(2);
        const auto type = p.t.scalar_type();
        const auto dev = p.t.device();
        if (!strided(p, {b, K + 1, V}, type, dev, true) || !strided(q, {b, K, V}, type, dev, false) ||
            !dense(tok, {b, K}, at::kInt, dev, true) || !dense(u, {b, K + 1}, at::kFloat, dev, true) ||
            !dense(lens, {b}, at::kInt, dev))
            return none();
        void *const stream = stream_of(a[5]);
        at::Tensor count, next, all, ws;
        ssd_status st;
        {
            const Unlocked unlocked;
            ssd_verify_shape s = {b, K, V, p.t.stride(0), p.t.stride(1), q.t.defined() ? q.t.stride(0) : 0,
                                  q.t.defined() ? q.t.stride(1) : 0};
            const size_t bytes = g_verify_bytes(&s, (ssd_dtype)code);
            const auto opt = tok.t.options();
            count = at::empty({b}, opt);
            next = at::empty({b}, opt);
            all = at::empty({b, K + 1}, opt);
            if (bytes > 0) ws = at::empty({(int64_t)bytes}, opt.dtype(at::kByte));
            st = g_verify(p.ptr(), q.ptr(), (const int32_t *)tok.ptr(), (const int32_t *)lens.ptr(),
                          (const float *)u.ptr(), (int32_t *)count.data_ptr(), (int32_t *)next.data_ptr(),
                          (int32_t *)all.data_ptr(), &s, (ssd_dtype)code, ws.defined() ? ws.data_ptr() : nullptr, bytes,
                          stream);
        }
        if (st != SSD_OK) return PyLong_FromLong(st);
        return three(wrap(count), wrap(next), wrap(all));
    });
}

// A float option given as a Python float (ints and others take the long way).
bool real(PyObject *o, float *v) {
    if (!PyFloat_CheckExact(o)) return false;
    *v = (float)PyFloat_AS_DOUBLE(o);
    return true;
}

// q, k, v, g, beta, init_state, state_out_idx, scale, qk_l2norm, final_state, return_final_state, stream
PyObject *delta(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 12 || !PyBool_Check(a[8]) || !PyBool_Check(a[10])) return none();
        const Arg q(a[0]), k(a[1]), v(a[2]), g(a[3]), beta(a[4]), init(a[5]), idx(a[6]);
        Arg fin(a[9]);
        const int code = code_of(q);
        if (code < 0 || q.t.dim() != 4 || !v.ok || !v.t.defined() || v.t.dim() != 4 || !beta.ok || !beta.t.defined())
            return none();
        const int64_t b = q.t.size(0), T = q.t.size(1), G = q.t.size(2), N = q.t.size(3), H = v.t.size(2),
                      P = v.t.size(3);
        const auto type = q.t.scalar_type();
        const auto dev = q.t.device();
        if (b == 0 || T == 0 || G == 0 || N == 0 || H == 0 || P == 0 || !strided(q, {b, T, G, N}, type, dev, true, 2) ||
            !strided(k, {b, T, G, N}, type, dev, true, 2) || !strided(v, {b, T, H, P}, type, dev, true, 2) ||
            !strided(g, {b, T, H}, at::kFloat, dev, false) || !strided(beta, {b, T, H}, at::kFloat, dev, true) ||
            !dense(init, {b, H, P, N}, at::kFloat, dev) || !dense(idx, {b}, at::kInt, dev) ||
            !dense(fin, {b, H, P, N}, at::kFloat, dev))
            return none();
        float scale;
        if (a[7] == Py_None) scale = (float)(1.0 / std::sqrt((double)N));
        else if (!real(a[7], &scale)) return none();
        const bool l2 = a[8] == Py_True, want_final = a[10] == Py_True;
        void *const stream = stream_of(a[11]);
        at::Tensor y, at_j, ws;
        ssd_status r;
        {
            const Unlocked unlocked;
            auto st = [](const Arg &t, int d) { return t.t.defined() ? t.t.stride(d) : 0; };
            ssd_delta_shape s = {b,        T,        H,        P,        N,        G,        st(q, 0),    st(q, 1),
                                 st(k, 0), st(k, 1), st(v, 0), st(v, 1), st(g, 0), st(g, 1), st(beta, 0), st(beta, 1)};
            const size_t bytes = g_delta_bytes(&s, (ssd_dtype)code);
            y = fresh({b, T, H, P}, type, dev);
            if (!fin.t.defined() && want_final) fin.t = fresh({b, H, P, N}, at::kFloat, dev);
            if (idx.t.defined()) at_j = fresh({b, H, P, N}, at::kFloat, dev);
            if (bytes > 0) ws = fresh({(int64_t)bytes}, at::kByte, dev);
            auto p = [](const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; };
            r = g_delta(q.ptr(), k.ptr(), v.ptr(), (const float *)g.ptr(), (const float *)beta.ptr(), scale, l2,
                        (const float *)init.ptr(), y.data_ptr(), (float *)fin.ptr(), (const int32_t *)idx.ptr(),
                        (float *)p(at_j), &s, (ssd_dtype)code, p(ws), bytes, stream);
        }
        if (r != SSD_OK) return PyLong_FromLong(r);
        return three(wrap(y), wrap(fin.t), wrap(at_j));
    });
}

// x, residual, weight, post_norm, post_weight, gate, gate_activation, layer_scale, residual_scale, branch_scale, eps,
// stream; x of two or three dimensions
PyObject *residual_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        float r_scale, b_scale, eps;
        if (n != 12 || !PyBool_Check(a[3]) || !real(a[8], &r_scale) || !real(a[9], &b_scale) || !real(a[10], &eps))
            return none();
        const Arg x(a[0]), res(a[1]), w(a[2]), post(a[4]), gate(a[5]), layer(a[7]);
        const int code = code_of(x);
        if (code < 0 || (x.t.dim() != 2 && x.t.dim() != 3) || x.t.numel() == 0 || !res.ok || !gate.ok) return none();
        const bool two = x.t.dim() == 2;
        const int64_t b = two ? 1 : x.t.size(0), T = x.t.size(-2), dim = x.t.size(-1);
        const auto dev = x.t.device();
        if (x.t.stride(-1) != 1 || !dense(w, {dim}, at::kFloat, dev) || !dense(post, {dim}, at::kFloat, dev) ||
            !dense(layer, {dim}, at::kFloat, dev))
            return none();
        auto like = [&](const at::Tensor &t) { return t.sizes() == x.t.sizes() && t.device() == dev && t.stride(-1) == 1; };
        auto type = x.t.scalar_type();
        if (gate.t.defined() && (!like(gate.t) || gate.t.scalar_type() != type)) return none();
        if (res.t.defined()) {
            if (!like(res.t) || (res.t.scalar_type() != type && res.t.scalar_type() != at::kFloat)) return none();
            type = res.t.scalar_type();
        }
        int act = SSD_ACT_NONE;
        if (a[6] != Py_None) {
            if (!PyUnicode_CheckExact(a[6])) return none();
            if (PyUnicode_CompareWithASCIIString(a[6], "silu") == 0) act = SSD_ACT_SILU;
            else if (PyUnicode_CompareWithASCIIString(a[6], "sigmoid") == 0) act = SSD_ACT_SIGMOID;
            else return none();
        }
        const bool post_norm = a[3] == Py_True;
        if (post.t.defined() && !post_norm) return none();
        void *const stream = stream_of(a[11]);
        at::Tensor out, h;
        ssd_status st;
        {
            const Unlocked unlocked;
            out = fresh(x.t.sizes(), x.t.scalar_type(), dev);
            h = fresh(x.t.sizes(), type, dev);
            auto bs = [&](const Arg &t) { return !t.t.defined() || two ? 0 : t.t.stride(0); };
            auto ts = [&](const Arg &t) { return t.t.defined() ? t.t.stride(-2) : 0; };
            ssd_residual_norm_shape s = {b, T, dim, bs(x), ts(x), bs(res), ts(res), bs(gate), ts(gate)};
            st = g_residual_norm(x.ptr(), res.ptr(), gate.ptr(), act, post_norm, (const float *)post.ptr(),
                                 (const float *)layer.ptr(), r_scale, b_scale, (const float *)w.ptr(), eps,
                                 out.data_ptr(), h.data_ptr(), &s, (ssd_dtype)code,
                                 type == at::kFloat ? SSD_DTYPE_F32 : SSD_DTYPE_BF16, stream);
        }
        if (st != SSD_OK) return PyLong_FromLong(st);
        PyObject *p = wrap(out), *q = wrap(h), *r = p && q ? PyTuple_Pack(2, p, q) : nullptr;
        Py_XDECREF(p);
        Py_XDECREF(q);
        return r;
    });
}

PyObject *bind_blocks(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "bind_blocks takes three addresses");
        return nullptr;
    }
    g_delta = (decltype(g_delta))PyLong_AsVoidPtr(a[0]);
    g_delta_bytes = (decltype(g_delta_bytes))PyLong_AsVoidPtr(a[1]);
    g_residual_norm = (decltype(g_residual_norm))PyLong_AsVoidPtr(a[2]);
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

// Addresses of the other C entry points, in the order of the pointers above.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
        return nullptr;
    }
    g_conv = (decltype(g_conv))PyLong_AsVoidPtr(a[0]);
    g_scan = (decltype(g_scan))PyLong_AsVoidPtr(a[1]);
    g_scan_bytes = (decltype(g_scan_bytes))PyLong_AsVoidPtr(a[2]);
    g_norm = (decltype(g_norm))PyLong_AsVoidPtr(a[3]);
    g_verify = (decltype(g_verify))PyLong_AsVoidPtr(a[4]);
    g_verify_bytes = (decltype(g_verify_bytes))PyLong_AsVoidPtr(a[5]);
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

#define FAST(f) (PyCFunction)(void (*)())f, METH_FASTCALL
PyMethodDef g_methods[] = {{"bind", FAST(bind), "addresses of the C entry points"},
                           {"bind_blocks", FAST(bind_blocks), "addresses of the gated delta rule and the residual norm"},
                           {"delta", FAST(delta), "ssd_gated_delta_fwd"},
                           {"residual_norm", FAST(residual_norm), "ssd_residual_norm_fwd"},
                           {"conv", FAST(conv), "ssd_causal_conv_fwd"},
                           {"scan", FAST(scan), "ssd_selective_scan_fwd"},
                           {"norm", FAST(norm), "ssd_gated_norm_fwd"},
                           {"verify", FAST(verify), "ssd_verify_drafts"},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fastcall", "short way through the binding", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall(void) { return PyModule_Create(&g_module); }
