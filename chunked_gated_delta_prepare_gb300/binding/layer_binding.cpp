// Python binding of libgdr's layer operators (include/gdr.h, "the layer around the recurrence"): argument checks,
// output allocation and the C ABI calls behind layer.py, which documents each function.
//
// It is native for the sake of single-token calls, whose kernels take a few microseconds: checking ten tensors and
// calling through ctypes took 13 to 21 microseconds of host time a call, here it is 4 (one output) to 7 (the norm's three).
// No arithmetic happens here.
//
// A shape, type or device that does not fit raises ValueError, a refusal of the library GdrError.  Everything runs on
// the current stream of the first tensor's device.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <array>
#include <sstream>

#include "gdr.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

// ---------------------------------------------------------------- arguments

bool is_none(PyObject* o) { return o == Py_None; }

const Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_VALUE(THPVariable_Check(o), name, ": a tensor is needed");
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
// A size as the library's 32-bit fields take it.  What does not fit stays too large for the library, which refuses it: cut
// to its lower 32 bits it could be a valid size that the outputs were not made for.
int32_t small(int64_t v) { return (int32_t)std::min<int64_t>(v, INT32_MAX); }
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v;
}

int io_of(ScalarType t) {
    if (t == at::kFloat) return GDR_F32;
    if (t == at::kBFloat16) return GDR_BF16;
    TORCH_CHECK_VALUE(t == at::kHalf, "io type ", t, ": float32, bfloat16 or float16 is needed");
    return GDR_F16;
}

[[noreturn]] void refuse(const Tensor& t, ScalarType type, IntArrayRef shape, const char* name, const char* what) {
    TORCH_CHECK_VALUE(false, name, ": a ", what, "device tensor ", shape, " of ", type, " is needed, got ", t.sizes(), " ",
                      t.scalar_type(), " on ", t.device());
    std::abort();   // not reached
}

// The checks of one call: every tensor on the device of the first.
struct Call {
    at::Device device;
    c10::cuda::OptionalCUDAGuard guard;
    ScalarType io;
    int io_code;

    explicit Call(const Tensor& first, const char* name) : device(first.device()), io(first.scalar_type()) {
        TORCH_CHECK_VALUE(device.is_cuda(), name, ": a device tensor is needed, got one on ", device);
        guard.set_device(device);
        io_code = io_of(io);
    }

    void check(const Tensor& t, ScalarType type, IntArrayRef shape, const char* name, const char* what = "") const {
        if (t.scalar_type() != type || t.device() != device || !t.sizes().equals(shape))
            refuse(t, type, shape, name, what);
    }
    // A contiguous tensor's address; nullptr for None.
    void* whole(PyObject* o, ScalarType type, IntArrayRef shape, const char* name) const {
        if (is_none(o)) return nullptr;
        const Tensor& t = tensor(o, name);
        if (!t.is_contiguous()) refuse(t, type, shape, name, "contiguous ");
        check(t, type, shape, name, "contiguous ");
        return t.data_ptr();
    }
    Tensor empty(IntArrayRef shape, ScalarType type) const {
        return at::empty(shape, at::TensorOptions().dtype(type).device(device));
    }
    void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
};

// Rows of tokens: the address of the first and the stride between them (0: contiguous).  Rows without one stride are
// copied; `copy` keeps the copy until the call is queued.
struct Rows {
    Tensor copy;
    void* p = nullptr;
    int64_t ld = 0;
};

// `inner` trailing dimensions make up a row's columns.
Rows rows(const Call& c, PyObject* o, IntArrayRef shape, const char* name, size_t inner = 1) {
    Rows r;
    if (is_none(o)) return r;
    const Tensor& t = tensor(o, name);
    c.check(t, c.io, shape, name);
    r.p = t.data_ptr();
    if (t.is_contiguous()) return r;
    const IntArrayRef st = t.strides();
    const size_t dims = shape.size(), lead = dims - inner;
    int64_t columns = 1;
    bool ok = true;
    for (size_t i = dims; i-- > lead;) {
        ok = ok && (shape[i] == 1 || st[i] == columns);
        columns *= shape[i];
    }
    int64_t inside = 0, tokens = 1;                // stride and number of the rows folded so far
    for (size_t i = lead; i-- > 0 && ok;) {
        if (shape[i] == 1) continue;
        if (inside == 0) {
            inside = st[i];
            ok = inside >= columns;
        } else {
            ok = st[i] == inside * tokens;
        }
        tokens *= shape[i];
    }
    if (ok) {
        r.ld = inside;
    } else {
        r.copy = t.contiguous();
        r.p = r.copy.data_ptr();
    }
    return r;
}

// A gradient as the library takes it: contiguous, copied if need be.  Undefined for None.
Tensor gradient(const Call& c, PyObject* o, ScalarType type, IntArrayRef shape, const char* name) {
    if (is_none(o)) return Tensor();
    const Tensor& t = tensor(o, name);
    c.check(t, type, shape, name);
    return t.contiguous();
}

void* at_or_null(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// The caller's workspace, or a new one of `need` bytes.
struct Workspace {
    Tensor t;
    void* p = nullptr;
    size_t bytes = 0;
    Workspace(const Call& c, PyObject* given, size_t need) {
        if (!is_none(given)) {
            t = tensor(given, "workspace");
            TORCH_CHECK_VALUE(t.device() == c.device && t.is_contiguous(), "workspace: a contiguous device tensor is needed");
            p = t.data_ptr();
            bytes = t.nbytes();
        } else if (need) {
            t = c.empty({(int64_t)need}, at::kByte);
            p = t.data_ptr();
            bytes = need;
        }
    }
};

// Packed or batched sequences: the tokens of x [B, T, D], or packed x [total, D] with cu_seqlens [n + 1].
struct Sequences {
    int64_t n, T = 0, total = 0;
    const int32_t* cu = nullptr;
    Sequences(const Call& c, const Tensor& x, PyObject* cu_seqlens) {
        if (is_none(cu_seqlens)) {
            TORCH_CHECK_VALUE(x.dim() == 3 && x.size(0) > 0 && x.size(1) > 0, "x: [B, T, D] is needed, got ", x.sizes());
            n = x.size(0);
            T = x.size(1);
        } else {
            TORCH_CHECK_VALUE(x.dim() == 2, "x: packed tokens [total, D] are needed with cu_seqlens, got ", x.sizes());
            const Tensor& t = tensor(cu_seqlens, "cu_seqlens");
            TORCH_CHECK_VALUE(t.dim() == 1 && t.numel() >= 2, "cu_seqlens: [n + 1] entries are needed");
            cu = (const int32_t*)c.whole(cu_seqlens, at::kInt, t.sizes(), "cu_seqlens");
            n = t.numel() - 1;
            total = x.size(0);
        }
    }
};

// ---------------------------------------------------------------- results

PyObject* gdr_error(int status, const char* where) {
    PyObject* m = PyImport_ImportModule("chunked_gated_delta_prepare_gb300.gdr");
    PyObject* type = m ? PyObject_GetAttrString(m, "GdrError") : nullptr;
    PyObject* e = type ? PyObject_CallFunction(type, "is", status, where) : nullptr;
    if (e) PyErr_SetObject(type, e);
    Py_XDECREF(e);
    Py_XDECREF(type);
    Py_XDECREF(m);
    return nullptr;
}

PyObject* wrap(const Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

template <size_t N> PyObject* results(const std::array<Tensor, N>& ts) {
    PyObject* r = PyTuple_New(N);
    if (!r) throw python_error();
    for (size_t i = 0; i < N; ++i) PyTuple_SET_ITEM(r, i, wrap(ts[i]));
    return r;
}

// The number of arguments is layer.py's to get right; a mistake there must not read past them.
void expect(Py_ssize_t got, Py_ssize_t want) { TORCH_CHECK(got == want, "layer binding: ", want, " arguments, got ", got); }

constexpr auto F32 = at::kFloat;

// ---------------------------------------------------------------- root-mean-square norm

// x, weight, residual, eps, group (-1: no 8-bit output, 0: a scale a row), want_y -> y, r, y8, scales
PyObject* norm_forward(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    expect(count, 6);
    const Tensor& x = tensor(a[0], "x");
    const Call c(x, "x");
    const IntArrayRef shape = x.sizes();
    TORCH_CHECK_VALUE(x.dim() >= 1, "x: [..., D] is needed");
    const int64_t D = shape.back(), group = integer(a[4]);
    const Rows xr = rows(c, a[0], shape, "x"), res = rows(c, a[2], shape, "residual");
    void* w = c.whole(a[1], c.io, {D}, "weight");
    const gdr_norm_problem p{D ? x.numel() / D : 0, D, xr.ld, res.ld, c.io_code, small(std::max<int64_t>(group, 0)),
                             (float)real(a[3])};
    std::array<Tensor, 4> out;
    if (truth(a[5])) out[0] = c.empty(shape, c.io);
    if (res.p || (!is_none(a[2]) && x.numel() == 0)) out[1] = c.empty(shape, c.io);
    if (group >= 0) {
        out[2] = c.empty(shape, at::kFloat8_e4m3fn);
        std::vector<int64_t> s(shape.begin(), shape.end());
        s.back() = group ? (D - 1) / group + 1 : 1;
        out[3] = c.empty(s, F32);
    }
    const int st = gdr_norm_forward(&p, xr.p, res.p, w, at_or_null(out[0]), at_or_null(out[1]), at_or_null(out[2]),
                                    (float*)at_or_null(out[3]), c.stream());
    return st ? gdr_error(st, "gdr_norm_forward") : results(out);
    END_HANDLE_TH_ERRORS
}

// dy, r, weight, d_r, eps, workspace -> dx, dweight
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    expect(count, 6);
    const Call c(tensor(a[1], "r"), "r");
    const IntArrayRef shape = tensor(a[1], "r").sizes();
    TORCH_CHECK_VALUE(shape.size() >= 1, "r: [..., D] is needed");
    const int64_t D = shape.back();
    const Tensor dy = gradient(c, a[0], c.io, shape, "dy"), r = gradient(c, a[1], c.io, shape, "r"),
                 dr = gradient(c, a[3], c.io, shape, "d_r");
    TORCH_CHECK_VALUE(dy.defined(), "dy: a tensor is needed");
    void* w = c.whole(a[2], c.io, {D}, "weight");
    const gdr_norm_problem p{D ? r.numel() / D : 0, D, 0, 0, c.io_code, 0, (float)real(a[4])};
    const std::array<Tensor, 2> out{c.empty(shape, c.io), c.empty({D}, F32)};
    const Workspace ws(c, a[5], gdr_norm_backward_workspace_bytes(&p));
    const int st = gdr_norm_backward(&p, dy.data_ptr(), r.data_ptr(), w, at_or_null(dr), out[0].data_ptr(),
                                     (float*)out[1].data_ptr(), ws.p, ws.bytes, c.stream());
    return st ? gdr_error(st, "gdr_norm_backward") : results(out);
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- short causal convolution

struct Conv {
    const Tensor& x;
    Call c;
    Sequences q;
    Rows xr;
    const void *w, *b;
    gdr_conv_problem p;
    std::array<int64_t, 3> states;

    Conv(PyObject* x_, PyObject* weight, PyObject* bias, PyObject* silu, PyObject* cu)
        : x(tensor(x_, "x")), c(x, "x"), q(c, x, cu), xr(rows(c, x_, x.sizes(), "x")) {
        const Tensor& wt = tensor(weight, "weight");
        TORCH_CHECK_VALUE(wt.dim() == 2, "weight: [D, W] is needed, got ", wt.sizes());
        const int64_t D = x.sizes().back(), W = wt.size(1);
        w = c.whole(weight, c.io, {D, W}, "weight");
        b = c.whole(bias, c.io, {D}, "bias");
        p = gdr_conv_problem{q.n, q.T, q.total, D, xr.ld, 0, small(W), c.io_code, truth(silu)};
        states = {q.n, W - 1, D};
    }
};

// x, weight, bias, state, silu, cu_seqlens, want_state -> y, state_out
PyObject* conv_forward(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    expect(count, 7);
    const Conv v(a[0], a[1], a[2], a[4], a[5]);
    const Call& c = v.c;
    void* state = c.whole(a[3], c.io, v.states, "state");
    std::array<Tensor, 2> out{c.empty(v.x.sizes(), c.io), Tensor()};
    // W - 1 < 0 cannot be allocated; the library refuses it below
    if (truth(a[6]) && v.states[1] > 0) out[1] = c.empty(v.states, c.io);
    const int st = gdr_conv_forward(&v.p, v.q.cu, v.xr.p, v.w, v.b, state, out[0].data_ptr(), at_or_null(out[1]),
                                    c.stream());
    return st ? gdr_error(st, "gdr_conv_forward") : results(out);
    END_HANDLE_TH_ERRORS
}

// x, weight, bias, dy, state, d_state_out, silu, cu_seqlens, workspace -> dx, dweight, dbias, dstate
PyObject* conv_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    expect(count, 9);
    const Conv v(a[0], a[1], a[2], a[6], a[7]);
    const Call& c = v.c;
    void* state = c.whole(a[4], c.io, v.states, "state");
    const Tensor dy = gradient(c, a[3], c.io, v.x.sizes(), "dy"), dout = gradient(c, a[5], c.io, v.states, "d_state_out");
    TORCH_CHECK_VALUE(dy.defined(), "dy: a tensor is needed");
    std::array<Tensor, 4> out{c.empty(v.x.sizes(), c.io), c.empty({v.p.D, v.p.W}, F32), c.empty({v.p.D}, F32), Tensor()};
    if (state) out[3] = c.empty(v.states, c.io);
    const Workspace ws(c, a[8], gdr_conv_backward_workspace_bytes(&v.p, v.q.cu != nullptr));
    const int st = gdr_conv_backward(&v.p, v.q.cu, v.xr.p, v.w, v.b, state, dy.data_ptr(), at_or_null(dout),
                                     out[0].data_ptr(), (float*)out[1].data_ptr(), (float*)out[2].data_ptr(),
                                     at_or_null(out[3]), ws.p, ws.bytes, c.stream());
    if (st) return gdr_error(st, "gdr_conv_backward");
    if (!v.b) out[2] = Tensor();
    return results(out);
    END_HANDLE_TH_ERRORS
}

// x, weight, bias, state, silu, slots -> y
PyObject* conv_step(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    expect(count, 6);
    const Tensor &x = tensor(a[0], "x"), &wt = tensor(a[1], "weight"), &state = tensor(a[3], "state");
    TORCH_CHECK_VALUE(x.dim() == 2 && wt.dim() == 2 && state.dim() == 3,
                      "x [n, D], weight [D, W] and state [pool, W - 1, D] are needed");
    const Call c(x, "x");
    const int64_t n = x.size(0), D = x.size(1), W = wt.size(1), pool = state.size(0);
    const Rows xr = rows(c, a[0], x.sizes(), "x");
    const gdr_conv_problem p{n, 1, 0, D, xr.ld, pool, small(W), c.io_code, truth(a[4])};
    void *w = c.whole(a[1], c.io, {D, W}, "weight"), *b = c.whole(a[2], c.io, {D}, "bias"),
         *h = c.whole(a[3], c.io, {pool, W - 1, D}, "state");
    const int32_t* slots = (const int32_t*)c.whole(a[5], at::kInt, {n}, "slots");
    const Tensor y = c.empty({n, D}, c.io);
    const int st = gdr_conv_step(&p, slots, xr.p, w, b, h, y.data_ptr(), c.stream());
    return st ? gdr_error(st, "gdr_conv_step") : wrap(y);
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- selective state space scan

struct Scan {
    Rows x, dt, z, B, C;
    const float *A, *D, *bias;
    gdr_ssm_problem p;

    Scan(const Call& c, const Tensor& xt, PyObject* const* a, PyObject* D_, PyObject* z_, PyObject* bias_, PyObject* softplus,
         int64_t n, int64_t T, int64_t total, int64_t pool) {
        const Tensor &At = tensor(a[2], "A"), &Bt = tensor(a[3], "B");
        const IntArrayRef shape = xt.sizes();
        TORCH_CHECK_VALUE(At.dim() == 2 && Bt.dim() == xt.dim() + 1, "A [D, N] and B [..., G, N] are needed");
        const int64_t ch = shape.back(), G = Bt.size(-2), N = Bt.size(-1);
        c10::SmallVector<int64_t, 5> bc(shape.begin(), shape.end() - 1);
        bc.push_back(G);
        bc.push_back(N);
        x = rows(c, a[0], shape, "x");
        dt = rows(c, a[1], shape, "dt");
        TORCH_CHECK_VALUE(!is_none(a[1]), "dt: a tensor is needed");
        z = rows(c, z_, shape, "z");
        B = rows(c, a[3], bc, "B", 2);
        C = rows(c, a[4], bc, "C", 2);
        TORCH_CHECK_VALUE(!is_none(a[4]), "C: a tensor is needed");
        A = (const float*)c.whole(a[2], F32, {ch, N}, "A");
        D = (const float*)c.whole(D_, F32, {ch}, "D");
        bias = (const float*)c.whole(bias_, F32, {ch}, "dt_bias");
        p = gdr_ssm_problem{n,    T,    total, ch,   N,    G,         x.ld,           dt.ld,
                            z.ld, B.ld, C.ld,  pool, c.io_code, truth(softplus)};
    }
};

// x, dt, A, B, C, D, z, dt_bias, h0, softplus, cu_seqlens, want_h_final, workspace -> y, h_final
PyObject* ssm_forward(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    expect(count, 13);
    const Tensor& x = tensor(a[0], "x");
    const Call c(x, "x");
    const Sequences q(c, x, a[10]);
    const Scan s(c, x, a, a[5], a[6], a[7], a[9], q.n, q.T, q.total, 0);
    const std::array<int64_t, 3> states{q.n, s.p.D, s.p.N};
    const float* h0 = (const float*)c.whole(a[8], F32, states, "h0");
    std::array<Tensor, 2> out{c.empty(x.sizes(), c.io), Tensor()};
    if (truth(a[11])) out[1] = c.empty(states, F32);
    const Workspace ws(c, a[12], gdr_ssm_forward_workspace_bytes(&s.p, q.cu != nullptr));
    const int st = gdr_ssm_forward(&s.p, q.cu, s.x.p, s.dt.p, s.A, s.B.p, s.C.p, s.D, s.z.p, s.bias, h0,
                                   out[0].data_ptr(), (float*)at_or_null(out[1]), ws.p, ws.bytes, c.stream());
    return st ? gdr_error(st, "gdr_ssm_forward") : results(out);
    END_HANDLE_TH_ERRORS
}

// x, dt, A, B, C, dy, D, z, dt_bias, h0, dh_final, softplus, cu_seqlens, workspace
//   -> dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0
PyObject* ssm_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    expect(count, 14);
    const Tensor& x = tensor(a[0], "x");
    const Call c(x, "x");
    const Sequences q(c, x, a[12]);
    const Scan s(c, x, a, a[6], a[7], a[8], a[11], q.n, q.T, q.total, 0);
    const std::array<int64_t, 3> states{q.n, s.p.D, s.p.N};
    const IntArrayRef shape = x.sizes(), bc = tensor(a[3], "B").sizes();
    const float* h0 = (const float*)c.whole(a[9], F32, states, "h0");
    const Tensor dy = gradient(c, a[5], c.io, shape, "dy"), dh = gradient(c, a[10], F32, states, "dh_final");
    TORCH_CHECK_VALUE(dy.defined(), "dy: a tensor is needed");
    std::array<Tensor, 9> out{c.empty(shape, c.io), c.empty(shape, c.io), c.empty({s.p.D, s.p.N}, F32), c.empty(bc, c.io),
                              c.empty(bc, c.io)};
    if (s.D) out[5] = c.empty({s.p.D}, F32);
    if (!is_none(a[7])) out[6] = c.empty(shape, c.io);
    if (s.bias) out[7] = c.empty({s.p.D}, F32);
    if (h0) out[8] = c.empty(states, F32);
    const Workspace ws(c, a[13], gdr_ssm_backward_workspace_bytes(&s.p, q.cu != nullptr));
    const int st = gdr_ssm_backward(&s.p, q.cu, s.x.p, s.dt.p, s.A, s.B.p, s.C.p, s.D, s.z.p, s.bias, h0, dy.data_ptr(),
                                    (const float*)at_or_null(dh), out[0].data_ptr(), out[1].data_ptr(),
                                    (float*)out[2].data_ptr(), out[3].data_ptr(), out[4].data_ptr(),
                                    (float*)at_or_null(out[5]), at_or_null(out[6]), (float*)at_or_null(out[7]),
                                    (float*)at_or_null(out[8]), ws.p, ws.bytes, c.stream());
    return st ? gdr_error(st, "gdr_ssm_backward") : results(out);
    END_HANDLE_TH_ERRORS
}

// x, dt, A, B, C, h, D, z, dt_bias, softplus, slots -> y
PyObject* ssm_step(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    expect(count, 11);
    const Tensor &x = tensor(a[0], "x"), &h = tensor(a[5], "h");
    TORCH_CHECK_VALUE(x.dim() == 2 && h.dim() == 3, "x [n, D] and h [pool, D, N] are needed");
    const Call c(x, "x");
    const int64_t n = x.size(0), pool = h.size(0);
    const Scan s(c, x, a, a[6], a[7], a[8], a[9], n, 1, 0, pool);
    float* hp = (float*)c.whole(a[5], F32, {pool, s.p.D, s.p.N}, "h");
    const int32_t* slots = (const int32_t*)c.whole(a[10], at::kInt, {n}, "slots");
    const Tensor y = c.empty(x.sizes(), c.io);
    const int st = gdr_ssm_step(&s.p, slots, s.x.p, s.dt.p, s.A, s.B.p, s.C.p, s.D, s.z.p, s.bias, hp, y.data_ptr(),
                                c.stream());
    return st ? gdr_error(st, "gdr_ssm_step") : wrap(y);
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- the gated delta rule, one token

// q, k, v, g, beta, h, scale, slots -> o
PyObject* delta_step(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    expect(count, 8);
    const Tensor &qt = tensor(a[0], "q"), &vt = tensor(a[2], "v"), &gt = tensor(a[3], "g"), &ht = tensor(a[5], "h");
    TORCH_CHECK_VALUE(qt.dim() == 3 && vt.dim() == 3 && ht.dim() == 4,
                      "q [B, H, K], v [B, HV, V] and h [pool, HV, K, V] are needed");
    const Call c(qt, "q");
    const int64_t B = qt.size(0), H = qt.size(1), K = qt.size(2), HV = vt.size(1), V = vt.size(2), pool = ht.size(0);
    const Rows q = rows(c, a[0], {B, H, K}, "q", 2), k = rows(c, a[1], {B, H, K}, "k", 2),
               v = rows(c, a[2], {B, HV, V}, "v", 2);
    const bool per_k = gt.dim() == 3;
    const gdr_step_problem p{B, H, HV, K, V, pool, q.ld, k.ld, v.ld, c.io_code, per_k, is_none(a[6]) ? -1.f : (float)real(a[6])};
    const std::array<int64_t, 3> gk{B, HV, K};
    const float* g = (const float*)c.whole(a[3], F32, IntArrayRef(gk.data(), per_k ? 3 : 2), "g");
    void* beta = c.whole(a[4], c.io, {B, HV}, "beta");
    float* h = (float*)c.whole(a[5], F32, {pool, HV, K, V}, "h");
    const int32_t* slots = (const int32_t*)c.whole(a[7], at::kInt, {B}, "slots");
    const Tensor o = c.empty({B, HV, V}, c.io);
    const int st = gdr_delta_step(&p, slots, q.p, k.p, v.p, g, beta, h, o.data_ptr(), c.stream());
    return st ? gdr_error(st, "gdr_delta_step") : wrap(o);
    END_HANDLE_TH_ERRORS
}

#define GDR_METHOD(name) {#name, (PyCFunction)(void*)name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GDR_METHOD(norm_forward), GDR_METHOD(norm_backward), GDR_METHOD(conv_forward),
                         GDR_METHOD(conv_backward), GDR_METHOD(conv_step), GDR_METHOD(ssm_forward),
                         GDR_METHOD(ssm_backward), GDR_METHOD(ssm_step), GDR_METHOD(delta_step), {}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdr_layer", "Argument checks and calls behind layer.py.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__gdr_layer() { return PyModule_Create(&module); }
