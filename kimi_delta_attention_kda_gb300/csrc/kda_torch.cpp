// kda_torch.cpp -- the operators around the prefill on PyTorch tensors: a
// CPython module that checks the arguments, takes new outputs from PyTorch's
// allocator and calls the C entry points of libkda.so (include/kda.h).
//
// For one token the call costs more than the kernel: through ctypes, with the
// checks in Python, la_decode of one sequence took 12.5 us on the host, here 4.0.
//
// Each function returns its output (or a tuple of them), the library's error
// code as an int, or None where an argument is not what it should be: ops.py,
// its only caller, then finds the fault and names it.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/kda.h"

namespace {

constexpr int64_t kDim = 128;
constexpr auto kBF16 = at::kBFloat16, kF32 = at::kFloat;

// libkda.so's entry points, in this order from bind().
decltype(&kda_la_prefill) la_prefill_fn = nullptr;
decltype(&kda_la_decode) la_decode_fn = nullptr;
decltype(&kda_decode) decode_fn = nullptr;
decltype(&kda_gated_norm) gated_norm_fn = nullptr;
decltype(&kda_residual_norm) residual_norm_fn = nullptr;

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 5) return PyErr_Format(PyExc_TypeError, "five addresses expected");
    void* p[5];
    for (int i = 0; i < 5; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(a[i]))) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "null address");
    la_prefill_fn = reinterpret_cast<decltype(la_prefill_fn)>(p[0]);
    la_decode_fn = reinterpret_cast<decltype(la_decode_fn)>(p[1]);
    decode_fn = reinterpret_cast<decltype(decode_fn)>(p[2]);
    gated_norm_fn = reinterpret_cast<decltype(gated_norm_fn)>(p[3]);
    residual_norm_fn = reinterpret_cast<decltype(residual_norm_fn)>(p[4]);
    Py_RETURN_NONE;
}

// The convolution's and the scan's, in this order from bind_scan().
decltype(&kda_conv_prefill) conv_prefill_fn = nullptr;
decltype(&kda_conv_decode) conv_decode_fn = nullptr;
decltype(&kda_ssm_prefill) ssm_prefill_fn = nullptr;
decltype(&kda_ssm_decode) ssm_decode_fn = nullptr;

PyObject* bind_scan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 4) return PyErr_Format(PyExc_TypeError, "four addresses expected");
    void* p[4];
    for (int i = 0; i < 4; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(a[i]))) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "null address");
    conv_prefill_fn = reinterpret_cast<decltype(conv_prefill_fn)>(p[0]);
    conv_decode_fn = reinterpret_cast<decltype(conv_decode_fn)>(p[1]);
    ssm_prefill_fn = reinterpret_cast<decltype(ssm_prefill_fn)>(p[2]);
    ssm_decode_fn = reinterpret_cast<decltype(ssm_decode_fn)>(p[3]);
    Py_RETURN_NONE;
}
bool bound(const void* fn) {
    if (!fn) PyErr_SetString(PyExc_RuntimeError, "the module is not bound to the library");
    return fn;
}

// A tensor argument; null for None and for anything else.
const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }
void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// The arguments of a call, checked one after the other.
struct Args {
    bool ok;
    int dev;
    explicit Args(const at::Tensor* first) : ok(first && first->is_cuda()), dev(ok ? first->get_device() : -1) {
        ok = ok && c10::cuda::current_device() == dev;
    }
    void want(bool x) { ok = ok && x; }
    void need(const at::Tensor* t, at::ScalarType type, at::IntArrayRef shape) {
        ok = ok && t && t->is_cuda() && t->get_device() == dev && t->scalar_type() == type && t->sizes() == shape &&
             t->is_contiguous();
    }
    // FP32 or BF16.
    void need_float(const at::Tensor* t, at::IntArrayRef shape) {
        if (ok && t) need(t, t->scalar_type() == kF32 ? kF32 : kBF16, shape);
        want(t);
    }
    // A contiguous row of the last `inner` sizes for each token, where the sizes
    // before are tokens; rows lie *ld elements apart, a row's width at least.
    void need_rows(const at::Tensor* t, at::ScalarType type, at::IntArrayRef shape, int inner, int64_t* ld) {
        ok = ok && t && t->is_cuda() && t->get_device() == dev && t->scalar_type() == type && t->sizes() == shape;
        if (!ok) return;
        const int dims = static_cast<int>(shape.size()), lead = dims - inner;
        int64_t width = 1, rows = 1, step = 0;
        if (t->numel() == 0) {   // no element has an address
            for (int i = lead; i < dims; ++i) width *= shape[i];
            *ld = width;
            return;
        }
        for (int i = dims - 1; i >= lead; --i) {
            ok = ok && (shape[i] == 1 || t->stride(i) == width);
            width *= shape[i];
        }
        for (int i = lead - 1; i >= 0; --i) {
            if (shape[i] == 1) continue;
            if (rows == 1)
                step = t->stride(i);
            else
                ok = ok && t->stride(i) == rows * step;
            rows *= shape[i];
        }
        *ld = rows > 1 ? step : width;
        ok = ok && *ld >= width;
    }
    // The same, BF16 or FP32.
    void need_rows_float(const at::Tensor* t, at::IntArrayRef shape, int inner, int64_t* ld) {
        if (ok && t) need_rows(t, t->scalar_type() == kF32 ? kF32 : kBF16, shape, inner, ld);
        want(t);
    }
    // None, or as need().
    void may(PyObject* o, const at::Tensor* t, at::ScalarType type, at::IntArrayRef shape) {
        if (o != Py_None) need(t, type, shape);
    }
    bool dims(const at::Tensor* t, int64_t n) {
        want(t && t->dim() == n);
        return ok;
    }
};

bool fp32(const at::Tensor* t) { return t && t->scalar_type() == kF32; }

// The stream's handle, or the current stream for None.
bool stream_of(PyObject* o, int dev, void** stream) {
    if (o == Py_None) {
        *stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
        return true;
    }
    *stream = PyLong_AsVoidPtr(o);
    return !PyErr_Occurred();
}
bool number(PyObject* o, double* x) {
    *x = PyFloat_AsDouble(o);
    return *x != -1.0 || !PyErr_Occurred();
}
// An argument's truth value, before anything runs: taking it may raise.
bool truth(PyObject* o, bool* x) {
    const int r = PyObject_IsTrue(o);
    *x = r > 0;
    return r >= 0;
}
bool counted(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments expected", want);
    return n == want;
}
// Other Python threads run while new outputs are allocated and the library is
// called: either may wait for the GPU (a pool that grows, a full launch queue,
// a device's set-up at its first call).  Nothing of Python is touched meanwhile.
class Released {
public:
    Released() : state_(PyEval_SaveThread()) {}
    ~Released() { PyEval_RestoreThread(state_); }
    Released(const Released&) = delete;
    Released& operator=(const Released&) = delete;

private:
    PyThreadState* state_;
};
template <class F>
int released(F f) {
    Released r;
    return f();
}
at::Tensor fresh(const at::Tensor& like) { return at::empty(like.sizes(), like.options()); }

PyObject* result(int rc, PyObject* given, const at::Tensor& out) {
    if (rc != KDA_OK) return PyLong_FromLong(rc);
    return given != Py_None ? Py_NewRef(given) : THPVariable_Wrap(out);
}
// A tuple of two results, which it takes over.
PyObject* two(PyObject* x, PyObject* y) {
    PyObject* both = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return both;
}

// q, k, v, g, init_state, cu_seqlens, out, final_state, want_final, state_fp32, scale, stream
PyObject* la_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!counted(n, 12)) return nullptr;
    const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *g = tensor(a[3]), *init = tensor(a[4]),
                     *cu = tensor(a[5]), *out = tensor(a[6]), *fin = tensor(a[7]);
    Args c(q);
    if (!c.dims(q, 4) || !c.dims(v, 4) || !g) Py_RETURN_NONE;
    const int64_t B = v->size(0), T = v->size(1), H = v->size(2), Hk = q->size(2);
    c.want(Hk > 0 && H % Hk == 0);
    c.need(q, kBF16, {B, T, Hk, kDim});
    c.need(k, kBF16, {B, T, Hk, kDim});
    c.need(v, kBF16, {B, T, H, kDim});
    if (g->dim() == 1)
        c.need(g, kF32, {H});
    else
        c.need(g, kF32, {B, T, H});
    int64_t N = B;
    if (a[5] != Py_None) {
        c.want(cu && B == 1 && cu->numel() > 0);
        if (!c.ok) Py_RETURN_NONE;
        N = cu->numel() - 1;
        c.need(cu, at::kLong, {N + 1});
    }
    bool f32, want_final;
    if (!truth(a[9], &f32) || !truth(a[8], &want_final)) return nullptr;
    const int64_t shape[] = {N, H, kDim, kDim};
    if (a[4] != Py_None) {
        c.need_float(init, shape);
        f32 = fp32(init);
    } else if (a[7] != Py_None) {
        c.need_float(fin, shape);
        f32 = fp32(fin);
    }
    c.may(a[7], fin, f32 ? kF32 : kBF16, shape);
    c.may(a[6], out, kBF16, v->sizes());
    if (!c.ok) Py_RETURN_NONE;
    void* stream;
    double scale;
    if (!stream_of(a[11], c.dev, &stream) || !number(a[10], &scale)) return nullptr;
    at::Tensor new_out, new_fin;
    want_final = want_final || fin;
    const int rc = released([&] {
        if (!out) out = &(new_out = fresh(*v));
        if (!fin && want_final) fin = &(new_fin = at::empty(shape, q->options().dtype(f32 ? kF32 : kBF16)));
        return la_prefill_fn(ptr(q), ptr(k), ptr(v), static_cast<const float*>(ptr(g)), ptr(init), ptr(out), ptr(fin), N, T, H,
                             Hk, static_cast<const int64_t*>(ptr(cu)), static_cast<float>(scale),
                             (f32 ? KDA_FLAG_STATE_F32 : 0u) | (g->dim() == 1 ? KDA_FLAG_G_PER_HEAD : 0u), stream);
    });
    if (rc != KDA_OK) return PyLong_FromLong(rc);
    return two(result(rc, a[6], new_out), !want_final ? Py_NewRef(Py_None) : result(rc, a[7], new_fin));
    END_HANDLE_TH_ERRORS
}

// The arguments that both steps share: q, k, v, state, slots, out.
bool step_args(Args& c, const at::Tensor* q, const at::Tensor* k, const at::Tensor* v, const at::Tensor* state,
               PyObject* slots_o, const at::Tensor* slots, PyObject* out_o, const at::Tensor* out) {
    if (!c.dims(q, 3) || !c.dims(v, 3) || !c.dims(state, 4)) return false;
    const int64_t N = q->size(0), Hk = q->size(1), H = v->size(1), pool = state->size(0);
    c.want(Hk > 0 && H % Hk == 0);
    c.need(q, kBF16, {N, Hk, kDim});
    c.need(k, kBF16, {N, Hk, kDim});
    c.need(v, kBF16, {N, H, kDim});
    c.need_float(state, {pool, H, kDim, kDim});
    if (slots_o == Py_None)
        c.want(N <= pool);
    else
        c.need(slots, at::kInt, {N});
    c.may(out_o, out, kBF16, {N, H, kDim});
    return c.ok;
}

// q, k, v, g, state, slots, out, scale, stream
PyObject* la_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!counted(n, 9)) return nullptr;
    const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *g = tensor(a[3]), *state = tensor(a[4]),
                     *slots = tensor(a[5]), *out = tensor(a[6]);
    Args c(q);
    if (!step_args(c, q, k, v, state, a[5], slots, a[6], out) || !g) Py_RETURN_NONE;
    const int64_t N = q->size(0), H = v->size(1);
    if (g->dim() == 1)
        c.need(g, kF32, {H});
    else
        c.need(g, kF32, {N, H});
    if (!c.ok) Py_RETURN_NONE;
    void* stream;
    double scale;
    if (!stream_of(a[8], c.dev, &stream) || !number(a[7], &scale)) return nullptr;
    at::Tensor made;
    const int rc = released([&] {
        if (!out) out = &(made = fresh(*v));
        return la_decode_fn(ptr(q), ptr(k), ptr(v), static_cast<const float*>(ptr(g)), ptr(state),
                            static_cast<const int32_t*>(ptr(slots)), ptr(out), N, H, q->size(1), state->size(0),
                            static_cast<float>(scale),
                            (fp32(state) ? KDA_FLAG_STATE_F32 : 0u) | (g->dim() == 1 ? KDA_FLAG_G_PER_HEAD : 0u), stream);
    });
    return result(rc, a[6], made);
    END_HANDLE_TH_ERRORS
}

// q, k, v, g, beta, state, slots, out, beta_is_logit, stream
PyObject* kda_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!counted(n, 10)) return nullptr;
    const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *g = tensor(a[3]), *beta = tensor(a[4]),
                     *state = tensor(a[5]), *slots = tensor(a[6]), *out = tensor(a[7]);
    Args c(q);
    if (!step_args(c, q, k, v, state, a[6], slots, a[7], out)) Py_RETURN_NONE;
    const int64_t N = q->size(0), H = v->size(1);
    c.want(q->size(1) == H);
    c.need(g, kF32, {N, H, kDim});
    c.need(beta, kBF16, {N, H});
    if (!c.ok) Py_RETURN_NONE;
    void* stream;
    bool logit;
    if (!stream_of(a[9], c.dev, &stream) || !truth(a[8], &logit)) return nullptr;
    at::Tensor made;
    const int rc = released([&] {
        if (!out) out = &(made = fresh(*v));
        return decode_fn(ptr(q), ptr(k), ptr(v), static_cast<const float*>(ptr(g)), ptr(beta), ptr(state),
                         static_cast<const int32_t*>(ptr(slots)), ptr(out), N, H, state->size(0),
                         (fp32(state) ? KDA_FLAG_STATE_F32 : 0u) | (logit ? KDA_FLAG_BETA_LOGIT : 0u), stream);
    });
    return result(rc, a[7], made);
    END_HANDLE_TH_ERRORS
}

// x, weight, gate, activation, gate_first, eps, out, stream
PyObject* gated_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!counted(n, 8)) return nullptr;
    const at::Tensor *x = tensor(a[0]), *weight = tensor(a[1]), *gate = tensor(a[2]), *out = tensor(a[6]);
    Args c(x);
    c.want(x && x->dim() > 0 && x->size(-1) == kDim);
    if (!c.ok) Py_RETURN_NONE;
    const long act = PyLong_AsLong(a[3]);
    c.need(x, kBF16, x->sizes());
    c.need_float(weight, {kDim});
    if (act) c.need(gate, kBF16, x->sizes());
    c.may(a[6], out, kBF16, x->sizes());
    if (!c.ok) Py_RETURN_NONE;
    void* stream;
    double eps;
    bool first;
    if (!stream_of(a[7], c.dev, &stream) || !number(a[5], &eps) || !truth(a[4], &first)) return nullptr;
    at::Tensor made;
    const int rc = released([&] {
        if (!out) out = &(made = fresh(*x));
        return gated_norm_fn(ptr(x), ptr(weight), act ? ptr(gate) : nullptr, ptr(out), x->numel() / kDim, static_cast<int>(act),
                             static_cast<float>(eps),
                             (fp32(weight) ? KDA_FLAG_WEIGHT_F32 : 0u) | (first ? KDA_FLAG_GATE_FIRST : 0u), stream);
    });
    return result(rc, a[6], made);
    END_HANDLE_TH_ERRORS
}

// x, residual, weight, post_weight, gate, scale, eps, out, residual_out, stream
PyObject* residual_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!counted(n, 10)) return nullptr;
    const at::Tensor *x = tensor(a[0]), *residual = tensor(a[1]), *weight = tensor(a[2]), *post = tensor(a[3]),
                     *gate = tensor(a[4]), *out = tensor(a[7]), *rout = tensor(a[8]);
    Args c(x);
    c.want(x && x->dim() > 0 && x->size(-1) > 0);
    if (!c.ok) Py_RETURN_NONE;
    const int64_t D = x->size(-1);
    c.need(x, kBF16, x->sizes());
    c.need_float(residual, x->sizes());
    c.need_float(weight, {D});
    if (!c.ok) Py_RETURN_NONE;
    c.may(a[3], post, weight->scalar_type(), {D});
    c.may(a[4], gate, weight->scalar_type(), {D});
    c.may(a[7], out, kBF16, x->sizes());
    c.may(a[8], rout, residual->scalar_type(), x->sizes());
    if (!c.ok) Py_RETURN_NONE;
    void* stream;
    double scale, eps;
    if (!stream_of(a[9], c.dev, &stream) || !number(a[5], &scale) || !number(a[6], &eps)) return nullptr;
    at::Tensor made, rmade;
    const int rc = released([&] {
        if (!out) out = &(made = fresh(*x));
        if (!rout) rout = &(rmade = fresh(*residual));
        return residual_norm_fn(ptr(x), ptr(residual), ptr(weight), ptr(post), ptr(gate), ptr(out), ptr(rout), x->numel() / D, D,
                                static_cast<float>(scale), static_cast<float>(eps),
                                (fp32(weight) ? KDA_FLAG_WEIGHT_F32 : 0u) | (fp32(residual) ? KDA_FLAG_RESIDUAL_F32 : 0u),
                                stream);
    });
    if (rc != KDA_OK) return PyLong_FromLong(rc);
    return two(result(rc, a[7], made), result(rc, a[8], rmade));
    END_HANDLE_TH_ERRORS
}

// x, weight, bias, init_state, cu_seqlens, silu, out, final_state, want_final, stream
PyObject* conv_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!counted(n, 10) || !bound(reinterpret_cast<void*>(conv_prefill_fn))) return nullptr;
    const at::Tensor *x = tensor(a[0]), *weight = tensor(a[1]), *bias = tensor(a[2]), *init = tensor(a[3]), *cu = tensor(a[4]),
                     *out = tensor(a[6]), *fin = tensor(a[7]);
    Args c(x);
    if (!c.dims(x, 3) || !c.dims(weight, 2)) Py_RETURN_NONE;
    const int64_t B = x->size(0), T = x->size(1), D = x->size(2), W = weight->size(1);
    int64_t ldx = 0;
    c.want(W >= 2 && W <= 4);
    c.need_rows(x, kBF16, {B, T, D}, 1, &ldx);
    c.need_float(weight, {D, W});
    if (!c.ok) Py_RETURN_NONE;
    c.may(a[2], bias, weight->scalar_type(), {D});
    int64_t N = B;
    if (a[4] != Py_None) {
        c.want(cu && B == 1 && cu->numel() > 0);
        if (!c.ok) Py_RETURN_NONE;
        N = cu->numel() - 1;
        c.need(cu, at::kLong, {N + 1});
    }
    const int64_t shape[] = {N, W - 1, D};
    c.may(a[3], init, kBF16, shape);
    c.may(a[6], out, kBF16, x->sizes());
    c.may(a[7], fin, kBF16, shape);
    if (!c.ok) Py_RETURN_NONE;
    void* stream;
    bool silu, want_final;
    if (!truth(a[5], &silu) || !truth(a[8], &want_final) || !stream_of(a[9], c.dev, &stream)) return nullptr;
    at::Tensor new_out, new_fin;
    want_final = want_final || fin;
    const int rc = released([&] {
        if (!out) out = &(new_out = at::empty(x->sizes(), x->options()));
        if (!fin && want_final) fin = &(new_fin = at::empty(shape, x->options()));
        return conv_prefill_fn(ptr(x), ldx, ptr(weight), ptr(bias), ptr(init), ptr(out), ptr(fin), N, T, D, static_cast<int>(W),
                               static_cast<const int64_t*>(ptr(cu)), silu ? KDA_ACT_SILU : KDA_ACT_NONE,
                               fp32(weight) ? KDA_FLAG_WEIGHT_F32 : 0u, stream);
    });
    if (rc != KDA_OK) return PyLong_FromLong(rc);
    return two(result(rc, a[6], new_out), !want_final ? Py_NewRef(Py_None) : result(rc, a[7], new_fin));
    END_HANDLE_TH_ERRORS
}

// x, weight, state, bias, slots, silu, out, stream
PyObject* conv_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!counted(n, 8) || !bound(reinterpret_cast<void*>(conv_decode_fn))) return nullptr;
    const at::Tensor *x = tensor(a[0]), *weight = tensor(a[1]), *state = tensor(a[2]), *bias = tensor(a[3]),
                     *slots = tensor(a[4]), *out = tensor(a[6]);
    Args c(x);
    if (!c.dims(x, 2) || !c.dims(weight, 2) || !c.dims(state, 3)) Py_RETURN_NONE;
    const int64_t N = x->size(0), D = x->size(1), W = weight->size(1), pool = state->size(0);
    int64_t ldx = 0;
    c.want(W >= 2 && W <= 4);
    c.need_rows(x, kBF16, {N, D}, 1, &ldx);
    c.need_float(weight, {D, W});
    c.need(state, kBF16, {pool, W - 1, D});
    if (!c.ok) Py_RETURN_NONE;
    c.may(a[3], bias, weight->scalar_type(), {D});
    if (a[4] == Py_None)
        c.want(N <= pool);
    else
        c.need(slots, at::kInt, {N});
    c.may(a[6], out, kBF16, x->sizes());
    if (!c.ok) Py_RETURN_NONE;
    void* stream;
    bool silu;
    if (!truth(a[5], &silu) || !stream_of(a[7], c.dev, &stream)) return nullptr;
    at::Tensor made;
    const int rc = released([&] {
        if (!out) out = &(made = at::empty(x->sizes(), x->options()));
        return conv_decode_fn(ptr(x), ldx, ptr(weight), ptr(bias), ptr(state), static_cast<const int32_t*>(ptr(slots)), ptr(out),
                              N, D, static_cast<int>(W), pool, silu ? KDA_ACT_SILU : KDA_ACT_NONE,
                              fp32(weight) ? KDA_FLAG_WEIGHT_F32 : 0u, stream);
    });
    return result(rc, a[6], made);
    END_HANDLE_TH_ERRORS
}

// What both forms of the scan read: x, dt, A, B, C, D, z, dt_bias, of `lead` tokens.
struct Scan {
    const at::Tensor *x, *dt, *A, *B, *C, *D, *z, *bias;
    int64_t dim = 0, groups = 0, S = 0, ldx = 0, lddt = 0, ldb = 0, ldc = 0, ldz = 0;
    Scan(Args& c, PyObject* const* a, int tokens_dims)
        : x(tensor(a[0])), dt(tensor(a[1])), A(tensor(a[2])), B(tensor(a[3])), C(tensor(a[4])), D(tensor(a[5])),
          z(tensor(a[6])), bias(tensor(a[7])) {
        const int64_t d = tokens_dims;
        if (!c.dims(x, d + 1) || !c.dims(A, 2) || !c.dims(B, d + 2)) return;
        dim = x->size(d);
        groups = B->size(d);
        S = A->size(1);
        c.want(groups > 0 && dim % groups == 0 && S > 0 && S <= 64);
        c.need_rows(x, kBF16, x->sizes(), 1, &ldx);
        c.need_rows_float(dt, x->sizes(), 1, &lddt);
        c.need(A, kF32, {dim, S});
        if (!c.ok) return;
        at::DimVector keys(x->sizes().begin(), x->sizes().end() - 1);
        keys.push_back(groups);
        keys.push_back(S);
        c.need_rows_float(B, keys, 2, &ldb);
        if (c.ok) c.need_rows(C, B->scalar_type(), keys, 2, &ldc);
        c.may(a[5], D, kF32, {dim});
        if (a[6] != Py_None) c.need_rows(z, kBF16, x->sizes(), 1, &ldz);
        c.may(a[7], bias, kF32, {dim});
    }
    uint32_t flags(bool state_f32, bool softplus) const {
        return (state_f32 ? KDA_FLAG_STATE_F32 : 0u) | (fp32(dt) ? KDA_FLAG_DT_F32 : 0u) | (fp32(B) ? KDA_FLAG_BC_F32 : 0u) |
               (softplus ? KDA_FLAG_DT_SOFTPLUS : 0u);
    }
    static const float* f(const at::Tensor* t) { return static_cast<const float*>(ptr(t)); }
};

// x, dt, A, B, C, D, z, dt_bias, dt_softplus, init_state, cu_seqlens, out, final_state, want_final, state_fp32, stream
PyObject* ssm_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!counted(n, 16) || !bound(reinterpret_cast<void*>(ssm_prefill_fn))) return nullptr;
    Args c(tensor(a[0]));
    const Scan s(c, a, 2);
    if (!c.ok) Py_RETURN_NONE;
    const at::Tensor *init = tensor(a[9]), *cu = tensor(a[10]), *out = tensor(a[11]), *fin = tensor(a[12]);
    const int64_t B = s.x->size(0), T = s.x->size(1);
    int64_t N = B;
    if (a[10] != Py_None) {
        c.want(cu && B == 1 && cu->numel() > 0);
        if (!c.ok) Py_RETURN_NONE;
        N = cu->numel() - 1;
        c.need(cu, at::kLong, {N + 1});
    }
    bool softplus, f32, want_final;
    if (!truth(a[8], &softplus) || !truth(a[14], &f32) || !truth(a[13], &want_final)) return nullptr;
    const int64_t shape[] = {N, s.dim, s.S};
    if (a[9] != Py_None) {
        c.need_float(init, shape);
        f32 = fp32(init);
    } else if (a[12] != Py_None) {
        c.need_float(fin, shape);
        f32 = fp32(fin);
    }
    c.may(a[12], fin, f32 ? kF32 : kBF16, shape);
    c.may(a[11], out, kBF16, s.x->sizes());
    if (!c.ok) Py_RETURN_NONE;
    void* stream;
    if (!stream_of(a[15], c.dev, &stream)) return nullptr;
    at::Tensor new_out, new_fin;
    want_final = want_final || fin;
    const int rc = released([&] {
        if (!out) out = &(new_out = at::empty(s.x->sizes(), s.x->options()));
        if (!fin && want_final) fin = &(new_fin = at::empty(shape, s.x->options().dtype(f32 ? kF32 : kBF16)));
        return ssm_prefill_fn(ptr(s.x), s.ldx, ptr(s.dt), s.lddt, Scan::f(s.A), ptr(s.B), s.ldb, ptr(s.C), s.ldc, Scan::f(s.D),
                              ptr(s.z), s.ldz, Scan::f(s.bias), ptr(init), ptr(out), ptr(fin), N, T, s.dim, s.groups, s.S,
                              static_cast<const int64_t*>(ptr(cu)), s.flags(f32, softplus), stream);
    });
    if (rc != KDA_OK) return PyLong_FromLong(rc);
    return two(result(rc, a[11], new_out), !want_final ? Py_NewRef(Py_None) : result(rc, a[12], new_fin));
    END_HANDLE_TH_ERRORS
}

// x, dt, A, B, C, D, z, dt_bias, dt_softplus, state, slots, out, stream
PyObject* ssm_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!counted(n, 13) || !bound(reinterpret_cast<void*>(ssm_decode_fn))) return nullptr;
    Args c(tensor(a[0]));
    const Scan s(c, a, 1);
    const at::Tensor *state = tensor(a[9]), *slots = tensor(a[10]), *out = tensor(a[11]);
    if (!c.dims(state, 3)) Py_RETURN_NONE;
    const int64_t N = s.x->size(0), pool = state->size(0);
    c.need_float(state, {pool, s.dim, s.S});
    if (a[10] == Py_None)
        c.want(N <= pool);
    else
        c.need(slots, at::kInt, {N});
    c.may(a[11], out, kBF16, s.x->sizes());
    if (!c.ok) Py_RETURN_NONE;
    void* stream;
    bool softplus;
    if (!truth(a[8], &softplus) || !stream_of(a[12], c.dev, &stream)) return nullptr;
    at::Tensor made;
    const int rc = released([&] {
        if (!out) out = &(made = at::empty(s.x->sizes(), s.x->options()));
        return ssm_decode_fn(ptr(s.x), s.ldx, ptr(s.dt), s.lddt, Scan::f(s.A), ptr(s.B), s.ldb, ptr(s.C), s.ldc, Scan::f(s.D),
                             ptr(s.z), s.ldz, Scan::f(s.bias), ptr(state), static_cast<const int32_t*>(ptr(slots)), ptr(out), N,
                             s.dim, s.groups, s.S, pool, s.flags(fp32(state), softplus), stream);
    });
    return result(rc, a[11], made);
    END_HANDLE_TH_ERRORS
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction method(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }

PyMethodDef methods[] = {
    {"bind", method(bind), METH_FASTCALL, nullptr},
    {"bind_scan", method(bind_scan), METH_FASTCALL, nullptr},
    {"conv_prefill", method(conv_prefill), METH_FASTCALL, nullptr},
    {"conv_decode", method(conv_decode), METH_FASTCALL, nullptr},
    {"ssm_prefill", method(ssm_prefill), METH_FASTCALL, nullptr},
    {"ssm_decode", method(ssm_decode), METH_FASTCALL, nullptr},
    {"la_prefill", method(la_prefill), METH_FASTCALL, nullptr},
    {"la_decode", method(la_decode), METH_FASTCALL, nullptr},
    {"kda_decode", method(kda_step), METH_FASTCALL, nullptr},
    {"gated_norm", method(gated_norm), METH_FASTCALL, nullptr},
    {"residual_norm", method(residual_norm), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_torch() { return PyModule_Create(&module); }
