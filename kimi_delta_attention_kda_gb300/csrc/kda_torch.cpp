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
    PyObject* o = result(rc, a[6], new_out);
    PyObject* f = !want_final ? Py_NewRef(Py_None) : result(rc, a[7], new_fin);
    PyObject* both = o && f ? PyTuple_Pack(2, o, f) : nullptr;
    Py_XDECREF(o);
    Py_XDECREF(f);
    return both;
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
    PyObject* o = result(rc, a[7], made);
    PyObject* r = result(rc, a[8], rmade);
    PyObject* both = o && r ? PyTuple_Pack(2, o, r) : nullptr;
    Py_XDECREF(o);
    Py_XDECREF(r);
    return both;
    END_HANDLE_TH_ERRORS
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction method(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }

PyMethodDef methods[] = {
    {"bind", method(bind), METH_FASTCALL, nullptr},
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
