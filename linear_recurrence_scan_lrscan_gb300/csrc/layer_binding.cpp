// Python binding of the operators around the scan (module layer): argument
// checks, output tensors, the current stream and the call of the C ABI, without
// Python code in between, so that a single-token call costs little more than
// its launch.  The functions take positional arguments from layer.py, which has
// their documentation; all arithmetic is behind the C ABI.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "lrscan.h"

namespace {

using at::Tensor;

struct Failed {};  // a Python exception is set

[[noreturn]] void raise(PyObject *type, const char *fmt, ...) {
    char text[400];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    PyErr_SetString(type, text);
    throw Failed{};
}

struct Api {
    decltype(&lrscan_fwd_gates) fwd_gates;
    decltype(&lrscan_bwd_gates) bwd_gates;
    decltype(&lrscan_step_gates) step_gates;
    decltype(&lrscan_fwd_conv) fwd_conv;
    decltype(&lrscan_bwd_conv) bwd_conv;
    decltype(&lrscan_step_conv) step_conv;
    decltype(&lrscan_fwd_embed) fwd_embed;
    decltype(&lrscan_bwd_embed) bwd_embed;
};
Api api{};
PyObject *check = nullptr;     // lrscan._check(rc, what)
PyObject *dtype_of = nullptr;  // {torch.dtype: LRSCAN_*}

const Tensor *tensor(PyObject *o, const char *name, bool optional) {
    if (o == Py_None && optional) return nullptr;
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return &THPVariable_Unpack(o);
}

// The tensor whose type and device the others of a call have to have.
struct Lead {
    const Tensor *t;
    at::ScalarType dtype;
    c10::Device device;
    int code;
};
int code_of(at::ScalarType t) {
    if (t == at::kFloat) return LRSCAN_F32;
    if (t == at::kBFloat16) return LRSCAN_BF16;
    raise(PyExc_ValueError, "unsupported dtype %s; lrscan takes float32 or bfloat16 storage", c10::toString(t));
}
Lead lead(PyObject *o, const char *name, int dims, const char *shape) {
    const Tensor *t = tensor(o, name, false);
    if (t->dim() != dims || !t->is_cuda()) raise(PyExc_ValueError, "%s must be a CUDA %s tensor", name, shape);
    return {t, t->scalar_type(), t->device(), code_of(t->scalar_type())};
}

using Sizes = std::initializer_list<int64_t>;
bool shaped(const Tensor &t, Sizes sizes) { return t.sizes() == at::IntArrayRef(sizes.begin(), sizes.size()); }
[[noreturn]] void wrong(const char *name, const Tensor &t, Sizes sizes, at::ScalarType dtype, const char *more) {
    char want[80] = "", got[80] = "";
    int n = 0, m = 0;
    for (int64_t s : sizes) n += std::snprintf(want + n, sizeof want - n, "%s%lld", n ? ", " : "", static_cast<long long>(s));
    for (int64_t s : t.sizes())
        if (m < 60) m += std::snprintf(got + m, sizeof got - m, "%s%lld", m ? ", " : "", static_cast<long long>(s));
    raise(PyExc_ValueError, "%s must be a %s%s tensor of shape (%s); got %s (%s) on %s", name, more, c10::toString(dtype), want,
          c10::toString(t.scalar_type()), got, t.device().str().c_str());
}

// A tensor with contiguous channels, as the library takes it.
lrscan_rows rows(const char *name, const Tensor &t, Sizes sizes, at::ScalarType dtype, const Lead &l) {
    if (t.device() != l.device || t.scalar_type() != dtype || !shaped(t, sizes)) wrong(name, t, sizes, dtype, "CUDA ");
    const auto st = t.strides();
    if (t.size(-1) > 1 && st[st.size() - 1] != 1)
        raise(PyExc_ValueError, "%s must have contiguous channels (stride 1 in the last dimension)", name);
    return {t.data_ptr(), st[0], st.size() == 3 ? st[1] : 0};
}
lrscan_rows rows(const char *name, PyObject *o, Sizes sizes, const Lead &l) {
    return rows(name, *tensor(o, name, false), sizes, l.dtype, l);
}
// Pointer of a contiguous tensor, or null.
void *dense(const char *name, const Tensor &t, Sizes sizes, at::ScalarType dtype, const Lead &l) {
    if (t.device() != l.device || t.scalar_type() != dtype || !shaped(t, sizes) || !t.is_contiguous())
        wrong(name, t, sizes, dtype, "contiguous CUDA ");
    return t.data_ptr();
}
template <class T = float>
T *dense(const char *name, PyObject *o, Sizes sizes, at::ScalarType dtype, const Lead &l, bool optional = true) {
    const Tensor *t = tensor(o, name, optional);
    return t ? static_cast<T *>(dense(name, *t, sizes, dtype, l)) : nullptr;
}

Tensor fresh(const Lead &l, Sizes sizes, at::ScalarType dtype) {
    return at::empty(at::IntArrayRef(sizes.begin(), sizes.size()), at::TensorOptions().dtype(dtype).device(l.device));
}
// The caller's output, or a new one.
Tensor output(const char *name, PyObject *o, const Lead &l, Sizes sizes, at::ScalarType dtype) {
    if (o == Py_None) return fresh(l, sizes, dtype);
    return *tensor(o, name, false);
}

// The call's device, stream and workspace.
struct Call {
    c10::cuda::OptionalCUDAGuard guard;
    void *stream;
    lrscan_opts opts{}, *with = nullptr;
    Call(const Lead &l, PyObject *on, PyObject *workspace) {
        if (l.device.index() != c10::cuda::current_device()) guard.set_device(l.device);
        if (on == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(l.device.index()).stream();
        } else {
            PyObject *p = PyObject_GetAttrString(on, "cuda_stream");
            if (!p) throw Failed{};
            stream = PyLong_AsVoidPtr(p);
            Py_DECREF(p);
            if (!stream && PyErr_Occurred()) throw Failed{};
        }
        if (workspace && workspace != Py_None) {
            const Tensor *w = tensor(workspace, "workspace", false);
            if (!w->is_cuda()) raise(PyExc_ValueError, "workspace must be a CUDA tensor");
            opts.workspace = w->data_ptr();
            opts.workspace_bytes = w->nbytes();
            with = &opts;
        }
    }
};
void done(int rc, const char *what) {
    if (rc == LRSCAN_OK) return;
    PyObject *r = PyObject_CallFunction(check, "is", rc, what);  // raises
    Py_XDECREF(r);
    if (r) PyErr_SetString(PyExc_RuntimeError, what);
    throw Failed{};
}

PyObject *wrap(const Tensor &t) { return THPVariable_Wrap(t); }
PyObject *none() { Py_RETURN_NONE; }
PyObject *tuple(std::initializer_list<PyObject *> items) {
    PyObject *t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
    Py_ssize_t k = 0;
    for (PyObject *o : items) PyTuple_SET_ITEM(t, k++, o);
    return t;
}
bool yes(PyObject *o) { return PyObject_IsTrue(o) == 1; }
float number(PyObject *o) {
    const double d = PyFloat_AsDouble(o);
    if (d == -1.0 && PyErr_Occurred()) throw Failed{};
    return static_cast<float>(d);
}

constexpr int64_t kSave = 16;  // tokens between the gated recurrence's saved states

// r, i, x, lam, c, h0, segment_pos, out, last, saved, want_saved, workspace, stream
PyObject *fwd_gates(PyObject *const *a) {
    const Lead l = lead(a[2], "x", 3, "[B, T, D]");
    const int64_t B = l.t->size(0), T = l.t->size(1), D = l.t->size(2), ns = (T + kSave - 1) / kSave;
    const lrscan_rows r = rows("r", a[0], {B, T, D}, l), i = rows("i", a[1], {B, T, D}, l), x = rows("x", a[2], {B, T, D}, l);
    const float *lam = dense("lam", a[3], {D}, at::kFloat, l, false);
    lrscan_state st{};
    st.h0 = dense("h0", a[5], {B, D}, at::kFloat, l);
    st.segment_pos = dense<int32_t>("segment_pos", a[6], {B, T}, at::kInt, l);
    const Tensor out = output("out", a[7], l, {B, T, D}, l.dtype), last = output("last", a[8], l, {B, D}, at::kFloat);
    Tensor saved;
    if (a[9] != Py_None || yes(a[10])) saved = output("saved", a[9], l, {B, ns, D}, at::kFloat);
    const lrscan_rows o = rows("out", out, {B, T, D}, l.dtype, l);
    float *lp = static_cast<float *>(dense("last", last, {B, D}, at::kFloat, l));
    float *sp = saved.defined() ? static_cast<float *>(dense("saved", saved, {B, ns, D}, at::kFloat, l)) : nullptr;
    const float c = number(a[4]);
    Call call(l, a[12], a[11]);
    done(api.fwd_gates(&r, &i, &x, lam, c, &o, lp, sp, &st, B, T, D, l.code, call.stream, call.with), "lrscan_fwd_gates");
    return tuple({wrap(out), wrap(last), saved.defined() ? wrap(saved) : none()});
}

// r, i, x, lam, saved, grad_out, c, segment_pos, grad_last, grad_r, grad_i, grad_x, grad_lam, grad_h0, want_grad_h0,
// workspace, stream
PyObject *bwd_gates(PyObject *const *a) {
    const Lead l = lead(a[2], "x", 3, "[B, T, D]");
    const int64_t B = l.t->size(0), T = l.t->size(1), D = l.t->size(2), ns = (T + kSave - 1) / kSave;
    const lrscan_rows r = rows("r", a[0], {B, T, D}, l), i = rows("i", a[1], {B, T, D}, l), x = rows("x", a[2], {B, T, D}, l);
    const float *lam = dense("lam", a[3], {D}, at::kFloat, l, false), *saved = dense("saved", a[4], {B, ns, D}, at::kFloat, l, false);
    const lrscan_rows go = rows("grad_out", a[5], {B, T, D}, l);
    lrscan_state st{};
    st.segment_pos = dense<int32_t>("segment_pos", a[7], {B, T}, at::kInt, l);
    st.grad_last = dense("grad_last", a[8], {B, D}, at::kFloat, l);
    const Tensor gr = output("grad_r", a[9], l, {B, T, D}, l.dtype), gi = output("grad_i", a[10], l, {B, T, D}, l.dtype),
                 gx = output("grad_x", a[11], l, {B, T, D}, l.dtype), gl = output("grad_lam", a[12], l, {D}, at::kFloat);
    Tensor gh;
    if (a[13] != Py_None || yes(a[14])) gh = output("grad_h0", a[13], l, {B, D}, at::kFloat);
    const lrscan_rows o0 = rows("grad_r", gr, {B, T, D}, l.dtype, l), o1 = rows("grad_i", gi, {B, T, D}, l.dtype, l),
                      o2 = rows("grad_x", gx, {B, T, D}, l.dtype, l);
    float *lp = static_cast<float *>(dense("grad_lam", gl, {D}, at::kFloat, l));
    if (gh.defined()) st.grad_h0 = static_cast<float *>(dense("grad_h0", gh, {B, D}, at::kFloat, l));
    const float c = number(a[6]);
    Call call(l, a[16], a[15]);
    done(api.bwd_gates(&r, &i, &x, lam, c, saved, &go, &o0, &o1, &o2, lp, &st, B, T, D, l.code, call.stream, call.with),
         "lrscan_bwd_gates");
    return tuple({wrap(gr), wrap(gi), wrap(gx), wrap(gl), gh.defined() ? wrap(gh) : none()});
}

// r, i, x, lam, state, slots, c, out, stream
PyObject *step_gates(PyObject *const *a) {
    const Lead l = lead(a[2], "x", 2, "[B, D]");
    const int64_t B = l.t->size(0), D = l.t->size(1);
    const lrscan_rows r = rows("r", a[0], {B, D}, l), i = rows("i", a[1], {B, D}, l), x = rows("x", a[2], {B, D}, l);
    const float *lam = dense("lam", a[3], {D}, at::kFloat, l, false);
    const Tensor *state = tensor(a[4], "state", false);
    if (state->dim() != 2) raise(PyExc_ValueError, "state must be a [S, D] tensor");
    const int64_t S = state->size(0);
    float *sp = static_cast<float *>(dense("state", *state, {S, D}, at::kFloat, l));
    const int32_t *slots = dense<int32_t>("slots", a[5], {B}, at::kInt, l);
    const float c = number(a[6]);
    const Tensor out = output("out", a[7], l, {B, D}, l.dtype);
    const lrscan_rows o = rows("out", out, {B, D}, l.dtype, l);
    Call call(l, a[8], nullptr);
    done(api.step_gates(&r, &i, &x, lam, c, sp, slots, &o, B, S, D, l.code, call.stream), "lrscan_step_gates");
    return wrap(out);
}

int64_t taps(const Tensor &w, int64_t D) {
    if (w.dim() != 2 || w.size(0) != D) raise(PyExc_ValueError, "w must be a [D, K] tensor, D = %lld", static_cast<long long>(D));
    return w.size(1);
}

// x, w, bias, x0, segment_pos, out, last, want_last, stream
PyObject *fwd_conv(PyObject *const *a) {
    const Lead l = lead(a[0], "x", 3, "[B, T, D]");
    const int64_t B = l.t->size(0), T = l.t->size(1), D = l.t->size(2), K = taps(*tensor(a[1], "w", false), D);
    const lrscan_rows x = rows("x", a[0], {B, T, D}, l);
    const float *w = dense("w", a[1], {D, K}, at::kFloat, l), *bias = dense("bias", a[2], {D}, at::kFloat, l);
    const void *x0 = dense<void>("x0", a[3], {B, K - 1, D}, l.dtype, l);
    const int32_t *seg = dense<int32_t>("segment_pos", a[4], {B, T}, at::kInt, l);
    const Tensor out = output("out", a[5], l, {B, T, D}, l.dtype);
    Tensor last;
    if (a[6] != Py_None || yes(a[7])) last = output("last", a[6], l, {B, K > 1 ? K - 1 : 0, D}, l.dtype);
    const lrscan_rows o = rows("out", out, {B, T, D}, l.dtype, l);
    void *lp = last.defined() ? dense("last", last, {B, K > 1 ? K - 1 : 0, D}, l.dtype, l) : nullptr;
    Call call(l, a[8], nullptr);
    done(api.fwd_conv(&x, w, bias, static_cast<int>(K), x0, seg, &o, lp, B, T, D, l.code, call.stream), "lrscan_fwd_conv");
    return tuple({wrap(out), last.defined() ? wrap(last) : none()});
}

// x, w, grad_out, x0, segment_pos, grad_last, grad_x, grad_w, grad_bias, grad_x0, want_grad_x0, workspace, stream
PyObject *bwd_conv(PyObject *const *a) {
    const Lead l = lead(a[0], "x", 3, "[B, T, D]");
    const int64_t B = l.t->size(0), T = l.t->size(1), D = l.t->size(2), K = taps(*tensor(a[1], "w", false), D);
    const lrscan_rows x = rows("x", a[0], {B, T, D}, l), go = rows("grad_out", a[2], {B, T, D}, l);
    const float *w = dense("w", a[1], {D, K}, at::kFloat, l);
    const void *x0 = dense<void>("x0", a[3], {B, K - 1, D}, l.dtype, l), *gl = dense<void>("grad_last", a[5], {B, K - 1, D}, l.dtype, l);
    const int32_t *seg = dense<int32_t>("segment_pos", a[4], {B, T}, at::kInt, l);
    const Tensor gx = output("grad_x", a[6], l, {B, T, D}, l.dtype), gw = output("grad_w", a[7], l, {D, K}, at::kFloat),
                 gb = output("grad_bias", a[8], l, {D}, at::kFloat);
    Tensor g0;
    if (a[9] != Py_None || yes(a[10])) g0 = output("grad_x0", a[9], l, {B, K > 1 ? K - 1 : 0, D}, l.dtype);
    const lrscan_rows o = rows("grad_x", gx, {B, T, D}, l.dtype, l);
    float *wp = static_cast<float *>(dense("grad_w", gw, {D, K}, at::kFloat, l)),
          *bp = static_cast<float *>(dense("grad_bias", gb, {D}, at::kFloat, l));
    void *p0 = g0.defined() ? dense("grad_x0", g0, {B, K > 1 ? K - 1 : 0, D}, l.dtype, l) : nullptr;
    Call call(l, a[12], a[11]);
    done(api.bwd_conv(&x, w, static_cast<int>(K), x0, seg, &go, gl, &o, wp, bp, p0, B, T, D, l.code, call.stream, call.with),
         "lrscan_bwd_conv");
    return tuple({wrap(gx), wrap(gw), wrap(gb), g0.defined() ? wrap(g0) : none()});
}

// x, w, state, bias, slots, out, stream
PyObject *step_conv(PyObject *const *a) {
    const Lead l = lead(a[0], "x", 2, "[B, D]");
    const int64_t B = l.t->size(0), D = l.t->size(1), K = taps(*tensor(a[1], "w", false), D);
    const lrscan_rows x = rows("x", a[0], {B, D}, l);
    const float *w = dense("w", a[1], {D, K}, at::kFloat, l), *bias = dense("bias", a[3], {D}, at::kFloat, l);
    const Tensor *state = tensor(a[2], "state", false);
    if (state->dim() != 3) raise(PyExc_ValueError, "state must be a [S, K-1, D] tensor");
    const int64_t S = state->size(0);
    void *sp = dense("state", *state, {S, K - 1, D}, l.dtype, l);
    const int32_t *slots = dense<int32_t>("slots", a[4], {B}, at::kInt, l);
    const Tensor out = output("out", a[5], l, {B, D}, l.dtype);
    const lrscan_rows o = rows("out", out, {B, D}, l.dtype, l);
    Call call(l, a[6], nullptr);
    done(api.step_conv(&x, w, bias, static_cast<int>(K), sp, slots, &o, B, S, D, l.code, call.stream), "lrscan_step_conv");
    return wrap(out);
}

struct Ids {
    const void *p;
    int bytes;
    int64_t n;
    at::IntArrayRef shape;
};
Ids ids_of(PyObject *o, const c10::Device &device) {
    const Tensor *t = tensor(o, "ids", false);
    if (t->scalar_type() != at::kInt && t->scalar_type() != at::kLong)
        raise(PyExc_ValueError, "ids must be int32 or int64, got %s", c10::toString(t->scalar_type()));
    if (!t->is_cuda() || t->device() != device)
        raise(PyExc_ValueError, "ids is on %s, expected %s", t->device().str().c_str(), device.str().c_str());
    if (!t->is_contiguous()) raise(PyExc_ValueError, "ids must be contiguous");
    return {t->data_ptr(), t->scalar_type() == at::kInt ? 4 : 8, t->numel(), t->sizes()};
}
// A torch.dtype, or the type to take in its absence.
at::ScalarType type_of(PyObject *o, at::ScalarType otherwise) {
    if (o == Py_None) return otherwise;
    PyObject *code = PyDict_GetItem(dtype_of, o);
    if (!code) raise(PyExc_ValueError, "unsupported dtype; lrscan takes float32 or bfloat16 storage");
    return PyLong_AsLong(code) == LRSCAN_F32 ? at::kFloat : at::kBFloat16;
}

// ids, weight, scale, dtype, out, stream
PyObject *fwd_embed(PyObject *const *a) {
    const Lead l = lead(a[1], "weight", 2, "[V, D]");
    const Ids ids = ids_of(a[0], l.device);
    const int64_t V = l.t->size(0), D = l.t->size(1);
    const void *w = dense("weight", *l.t, {V, D}, l.dtype, l);
    c10::SmallVector<int64_t, 6> shape(ids.shape.begin(), ids.shape.end());
    shape.push_back(D);
    Tensor out;
    if (a[4] == Py_None) {
        out = at::empty(shape, at::TensorOptions().dtype(type_of(a[3], l.dtype)).device(l.device));
    } else {
        out = *tensor(a[4], "out", false);
        if (out.sizes() != at::IntArrayRef(shape) || out.device() != l.device || !out.is_contiguous())
            raise(PyExc_ValueError, "out must be a contiguous CUDA tensor of shape [*ids.shape, D]");
    }
    const int code = code_of(out.scalar_type());
    const float scale = number(a[2]);
    Call call(l, a[5], nullptr);
    done(api.fwd_embed(ids.p, ids.bytes, w, l.code, scale, out.data_ptr(), code, ids.n, V, D, call.stream), "lrscan_fwd_embed");
    return wrap(out);
}

// ids, grad_out, V, scale, dtype, grad_weight, accumulate, workspace, stream
PyObject *bwd_embed(PyObject *const *a) {
    const Tensor *go = tensor(a[1], "grad_out", false);
    if (!go->is_cuda()) raise(PyExc_ValueError, "grad_out must be on a CUDA device");
    const Lead l{go, go->scalar_type(), go->device(), code_of(go->scalar_type())};
    const Ids ids = ids_of(a[0], l.device);
    const int64_t dims = static_cast<int64_t>(ids.shape.size());
    if (go->dim() != dims + 1 || go->sizes().slice(0, dims) != ids.shape)
        raise(PyExc_ValueError, "grad_out must be a [*ids.shape, D] tensor");
    if (!go->is_contiguous()) raise(PyExc_ValueError, "grad_out must be contiguous");
    const bool add = yes(a[6]);
    if (add && a[5] == Py_None) raise(PyExc_ValueError, "accumulate needs grad_weight");
    const int64_t V = PyLong_AsLongLong(a[2]), D = go->size(-1);
    if (V == -1 && PyErr_Occurred()) throw Failed{};
    if (V < 0) raise(PyExc_ValueError, "V is negative");
    Tensor gw;
    if (a[5] == Py_None) {
        gw = fresh(l, {V, D}, type_of(a[4], at::kFloat));
    } else {
        gw = *tensor(a[5], "grad_weight", false);
    }
    void *wp = dense("grad_weight", gw, {V, D}, gw.scalar_type(), l);
    const int code = code_of(gw.scalar_type());
    const float scale = number(a[3]);
    Call call(l, a[8], a[7]);
    done(api.bwd_embed(ids.p, ids.bytes, go->data_ptr(), l.code, scale, wp, code, add, ids.n, V, D, call.stream, call.with),
         "lrscan_bwd_embed");
    return wrap(gw);
}

template <PyObject *(*F)(PyObject *const *), int N> PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    if (!api.fwd_gates) {
        PyErr_SetString(PyExc_RuntimeError, "the binding has not been given the library");
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Failed &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// bind(addresses of the eight functions in the order of Api, check, dtypes)
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    void *at[8];
    if (n != 3 || !PyTuple_Check(args[0]) || PyTuple_GET_SIZE(args[0]) != 8) {
        PyErr_SetString(PyExc_TypeError, "bind takes eight addresses, a function and a dict");
        return nullptr;
    }
    for (int k = 0; k < 8; ++k) {
        at[k] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args[0], k));
        if (!at[k]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "a NULL address");
    }
    Py_INCREF(args[1]);
    Py_INCREF(args[2]);
    check = args[1];
    dtype_of = args[2];
    api = {reinterpret_cast<decltype(api.fwd_gates)>(at[0]), reinterpret_cast<decltype(api.bwd_gates)>(at[1]),
           reinterpret_cast<decltype(api.step_gates)>(at[2]), reinterpret_cast<decltype(api.fwd_conv)>(at[3]),
           reinterpret_cast<decltype(api.bwd_conv)>(at[4]), reinterpret_cast<decltype(api.step_conv)>(at[5]),
           reinterpret_cast<decltype(api.fwd_embed)>(at[6]), reinterpret_cast<decltype(api.bwd_embed)>(at[7])};
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), int N> PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    method<fwd_gates, 13>("fwd_gates"),
    method<bwd_gates, 17>("bwd_gates"),
    method<step_gates, 9>("step_gates"),
    method<fwd_conv, 9>("fwd_conv"),
    method<bwd_conv, 13>("bwd_conv"),
    method<step_conv, 7>("step_conv"),
    method<fwd_embed, 6>("fwd_embed"),
    method<bwd_embed, 9>("bwd_embed"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "lrscan_layer", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_lrscan_layer() { return PyModule_Create(&module); }
