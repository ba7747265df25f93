// Argument marshalling of the operators around the KDA layer for Python: tensors in, the C entry points of
// libkda.so called on the current stream.  These operators are called once a layer and token, where the
// time to unpack fifteen arguments in Python (6 us) would exceed the call itself (4 us); here it takes
// well under one.  Shapes, types, strides and devices are checked here, everything else by the entry points; a refused call
// raises the binding's KDAError.  Nothing is computed, allocated or kept.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "../../include/kda.h"

namespace {

PyObject *g_error = nullptr;   // the binding's KDAError(fn, status, message)

struct Refused {
    int status;
    const char *why = nullptr;
};

struct Rows {
    void *p;
    int64_t ld;
};

// The arguments of one call; throws Refused where a tensor does not fit.
struct Args {
    PyObject *const *a;
    Py_ssize_t n, at = 0;
    Args(PyObject *const *args, Py_ssize_t count, Py_ssize_t want) : a(args), n(count)
    {
        if (count != want) throw Refused{KDA_ERR_INVALID_ARG};
    }
    PyObject *next() { return a[at++]; }
    const at::Tensor *tensor(bool may_be_none = true)
    {
        PyObject *o = next();
        if (o == Py_None && may_be_none) return nullptr;
        if (!THPVariable_Check(o)) throw Refused{KDA_ERR_INVALID_ARG};
        return &THPVariable_Unpack(o);
    }
    int64_t integer()
    {
        const long long v = PyLong_AsLongLong(next());
        if (v == -1 && PyErr_Occurred()) throw Refused{KDA_ERR_INVALID_ARG};
        return v;
    }
    float real()
    {
        const double v = PyFloat_AsDouble(next());
        if (v == -1.0 && PyErr_Occurred()) throw Refused{KDA_ERR_INVALID_ARG};
        return static_cast<float>(v);
    }
    // None: the current stream of the current device; an integer or an object with 'cuda_stream'.
    void *stream()
    {
        PyObject *o = next();
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
        PyObject *v = PyLong_Check(o) ? (Py_INCREF(o), o) : PyObject_GetAttrString(o, "cuda_stream");
        if (!v) throw Refused{KDA_ERR_INVALID_ARG};
        void *p = PyLong_AsVoidPtr(v);
        Py_DECREF(v);
        if (PyErr_Occurred()) throw Refused{KDA_ERR_INVALID_ARG};
        return p;
    }
};

void need(bool ok)
{
    if (!ok) throw Refused{KDA_ERR_INVALID_ARG};
}

// The work goes to the current device: a tensor has to be there.
thread_local int t_device = -1;    // of this call, once it is known
void here(const at::Tensor &t)
{
    need(t.is_cuda());
    if (t_device < 0) t_device = c10::cuda::current_device();
    if (t.device().index() != t_device) throw Refused{KDA_ERR_INVALID_ARG, "a tensor is on another device than the current one"};
}

int32_t i32(int64_t v)
{
    need(v >= INT32_MIN && v <= INT32_MAX);
    return static_cast<int32_t>(v);
}

int type_code(at::ScalarType t)
{
    if (t == at::kBFloat16) return KDA_TYPE_BF16;
    if (t == at::kHalf) return KDA_TYPE_F16;
    need(t == at::kFloat);
    return KDA_TYPE_F32;
}

// Address and row stride of a [rows, width] tensor whose channels are adjacent (trailing axes count as one).
Rows rows_of(const at::Tensor *t, int64_t rows, int64_t width, at::ScalarType type)
{
    if (!t) return Rows{nullptr, 0};
    here(*t);
    need(t->scalar_type() == type && t->dim() >= 2 && t->size(0) == rows);
    int64_t n = 1;
    for (int64_t d = t->dim() - 1; d > 0; --d) {
        need(t->size(d) == 1 || t->stride(d) == n);
        n *= t->size(d);
    }
    need(n == width);
    return Rows{t->data_ptr(), rows > 1 ? t->stride(0) : width};
}

template <typename T> T *flat(const at::Tensor *t, int64_t numel, at::ScalarType type)
{
    if (!t) return nullptr;
    here(*t);
    need(t->scalar_type() == type && t->numel() == numel && t->is_contiguous());
    return static_cast<T *>(t->data_ptr());
}
float *floats(const at::Tensor *t, int64_t numel) { return flat<float>(t, numel, at::kFloat); }

struct Bytes {
    void *p;
    size_t n;
};
Bytes workspace(const at::Tensor *t)
{
    if (!t) return Bytes{nullptr, 0};
    here(*t);
    need(t->is_contiguous());
    return Bytes{t->data_ptr(), static_cast<size_t>(t->numel()) * t->element_size()};
}

// A host plan (int32 words in a buffer) and its device copy.
struct Plan {
    Py_buffer view = {};
    const int32_t *words = nullptr, *dev = nullptr;
    explicit Plan(Args &a)
    {
        if (PyObject_GetBuffer(a.next(), &view, PyBUF_SIMPLE) != 0) throw Refused{KDA_ERR_INVALID_ARG};
        try {
            words = static_cast<const int32_t *>(view.buf);
            const int64_t n = view.len / 4;
            need(n >= KDA_PLAN_HEADER_WORDS && words[KDA_PH_TOTAL] >= KDA_PLAN_HEADER_WORDS && n >= words[KDA_PH_TOTAL]);
            const at::Tensor *t = a.tensor(false);
            here(*t);
            need(t->scalar_type() == at::kInt && t->is_contiguous() && t->numel() >= words[KDA_PH_TOTAL]);
            dev = static_cast<const int32_t *>(t->data_ptr());
        } catch (...) {
            PyBuffer_Release(&view);
            throw;
        }
    }
    ~Plan() { PyBuffer_Release(&view); }
    Plan(const Plan &) = delete;
};

// Runs a call; its status, or what it threw, becomes the Python result.
template <typename F> PyObject *call(const char *name, F f)
{
    int status = KDA_ERR_INVALID_ARG;
    const char *why = nullptr;
    t_device = -1;
    try {
        status = f();
    } catch (const Refused &r) {
        status = r.status;
        why = r.why;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    PyErr_Clear();
    if (status == KDA_OK) Py_RETURN_NONE;
    PyObject *text = status == KDA_ERR_CUDA
                         ? PyUnicode_FromFormat("%s (cudaError %d)", kda_status_string(status), kda_last_cuda_error())
                     : why ? PyUnicode_FromFormat("%s (%s)", kda_status_string(status), why)
                           : PyUnicode_FromString(kda_status_string(status));
    PyObject *e = text ? PyObject_CallFunction(g_error, "siO", name, status, text) : nullptr;
    Py_XDECREF(text);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

PyObject *gated_scan_forward(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call("kda_gated_scan_forward", [&] {
        Args a(args, n, 11);
        const Plan plan(a);
        const int64_t T = plan.words[KDA_PH_T], N = plan.words[KDA_PH_N];
        const at::Tensor *x = a.tensor(false);
        need(x->dim() == 2);
        const int64_t D = x->size(1);
        const at::ScalarType ty = x->scalar_type();
        const Rows xr = rows_of(x, T, D, ty), ir = rows_of(a.tensor(), T, D, ty), g = rows_of(a.tensor(false), T, D, at::kFloat);
        const float *h0 = floats(a.tensor(), N * D);
        const Rows h = rows_of(a.tensor(false), T, D, ty);
        float *fin = floats(a.tensor(), N * D), *states = floats(a.tensor(), (T + KDA_SCAN_TILE - 1) / KDA_SCAN_TILE * D);
        const Bytes ws = workspace(a.tensor());
        return kda_gated_scan_forward(plan.words, plan.dev, i32(D), type_code(ty), xr.p, xr.ld, ir.p, ir.ld, static_cast<float *>(g.p), g.ld,
                                      h0, h.p, h.ld, fin, states, ws.p, ws.n, a.stream());
    });
}

PyObject *gated_scan_backward(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call("kda_gated_scan_backward", [&] {
        Args a(args, n, 15);
        const Plan plan(a);
        const int64_t T = plan.words[KDA_PH_T], N = plan.words[KDA_PH_N];
        const at::Tensor *x = a.tensor(false);
        need(x->dim() == 2);
        const int64_t D = x->size(1);
        const at::ScalarType ty = x->scalar_type();
        const Rows xr = rows_of(x, T, D, ty), ir = rows_of(a.tensor(), T, D, ty), g = rows_of(a.tensor(false), T, D, at::kFloat);
        const float *h0 = floats(a.tensor(), N * D), *states = floats(a.tensor(false), (T + KDA_SCAN_TILE - 1) / KDA_SCAN_TILE * D);
        const Rows dh = rows_of(a.tensor(false), T, D, ty);
        const float *dfinal = floats(a.tensor(), N * D);
        const Rows dx = rows_of(a.tensor(false), T, D, ty), di = rows_of(a.tensor(), T, D, ty);
        const Rows dg = rows_of(a.tensor(false), T, D, at::kFloat);
        float *dh0 = floats(a.tensor(), N * D);
        const Bytes ws = workspace(a.tensor());
        return kda_gated_scan_backward(plan.words, plan.dev, i32(D), type_code(ty), xr.p, xr.ld, ir.p, ir.ld, static_cast<float *>(g.p), g.ld,
                                       h0, states, dh.p, dh.ld, dfinal, dx.p, dx.ld, di.p, di.ld, static_cast<float *>(dg.p), dg.ld,
                                       dh0, ws.p, ws.n, a.stream());
    });
}

PyObject *gated_scan_step(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call("kda_gated_scan_step", [&] {
        Args a(args, n, 7);
        const at::Tensor *slots = a.tensor(), *x = a.tensor(false);
        need(x->dim() == 2);
        const int64_t B = x->size(0), D = x->size(1);
        const at::ScalarType ty = x->scalar_type();
        const Rows xr = rows_of(x, B, D, ty), ir = rows_of(a.tensor(), B, D, ty), g = rows_of(a.tensor(false), B, D, at::kFloat);
        const at::Tensor *state = a.tensor(false);
        need(state->dim() >= 1);
        const int64_t pool = state->size(0);
        float *s = floats(state, pool * D);
        const Rows h = rows_of(a.tensor(false), B, D, ty);
        return kda_gated_scan_step(i32(B), i32(D), type_code(ty), flat<int32_t>(slots, B, at::kInt), i32(pool), xr.p, xr.ld, ir.p, ir.ld,
                                   static_cast<float *>(g.p), g.ld, s, h.p, h.ld, a.stream());
    });
}

// The first tensor that is there; its rows and channels.
const at::Tensor &first_of(std::initializer_list<const at::Tensor *> all)
{
    for (const at::Tensor *t : all)
        if (t) return *t;
    throw Refused{KDA_ERR_INVALID_ARG};
}
int64_t channels(const at::Tensor &t)
{
    need(t.dim() >= 2);
    int64_t n = 1;
    for (int64_t d = 1; d < t.dim(); ++d) n *= t.size(d);
    return n;
}

PyObject *block_norm_forward(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call("kda_block_norm_forward", [&] {
        Args a(args, n, 13);
        const at::Tensor *r = a.tensor(), *o = a.tensor(), *z = a.tensor();
        const int64_t gate = a.integer(), group = a.integer();
        const at::Tensor *w_post = a.tensor();
        const float scale = a.real();
        const at::Tensor *ls = a.tensor(), *w_pre = a.tensor();
        const float eps = a.real();
        const at::Tensor *r_out = a.tensor(), *y = a.tensor();
        const at::Tensor &res = first_of({r, r_out, o}), &act = first_of({o, y, &res});
        const int64_t T = res.size(0), D = channels(res), G = group ? group : D;
        const at::ScalarType rt = res.scalar_type(), ty = act.scalar_type();
        const Rows rr = rows_of(r, T, D, rt), ro = rows_of(o, T, D, ty), rz = rows_of(z, T, D, ty);
        const Rows out = rows_of(r_out, T, D, rt), ry = rows_of(y, T, D, ty);
        return kda_block_norm_forward(T, i32(D), type_code(rt), type_code(ty), rr.p, rr.ld, ro.p, ro.ld, rz.p, rz.ld, i32(gate), i32(group),
                                      floats(w_post, G), scale, floats(ls, D), floats(w_pre, D), eps, out.p, out.ld, ry.p, ry.ld,
                                      a.stream());
    });
}

PyObject *block_norm_backward(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call("kda_block_norm_backward", [&] {
        Args a(args, n, 20);
        const at::Tensor *r_out = a.tensor(), *o = a.tensor(), *z = a.tensor();
        const int64_t gate = a.integer(), group = a.integer();
        const at::Tensor *w_post = a.tensor();
        const float scale = a.real();
        const at::Tensor *ls = a.tensor(), *w_pre = a.tensor();
        const float eps = a.real();
        const at::Tensor *dr_out = a.tensor(), *dy = a.tensor(), *dr = a.tensor(), *d_o = a.tensor(), *dz = a.tensor();
        const at::Tensor *dw_post = a.tensor(), *dls = a.tensor(), *dw_pre = a.tensor();
        const Bytes ws = workspace(a.tensor());
        const at::Tensor &res = first_of({dr_out, dr, r_out, dy, o}), &act = first_of({o, dy, d_o, &res});
        const int64_t T = res.size(0), D = channels(res), G = group ? group : D;
        const at::ScalarType rt = res.scalar_type(), ty = act.scalar_type();
        const Rows rr = rows_of(r_out, T, D, rt), ro = rows_of(o, T, D, ty), rz = rows_of(z, T, D, ty);
        const Rows gr = rows_of(dr_out, T, D, rt), gy = rows_of(dy, T, D, ty), out = rows_of(dr, T, D, rt);
        const Rows go = rows_of(d_o, T, D, ty), gz = rows_of(dz, T, D, ty);
        return kda_block_norm_backward(T, i32(D), type_code(rt), type_code(ty), rr.p, rr.ld, ro.p, ro.ld, rz.p, rz.ld, i32(gate), i32(group),
                                       floats(w_post, G), scale, floats(ls, D), floats(w_pre, D), eps, gr.p, gr.ld, gy.p, gy.ld, out.p,
                                       out.ld, go.p, go.ld, gz.p, gz.ld, floats(dw_post, G), floats(dls, D), floats(dw_pre, D), ws.p,
                                       ws.n, a.stream());
    });
}

PyObject *decode_step(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return call("kda_decode_step", [&] {
        Args a(args, n, 10);
        const at::Tensor *slots = a.tensor(), *q = a.tensor(false);
        need(q->dim() == 3 && q->size(2) == KDA_HEAD_DIM_K);
        const int64_t B = q->size(0), H = q->size(1), W = H * KDA_HEAD_DIM_K;
        const at::ScalarType ty = q->scalar_type();
        const Rows qr = rows_of(q, B, W, ty), k = rows_of(a.tensor(false), B, W, ty), v = rows_of(a.tensor(false), B, W, ty);
        const Rows g = rows_of(a.tensor(false), B, W, at::kFloat), beta = rows_of(a.tensor(false), B, H, at::kFloat);
        const float scale = a.real();
        const at::Tensor *state = a.tensor(false);
        need(state->dim() >= 1);
        const int64_t pool = state->size(0);
        float *s = floats(state, pool * W * KDA_HEAD_DIM_V);
        const Rows o = rows_of(a.tensor(false), B, W, ty);
        return kda_decode_step(i32(B), i32(H), type_code(ty), flat<int32_t>(slots, B, at::kInt), i32(pool), qr.p, qr.ld, k.p, k.ld, v.p, v.ld,
                               static_cast<float *>(g.p), g.ld, static_cast<float *>(beta.p), beta.ld, scale, s, o.p, o.ld, a.stream());
    });
}

PyObject *set_error(PyObject *, PyObject *cls)
{
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(gated_scan_forward), FAST(gated_scan_backward), FAST(gated_scan_step),
                           FAST(block_norm_forward), FAST(block_norm_backward), FAST(decode_step),
                           {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ops", "Argument marshalling of the operators around the KDA layer.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops(void) { return PyModule_Create(&g_module); }
