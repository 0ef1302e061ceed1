// fq_binding.cpp -- the argument marshalling of the row operators (norm,
// expert sorting, optimizer) as a CPython extension over the C ABI.
//
// Such a call's kernels take 2 to 5 us on a small batch; checking seven
// tensors and calling through ctypes took 8 us of host time before the launch,
// reading the tensors' fields here takes below 1.  Same rules as the ctypes
// binding: the library sees only pointers and sizes, so each operand is checked
// for what the library cannot see (a GPU tensor, contiguous, of its type, long
// enough; a smaller buffer would be written past its end).  Python's wrappers
// fill in missing outputs; every function here takes all arguments by
// position, the stream last, and returns the library's status.  The
// interpreter's lock is released around the library's call.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fq.h"

namespace {

using at::ScalarType;

PyObject *g_raw_stream = nullptr;     // torch._C._cuda_getCurrentRawStream
PyObject *g_device = nullptr;         // torch._C._cuda_getDevice
PyObject *g_cuda_stream = nullptr;    // "cuda_stream"

const char *type_name(ScalarType t)
{
    return t == at::kBFloat16 ? "bfloat16" : t == at::kFloat ? "float32" : t == at::kInt ? "int32"
                                                                                : c10::toString(t);
}

// Set by the first failed check of a call; later checks then do nothing.
struct Call {
    PyObject *const *args;
    bool ok = true;

    Call(PyObject *const *a, Py_ssize_t n, Py_ssize_t want) : args(a)
    {
        if (n != want) {
            PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, want);
            ok = false;
        }
    }
    void refuse(const char *fmt, const char *name, const char *more = "", long long a = 0,
                long long b = 0)
    {
        PyErr_Format(PyExc_ValueError, fmt, name, more, a, b);
        ok = false;
    }
    long long i64(int i)
    {
        if (!ok) return 0;
        const long long v = PyLong_AsLongLong(args[i]);
        if (v == -1 && PyErr_Occurred()) ok = false;
        return v;
    }
    unsigned long long u64(int i)        // modulo 2^64, as ctypes takes a seed
    {
        if (!ok) return 0;
        const unsigned long long v = PyLong_AsUnsignedLongLongMask(args[i]);
        if (v == ~0ull && PyErr_Occurred()) ok = false;
        return v;
    }
    double f64(int i)
    {
        if (!ok) return 0;
        const double v = PyFloat_AsDouble(args[i]);
        if (v == -1.0 && PyErr_Occurred()) ok = false;
        return v;
    }
    // Tensor or None (null).
    const at::Tensor *tensor(int i, const char *name)
    {
        if (!ok || args[i] == Py_None) return nullptr;
        if (!THPVariable_Check(args[i])) {
            PyErr_Format(PyExc_TypeError, "%s must be a tensor, not %s", name,
                         Py_TYPE(args[i])->tp_name);
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(args[i]);
    }
    void *pointer(const at::Tensor &t, long long n, const char *name)
    {
        if (!ok) return nullptr;
        if (!t.is_cuda()) {
            refuse("%s must be a GPU tensor%s", name);
        } else if (!t.is_contiguous()) {
            refuse("%s must be contiguous (row-major)%s", name);
        } else if (t.numel() < n) {
            refuse("%s%s holds %lld elements, %lld are needed", name, "", t.numel(), n);
        } else {
            return t.data_ptr();
        }
        return nullptr;
    }
    // Operand of one type, `n` elements at least.
    void *typed(int i, ScalarType type, long long n, const char *name)
    {
        const at::Tensor *t = tensor(i, name);
        if (!t) return nullptr;
        if (t->scalar_type() != type)
            return refuse("%s must be %s", name, type_name(type)), nullptr;
        return pointer(*t, n, name);
    }
    // Operand of any one-byte type (codes, scales, workspaces).
    void *bytes(int i, long long n, const char *name)
    {
        const at::Tensor *t = tensor(i, name);
        if (!t) return nullptr;
        if (t->element_size() != 1)
            return refuse("%s%s has %lld-byte elements, expected 1", name, "", t->element_size()),
                   nullptr;
        return pointer(*t, n, name);
    }
    // BF16 or FP32 operand; *type its FQ_TYPE_* (unchanged for None).
    void *real(int i, long long n, const char *name, int32_t *type)
    {
        const at::Tensor *t = tensor(i, name);
        if (!t) return nullptr;
        if (t->scalar_type() == at::kBFloat16) *type = FQ_TYPE_BF16;
        else if (t->scalar_type() == at::kFloat) *type = FQ_TYPE_F32;
        else
            return refuse("%s must be bfloat16 or float32, not %s", name,
                          type_name(t->scalar_type())), nullptr;
        return pointer(*t, n, name);
    }
    // rows and cols of a matrix operand
    bool shape(int i, const char *name, long long *rows, long long *cols)
    {
        const at::Tensor *t = tensor(i, name);
        if (!ok) return false;
        if (!t || t->dim() != 2) return refuse("%s must be a matrix%s", name), false;
        *rows = t->size(0);
        *cols = t->size(1);
        return true;
    }
    void *workspace(int i, size_t *n)
    {
        const at::Tensor *t = tensor(i, "ws");
        *n = 0;
        if (!t || t->numel() == 0) return nullptr;
        *n = (size_t)t->numel() * t->element_size();
        return pointer(*t, 0, "ws");
    }
    void *scales8(int i, int f8, long long rows, long long cols)
    {
        if (f8 == FQ_F8_ROW) return typed(i, at::kFloat, rows, "scales");
        return bytes(i, f8 == FQ_F8_MX ? rows * (cols / 32) : 0, "scales");
    }
    // A torch stream, or None: the current one of the current device.
    void *stream(int i)
    {
        if (!ok) return nullptr;
        PyObject *v = nullptr;
        if (args[i] == Py_None) {
            PyObject *dev = PyObject_CallNoArgs(g_device);
            if (dev) v = PyObject_CallOneArg(g_raw_stream, dev);
            Py_XDECREF(dev);
        } else {
            v = PyObject_GetAttr(args[i], g_cuda_stream);
        }
        void *s = v ? PyLong_AsVoidPtr(v) : nullptr;
        Py_XDECREF(v);
        if (PyErr_Occurred()) ok = false;
        return s;
    }
};

template <typename F>
PyObject *launch(const Call &c, F call)
{
    if (!c.ok) return nullptr;
    fq_status s;
    Py_BEGIN_ALLOW_THREADS
    s = call();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(s);
}

// (x, gamma, eps, res, f8, h, y, codes, scales, rstd, stream)
PyObject *rmsnorm_fwd(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    Call c(args, nargs, 11);
    long long rows = 0, cols = 0;
    if (!c.ok || !c.shape(0, "x", &rows, &cols)) return nullptr;
    const long long n = rows * cols;
    int32_t stream_type = FQ_TYPE_BF16, gamma_type = FQ_TYPE_F32;
    const void *x = c.typed(0, at::kBFloat16, n, "x");
    const void *res = c.real(3, n, "res", &stream_type);
    const void *gamma = c.real(1, cols, "gamma", &gamma_type);
    const float eps = (float)c.f64(2);
    const int f8 = (int)c.i64(4);
    void *h = c.typed(5, stream_type == FQ_TYPE_F32 ? at::kFloat : at::kBFloat16, n, "h");
    void *y = c.typed(6, at::kBFloat16, n, "y");
    void *codes = c.bytes(7, n, "codes");
    void *scales = c.scales8(8, f8, rows, cols);
    float *rstd = (float *)c.typed(9, at::kFloat, rows, "rstd");
    void *st = c.stream(10);
    return launch(c, [&] {
        return fq_rmsnorm_fwd(x, res, stream_type, gamma, gamma_type, eps, rows, cols, f8, h, y,
                              codes, scales, rstd, st);
    });
}

// (dy, h, gamma, rstd, dres, dh, dx, dgamma, ws, stream)
PyObject *rmsnorm_bwd(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    Call c(args, nargs, 10);
    long long rows = 0, cols = 0;
    if (!c.ok || !c.shape(0, "dy", &rows, &cols)) return nullptr;
    const long long n = rows * cols;
    int32_t stream_type = FQ_TYPE_BF16, gamma_type = FQ_TYPE_F32;
    const void *dy = c.typed(0, at::kBFloat16, n, "dy");
    const void *h = c.real(1, n, "h", &stream_type);
    const void *gamma = c.real(2, cols, "gamma", &gamma_type);
    const float *rstd = (const float *)c.typed(3, at::kFloat, rows, "rstd");
    const ScalarType wide = stream_type == FQ_TYPE_F32 ? at::kFloat : at::kBFloat16;
    const void *dres = c.typed(4, wide, n, "dres");
    void *dh = c.typed(5, wide, n, "dh");
    void *dx = c.typed(6, at::kBFloat16, n, "dx");
    float *dgamma = (float *)c.typed(7, at::kFloat, cols, "dgamma");
    size_t ws_bytes = 0;
    void *ws = c.workspace(8, &ws_bytes);
    void *st = c.stream(9);
    return launch(c, [&] {
        return fq_rmsnorm_bwd(dy, h, stream_type, gamma, gamma_type, rstd, dres, rows, cols, dh,
                              dx, dgamma, ws, ws_bytes, st);
    });
}

// (experts_of, experts, align, offsets, pos, src, ws, stream)
PyObject *moe_sort(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    Call c(args, nargs, 8);
    long long tokens = 0, k = 0;
    if (!c.ok || !c.shape(0, "experts_of", &tokens, &k)) return nullptr;
    const long long experts = c.i64(1), align = c.i64(2);
    const int32_t *ids = (const int32_t *)c.typed(0, at::kInt, tokens * k, "experts_of");
    int32_t *offsets = (int32_t *)c.typed(3, at::kInt, experts + 1, "offsets");
    int32_t *pos = (int32_t *)c.typed(4, at::kInt, tokens * k, "pos");
    int32_t *src = (int32_t *)c.typed(5, at::kInt, 0, "src");
    const at::Tensor *t = c.tensor(5, "src");
    const long long rows = t ? t->numel() : 0;
    size_t ws_bytes = 0;
    void *ws = c.workspace(6, &ws_bytes);
    void *st = c.stream(7);
    return launch(c, [&] {
        return fq_moe_sort(ids, tokens, k, experts, align, rows, offsets, pos, src, ws, ws_bytes,
                           st);
    });
}

// pos [tokens, k] and, where the operator reads it, src [rows]
struct Sorted {
    long long tokens = 0, k = 0, rows = 0;
    const int32_t *pos = nullptr, *src = nullptr;
    Sorted(Call &c, int at)
    {
        if (!c.shape(at, "pos", &tokens, &k)) return;
        pos = (const int32_t *)c.typed(at, at::kInt, tokens * k, "pos");
        src = (const int32_t *)c.typed(at + 1, at::kInt, 0, "src");
        if (const at::Tensor *t = c.tensor(at + 1, "src")) rows = t->numel();
    }
};

// (x, f8, scales, pos, src, y, stream)
PyObject *moe_dispatch(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    Call c(args, nargs, 7);
    long long tokens = 0, cols = 0;
    if (!c.ok || !c.shape(0, "x", &tokens, &cols)) return nullptr;
    const int f8 = (int)c.i64(1);
    const Sorted q(c, 3);
    if (c.ok && tokens != q.tokens)
        c.refuse("%s has %s%lld rows, %lld tokens were sorted", "x", "", tokens, q.tokens);
    const void *x = f8 == FQ_F8_NONE ? c.typed(0, at::kBFloat16, tokens * cols, "x")
                                     : c.bytes(0, tokens * cols, "x");
    const void *scales = c.scales8(2, f8, tokens, cols);
    void *y = c.typed(5, at::kBFloat16, q.rows * cols, "y");
    void *st = c.stream(6);
    return launch(c, [&] {
        return fq_moe_dispatch(x, f8, scales, tokens, q.k, cols, q.rows, q.pos, q.src, y, st);
    });
}

// (y, weights, pos, src, out, stream)
PyObject *moe_combine(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    Call c(args, nargs, 6);
    long long rows = 0, cols = 0;
    if (!c.ok || !c.shape(0, "y", &rows, &cols)) return nullptr;
    const Sorted q(c, 2);
    const void *y = c.typed(0, at::kBFloat16, q.rows * cols, "y");
    const float *w = (const float *)c.typed(1, at::kFloat, q.tokens * q.k, "weights");
    void *out = c.typed(4, at::kBFloat16, q.tokens * cols, "out");
    void *st = c.stream(5);
    return launch(c, [&] {
        return fq_moe_combine(y, w, q.tokens, q.k, cols, q.rows, q.pos, out, st);
    });
}

// (dout, y, weights, pos, src, dy, dweights, stream)
PyObject *moe_combine_bwd(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    Call c(args, nargs, 8);
    long long tokens = 0, cols = 0;
    if (!c.ok || !c.shape(0, "dout", &tokens, &cols)) return nullptr;
    const Sorted q(c, 3);
    const void *dout = c.typed(0, at::kBFloat16, q.tokens * cols, "dout");
    const void *y = c.typed(1, at::kBFloat16, q.rows * cols, "y");
    const float *w = (const float *)c.typed(2, at::kFloat, q.tokens * q.k, "weights");
    void *dy = c.typed(5, at::kBFloat16, q.rows * cols, "dy");
    float *dw = (float *)c.typed(6, at::kFloat, q.tokens * q.k, "dweights");
    void *st = c.stream(7);
    return launch(c, [&] {
        return fq_moe_combine_bwd(dout, y, w, q.tokens, q.k, cols, q.rows, q.pos, q.src, dy, dw,
                                  st);
    });
}

// (address of the plan in host memory, the plan in device memory or None,
//  state_type, lr, beta1, beta2, eps, step, seed, grad_scale, stream, handle of
//  the stream that the device copy belongs to, what to call with another one)
PyObject *adamw_step(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    Call c(args, nargs, 13);
    if (!c.ok) return nullptr;
    const void *plan = (const void *)(uintptr_t)c.u64(0);
    const void *plan_device = c.bytes(1, 0, "plan");
    fq_adamw_hyper h = {};
    h.state_type = (int32_t)c.i64(2);
    h.lr = c.f64(3);
    h.beta1 = c.f64(4);
    h.beta2 = c.f64(5);
    h.eps = c.f64(6);
    h.step = c.i64(7);
    h.seed = c.u64(8);
    h.grad_scale = (const float *)c.typed(9, at::kFloat, 1, "grad_scale");
    void *st = c.stream(10);
    if (c.u64(11) != (uintptr_t)st && c.ok) {
        PyObject *r = PyObject_CallOneArg(args[12], args[10]);
        if (!r) return nullptr;
        Py_DECREF(r);
    }
    return launch(c, [&] { return fq_adamw_step_plan(&h, plan, plan_device, st); });
}

// A tensor without storage or strides throws where it is asked for them: that
// becomes a Python exception, and nothing is launched.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    try {
        return F(self, args, nargs);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_ValueError, "an operand cannot be read");
    }
    return nullptr;
}

#define FQ_METHOD(name) {#name, (PyCFunction)(void *)guarded<name>, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {
    FQ_METHOD(rmsnorm_fwd),  FQ_METHOD(rmsnorm_bwd),     FQ_METHOD(moe_sort),
    FQ_METHOD(moe_dispatch), FQ_METHOD(moe_combine),     FQ_METHOD(moe_combine_bwd),
    FQ_METHOD(adamw_step),   {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fq_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fq_binding()
{
    PyObject *torch_c = PyImport_ImportModule("torch._C");
    if (!torch_c) return nullptr;
    g_raw_stream = PyObject_GetAttrString(torch_c, "_cuda_getCurrentRawStream");
    g_device = PyObject_GetAttrString(torch_c, "_cuda_getDevice");
    g_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    Py_DECREF(torch_c);
    if (!g_raw_stream || !g_device || !g_cuda_stream) return nullptr;
    return PyModule_Create(&kModule);
}
