/* calls.c — the short way from the Python binding into the library, for the calls of
 * include/qmoe.h that take a few microseconds on the GPU: routing, sorting by expert,
 * weighted sums and the 4-bit products.  (Through ctypes and checks in Python a call of
 * six arrays cost the host 8 us, the kernel 3.)
 *
 * A function here takes the arguments of its namesake in the binding by position, makes
 * the checks that hold for nearly every call (arrays on the current device, of the
 * type named, contiguous, large enough) and calls the library.  Whatever fails them, is
 * an address instead of a tensor, or names a stream, it leaves alone: it returns None and
 * the binding goes its long way, which accepts or refuses with a message.  A status other
 * than QMOE_OK is returned as such.
 *
 * bind(addresses, dtypes, get_device, get_stream) hands over the library's functions, in
 * the order of enum fn, the torch dtypes (f32, bf16, f16, int32, uint8), and torch's
 * functions for the current device and its current stream. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/qmoe.h"

enum fn { ROUTE, ROUTE_BACKWARD, PERMUTE, COMBINE, COMBINE_BACKWARD, W4_MM, W4_MM_GROUPED, N_FN };
enum type { T_F32, T_BF16, T_F16, T_I32, T_U8, T_ANY, N_TYPES = T_ANY };

static void* address[N_FN];
static PyObject *dtype[N_TYPES], *get_device, *get_stream;
static PyObject *s_get_device, *s_dtype, *s_is_contiguous, *s_numel, *s_data_ptr, *s_nbytes;

static int type_of(int64_t code) {
    return code == QMOE_F32 ? T_F32 : code == QMOE_BF16 ? T_BF16 : code == QMOE_F16 ? T_F16 : -1;
}

/* What a call gathers: the device its tensors are on (-1 before the first). */
typedef struct {
    long dev;
    int ok;   /* 0: the long way */
} call;

static int64_t call_int(PyObject* o, PyObject* name, call* c) {
    PyObject* r = PyObject_CallMethodNoArgs(o, name);
    int64_t v = -1;
    if (r) {
        v = PyLong_AsLongLong(r);
        Py_DECREF(r);
    }
    if (PyErr_Occurred()) {
        PyErr_Clear();
        c->ok = 0;
    }
    return v;
}

/* Address of a tensor of at least `need` elements of `type`; null for None. */
static void* array(PyObject* t, int type, int64_t need, call* c) {
    if (!c->ok || t == Py_None) return NULL;
    if (PyLong_Check(t) || type < 0) {
        c->ok = 0;
        return NULL;
    }
    const int64_t dev = call_int(t, s_get_device, c);
    if (!c->ok || dev < 0 || (c->dev >= 0 && dev != c->dev)) {
        c->ok = 0;
        return NULL;
    }
    c->dev = (long)dev;
    if (type != T_ANY) {
        PyObject* d = PyObject_GetAttr(t, s_dtype);
        if (d != dtype[type]) c->ok = 0;
        if (!d) PyErr_Clear();
        Py_XDECREF(d);
        if (!c->ok) return NULL;
    }
    PyObject* r = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (r != Py_True) c->ok = 0;
    if (!r) PyErr_Clear();
    Py_XDECREF(r);
    if (!c->ok) return NULL;
    if (call_int(t, s_numel, c) < need) c->ok = 0;
    if (!c->ok) return NULL;
    return (void*)(intptr_t)call_int(t, s_data_ptr, c);
}

/* The current stream of the tensors' device, which has to be the current one. */
static void* stream_of(PyObject* given, call* c) {
    if (!c->ok || given != Py_None || c->dev < 0) {
        c->ok = 0;
        return NULL;
    }
    PyObject* d = PyObject_CallNoArgs(get_device);
    PyObject* s = NULL;
    if (d && PyLong_AsLong(d) == c->dev) s = PyObject_CallOneArg(get_stream, d);
    void* p = s ? (void*)(intptr_t)PyLong_AsLongLong(s) : NULL;
    if (!s || PyErr_Occurred()) {
        PyErr_Clear();
        c->ok = 0;
    }
    Py_XDECREF(d);
    Py_XDECREF(s);
    return p;
}

/* Integer arguments; anything that is no int of 64 bits goes the long way. */
static int64_t integer(PyObject* o, call* c) {
    if (!PyLong_Check(o)) {
        c->ok = 0;
        return 0;
    }
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        c->ok = 0;
    }
    return v;
}
/* Sizes: those whose products could pass 64 bits go the long way too (and are refused). */
static int64_t size(PyObject* o, call* c) {
    const int64_t v = integer(o, c);
    if (v < 0 || v > 0x7fffffff) c->ok = 0;
    return v;
}

#define ARGS(n)                                                                     \
    call c = {-1, 1};                                                               \
    if (count != (n)) {                                                             \
        PyErr_Format(PyExc_TypeError, "%d arguments are needed, not %zd", n, count); \
        return NULL;                                                                \
    }                                                                               \
    (void)self
#define ANSWER(call_expr)         \
    do {                          \
        long status;              \
        if (!c.ok) Py_RETURN_NONE; \
        Py_BEGIN_ALLOW_THREADS    \
        status = (long)(call_expr); \
        Py_END_ALLOW_THREADS      \
        return PyLong_FromLong(status); \
    } while (0)

/* ltype, logits, n_tokens, num_experts, top_k, topk_idx, topk_w, flags, stream */
static PyObject* route(PyObject* self, PyObject* const* a, Py_ssize_t count) {
    ARGS(9);
    const int64_t lt = integer(a[0], &c), t = size(a[2], &c), e = size(a[3], &c),
                  k = size(a[4], &c), flags = size(a[7], &c);
    if (!c.ok || k > 0xffff) Py_RETURN_NONE;
    void* x = array(a[1], type_of(lt), t * e, &c);
    void* idx = array(a[5], T_I32, t * k, &c);
    void* w = array(a[6], T_F32, t * k, &c);
    void* st = stream_of(a[8], &c);
    ANSWER(((__typeof__(&moe_route))address[ROUTE])((int)lt, x, t, (int32_t)e, e, (int32_t)k,
                                                    (int32_t)flags, idx, w, st));
}

/* ltype, logits, n_tokens, num_experts, top_k, topk_idx, topk_w, grad_w, grad_logits, flags,
 * stream */
static PyObject* route_backward(PyObject* self, PyObject* const* a, Py_ssize_t count) {
    ARGS(11);
    const int64_t lt = integer(a[0], &c), t = size(a[2], &c), e = size(a[3], &c),
                  k = size(a[4], &c), flags = size(a[9], &c);
    if (!c.ok || k > 0xffff) Py_RETURN_NONE;
    void* x = array(a[1], type_of(lt), t * e, &c);
    void* idx = array(a[5], T_I32, t * k, &c);
    void* w = array(a[6], T_F32, t * k, &c);
    void* dw = array(a[7], T_F32, t * k, &c);
    void* g = array(a[8], type_of(lt), t * e, &c);
    void* st = stream_of(a[10], &c);
    ANSWER(((__typeof__(&moe_route_backward))address[ROUTE_BACKWARD])(
        (int)lt, x, t, (int32_t)e, e, (int32_t)k, (int32_t)flags, idx, w, dw, g, e, st));
}

/* xtype, x, n_tokens, cols, topk_idx, num_experts, top_k, rows, offsets, pos, ws, stream */
static PyObject* permute(PyObject* self, PyObject* const* a, Py_ssize_t count) {
    ARGS(12);
    const int64_t xt = integer(a[0], &c), t = size(a[2], &c), h = size(a[3], &c),
                  e = size(a[5], &c), k = size(a[6], &c);
    if (!c.ok || k > 0xffff || h > 0xffffff || a[10] == Py_None) Py_RETURN_NONE;
    void* x = array(a[1], type_of(xt), t * h, &c);
    void* idx = array(a[4], T_I32, t * k, &c);
    void* rows = t * k <= 0x7fffffff ? array(a[7], type_of(xt), t * k * h, &c) : (c.ok = 0, NULL);
    void* off = array(a[8], T_I32, e + 1, &c);
    void* pos = array(a[9], T_I32, t * k, &c);
    void* ws = array(a[10], T_ANY, 0, &c);
    int64_t bytes = 0;
    if (c.ok) {
        PyObject* n = PyObject_GetAttr(a[10], s_nbytes);
        bytes = n ? PyLong_AsLongLong(n) : -1;
        Py_XDECREF(n);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            c.ok = 0;
        }
    }
    void* st = stream_of(a[11], &c);
    ANSWER(((__typeof__(&moe_permute))address[PERMUTE])((int)xt, x, t, h, h, idx, (int32_t)e,
                                                        (int32_t)k, rows, h, off, pos, ws,
                                                        (size_t)bytes, st));
}

/* ytype, y, n_rows, cols, pos, topk_w, n_tokens, top_k, otype, residual, out, stream */
static PyObject* combine(PyObject* self, PyObject* const* a, Py_ssize_t count) {
    ARGS(12);
    const int64_t yt = integer(a[0], &c), n = size(a[2], &c), h = size(a[3], &c),
                  t = size(a[6], &c), k = size(a[7], &c), ot = integer(a[8], &c);
    if (!c.ok || k > 0xffff) Py_RETURN_NONE;
    void* y = array(a[1], type_of(yt), n * h, &c);
    void* pos = array(a[4], T_I32, t * k, &c);
    void* w = array(a[5], T_F32, t * k, &c);
    void* res = array(a[9], type_of(ot), t * h, &c);
    void* out = array(a[10], type_of(ot), t * h, &c);
    void* st = stream_of(a[11], &c);
    ANSWER(((__typeof__(&moe_combine))address[COMBINE])((int)yt, y, n, h, h, pos, w, t, (int32_t)k,
                                                        (int)ot, res, out, h, st));
}

/* ytype, y, n_rows, cols, pos, topk_w, n_tokens, top_k, otype, grad_out, grad_y, grad_w,
 * stream */
static PyObject* combine_backward(PyObject* self, PyObject* const* a, Py_ssize_t count) {
    ARGS(13);
    const int64_t yt = integer(a[0], &c), n = size(a[2], &c), h = size(a[3], &c),
                  t = size(a[6], &c), k = size(a[7], &c), ot = integer(a[8], &c);
    if (!c.ok || k > 0xffff) Py_RETURN_NONE;
    void* y = array(a[1], type_of(yt), n * h, &c);
    void* pos = array(a[4], T_I32, t * k, &c);
    void* w = array(a[5], T_F32, t * k, &c);
    void* go = array(a[9], type_of(ot), t * h, &c);
    void* gy = array(a[10], type_of(yt), n * h, &c);
    void* gw = array(a[11], T_F32, t * k, &c);
    void* st = stream_of(a[12], &c);
    ANSWER(((__typeof__(&moe_combine_backward))address[COMBINE_BACKWARD])(
        (int)yt, y, n, h, h, pos, w, t, (int32_t)k, (int)ot, go, h, gy, h, gw, st));
}

/* The 4-bit products: W, stype, scale, zero, scale_cols, num_groups (-1: w4_mm), rows, cols,
 * xtype, x, n_rows, offsets, ytype, y, stream */
static PyObject* w4(PyObject* self, PyObject* const* a, Py_ssize_t count) {
    ARGS(15);
    const int64_t stype = integer(a[1], &c), sc = size(a[4], &c), e = integer(a[5], &c),
                  n = size(a[6], &c), k = size(a[7], &c), xt = integer(a[8], &c),
                  m = size(a[10], &c), yt = integer(a[12], &c);
    if (!c.ok || sc == 0 || e < -1 || e == 0 || e > 0xffff || k > 0xffffff) Py_RETURN_NONE;
    const int64_t rows = (e > 0 ? e : 1) * n;
    if (rows > (1LL << 38)) Py_RETURN_NONE;
    void* W = array(a[0], T_U8, (rows * k + 1) / 2, &c);
    void* s = array(a[2], type_of(stype), rows * (k / sc), &c);
    void* z = array(a[3], T_U8, rows * (k / sc), &c);
    void* x = array(a[9], type_of(xt), m * k, &c);
    void* off = e > 0 ? array(a[11], T_I32, e + 1, &c) : NULL;
    void* y = array(a[13], type_of(yt), m * n, &c);
    void* st = stream_of(a[14], &c);
    if (e > 0) {
        ANSWER(((__typeof__(&w4_mm_grouped))address[W4_MM_GROUPED])(
            W, (int)stype, s, z, (int32_t)sc, (int32_t)e, n, k, (int)xt, x, m, k, off, (int)yt, y, n,
            st));
    }
    ANSWER(((__typeof__(&w4_mm))address[W4_MM])(W, (int)stype, s, z, (int32_t)sc, n, k, (int)xt, x,
                                                m, k, (int)yt, y, n, st));
}

static PyObject* bind(PyObject* self, PyObject* args) {
    PyObject *addr, *types, *dev, *st;
    (void)self;
    if (!PyArg_ParseTuple(args, "O!O!OO", &PyTuple_Type, &addr, &PyTuple_Type, &types, &dev, &st))
        return NULL;
    if (PyTuple_GET_SIZE(addr) != N_FN || PyTuple_GET_SIZE(types) != N_TYPES) {
        PyErr_SetString(PyExc_ValueError, "bind: addresses or dtypes");
        return NULL;
    }
    for (int i = 0; i < N_FN; ++i) {
        address[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addr, i));
        if (PyErr_Occurred()) return NULL;
    }
    for (int i = 0; i < N_TYPES; ++i) {
        Py_INCREF(PyTuple_GET_ITEM(types, i));
        Py_XSETREF(dtype[i], PyTuple_GET_ITEM(types, i));
    }
    Py_INCREF(dev);
    Py_XSETREF(get_device, dev);
    Py_INCREF(st);
    Py_XSETREF(get_stream, st);
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, NULL},
    {"route", (PyCFunction)(void (*)(void))route, METH_FASTCALL, NULL},
    {"route_backward", (PyCFunction)(void (*)(void))route_backward, METH_FASTCALL, NULL},
    {"permute", (PyCFunction)(void (*)(void))permute, METH_FASTCALL, NULL},
    {"combine", (PyCFunction)(void (*)(void))combine, METH_FASTCALL, NULL},
    {"combine_backward", (PyCFunction)(void (*)(void))combine_backward, METH_FASTCALL, NULL},
    {"w4", (PyCFunction)(void (*)(void))w4, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void) {
    struct { PyObject** at; const char* name; } names[] = {
        {&s_get_device, "get_device"}, {&s_dtype, "dtype"}, {&s_is_contiguous, "is_contiguous"},
        {&s_numel, "numel"}, {&s_data_ptr, "data_ptr"}, {&s_nbytes, "nbytes"}};
    for (size_t i = 0; i < sizeof names / sizeof *names; ++i)
        if (!(*names[i].at = PyUnicode_InternFromString(names[i].name))) return NULL;
    return PyModule_Create(&module);
}
