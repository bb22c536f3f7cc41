/* fastcall.c -- a CPython module that makes the attention operators' calls
 * from PyTorch tensors without ctypes.
 *
 * At decode sizes a call's kernels take a few microseconds, and reading the
 * tensors' attributes in Python and converting twenty arguments through ctypes
 * takes as long again.  Each function here checks its tensors (device, dtype,
 * dense trailing dimensions, sizes), reads the current stream and calls the C
 * entry point; it returns the entry point's status.  Whatever it does not
 * take (another dtype, a stride, a wrong size, any Python error) it answers
 * with None before anything is launched, and the caller's Python path then
 * does the call or raises the error that says what is wrong.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "../../include/moe_gb300.h"

static PyObject *s_dtype, *s_is_cuda, *s_shape, *s_stride, *s_data_ptr, *s_is_contiguous, *s_numel, *s_get_device, *s_ref, *s_S,
    *s_n_kv, *s_head_dim, *s_T;
static PyObject *t_bf16, *t_f32, *t_i32, *t_u8, *f_stream; /* torch.bfloat16, ..., torch._C._cuda_getCurrentRawStream */

/* The entry points, as addresses that setup() is given. */
static moe_status_t (*p_rope)(const void*, int, long long, int, int, int, int, const float*, const float*, float, const moe_rope_params*,
                              void*, long long, void*, long long, const moe_kv4_cache*, const int32_t*, moe_dev_status*, void*);
static moe_status_t (*p_read)(const moe_kv4_cache*, const int32_t*, int, void*, void*, moe_dev_status*, void*);
static moe_status_t (*p_attention)(const void*, long long, int, int, const moe_kv4_cache*, const int32_t*, int, float, int, void*,
                                   long long, float*, void*, size_t, moe_dev_status*, void*);
static moe_status_t (*p_reserve)(const moe_kv4_pool*, const int32_t*, void*, size_t, moe_dev_status*, void*);
static moe_status_t (*p_assign)(const moe_kv4_pool*, const int32_t*, moe_dev_status*, void*);
static moe_status_t (*p_compact)(const moe_kv4_pool*, int32_t*, void*, size_t, moe_dev_status*, void*);

/* Whether an attribute is that very object. */
static int attr_is(PyObject* o, PyObject* name, PyObject* want) {
    PyObject* v = PyObject_GetAttr(o, name);
    if (v == NULL) return 0;
    const int same = v == want;
    Py_DECREF(v);
    return same;
}
static int as_longlong(PyObject* v, long long* out) { /* takes the reference */
    if (v == NULL) return 0;
    *out = PyLong_AsLongLong(v);
    Py_DECREF(v);
    return !(*out == -1 && PyErr_Occurred());
}
static int attr_int(PyObject* o, PyObject* name, long long* out) { return as_longlong(PyObject_GetAttr(o, name), out); }
static int method_int(PyObject* o, PyObject* name, long long* out) { return as_longlong(PyObject_CallMethodNoArgs(o, name), out); }
static int address(PyObject* t, void** out) {
    PyObject* v = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (v == NULL) return 0;
    *out = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(v);
    Py_DECREF(v);
    return !PyErr_Occurred();
}

/* A dense CUDA tensor of the dtype and, if n >= 0, of n numbers; None gives NULL. */
static int dense(PyObject* t, PyObject* dtype, long long n, void** out) {
    long long have;
    if (t == Py_None) {
        *out = NULL;
        return 1;
    }
    if (!attr_is(t, s_is_cuda, Py_True) || !attr_is(t, s_dtype, dtype)) return 0;
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (c == NULL) return 0;
    Py_DECREF(c);
    if (c != Py_True) return 0;
    if (n >= 0 && (!method_int(t, s_numel, &have) || have != n)) return 0;
    return address(t, out);
}

/* A device status: two numbers, or NULL for None. */
static int status(PyObject* t, void** out) {
    long long n;
    return dense(t, t_i32, -1, out) && (t == Py_None || (method_int(t, s_numel, &n) && n >= 2));
}

/* Rows of numbers whose trailing dimensions are dense: address, rows, numbers of a row, leading dimension. */
static int rows(PyObject* t, PyObject* dtype, void** out, long long* n_rows, long long* width, long long* ld) {
    int ok = 0;
    PyObject *shape = NULL, *stride = NULL;
    if (!attr_is(t, s_is_cuda, Py_True) || !attr_is(t, s_dtype, dtype)) return 0;
    shape = PyObject_GetAttr(t, s_shape);
    stride = PyObject_CallMethodNoArgs(t, s_stride);
    if (shape != NULL && stride != NULL && PyTuple_Check(shape) && PyTuple_Check(stride) && PyTuple_GET_SIZE(shape) >= 2 &&
        PyTuple_GET_SIZE(shape) == PyTuple_GET_SIZE(stride)) {
        long long n = 1;
        Py_ssize_t k;
        ok = 1;
        for (k = PyTuple_GET_SIZE(shape) - 1; k > 0; --k) {
            const long long d = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, k)), s = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, k));
            if (s != n && d != 1) ok = 0;
            n *= d;
        }
        *n_rows = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0));
        *ld = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 0));
        if (*n_rows <= 1 && *ld < n) *ld = n;
        *width = n;
        if (PyErr_Occurred()) ok = 0;
    }
    Py_XDECREF(shape);
    Py_XDECREF(stride);
    return ok && address(t, out);
}

/* The current stream of the tensor's device. */
static int current_stream(PyObject* t, void** out) {
    PyObject* d = PyObject_CallMethodNoArgs(t, s_get_device);
    if (d == NULL) return 0;
    PyObject* s = PyObject_CallOneArg(f_stream, d);
    Py_DECREF(d);
    if (s == NULL) return 0;
    *out = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(s);
    Py_DECREF(s);
    return !PyErr_Occurred();
}

/* A handle's parameter struct (its _ref), or NULL for None. */
static int handle(PyObject* h, void** out) {
    long long v;
    if (h == Py_None) {
        *out = NULL;
        return 1;
    }
    if (!attr_int(h, s_ref, &v)) return 0;
    *out = (void*)(uintptr_t)v;
    return 1;
}
static int fits_int(long long v) { return v >= INT32_MIN && v <= INT32_MAX; }

static PyObject* decline(void) {
    PyErr_Clear();
    Py_RETURN_NONE;
}

/* qkv, n_q, n_kv, q_out, k_out, q_weight, k_weight, eps, rope, cache, q_start, st */
static PyObject* qk_norm_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void *x, *q = NULL, *k = NULL, *qw, *kw, *rope, *cache, *qs = NULL, *st, *stream;
    long long T, width, ld, Tq, wq, ld_q = 0, Tk, wk, ld_k = 0, S, heads, D, rope_T;
    (void)self;
    if (n != 12) return decline();
    const long long n_q = PyLong_AsLongLong(a[1]), n_kv = PyLong_AsLongLong(a[2]);
    const double eps = PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred() || n_q < 0 || n_kv < 1 || n_q > 4096 || n_kv > 4096) return decline();
    const int bf = attr_is(a[0], s_dtype, t_bf16);
    PyObject* dt = bf ? t_bf16 : t_f32;
    if (!rows(a[0], dt, &x, &T, &width, &ld)) return decline();
    heads = n_q + 2 * n_kv;
    D = width / heads;
    if (width % heads != 0 || !fits_int(T) || !fits_int(D)) return decline();
    if (n_q > 0 && (!rows(a[3], dt, &q, &Tq, &wq, &ld_q) || Tq != T || wq != n_q * D)) return decline();
    if (a[4] != Py_None && (!rows(a[4], dt, &k, &Tk, &wk, &ld_k) || Tk != T || wk != n_kv * D)) return decline();
    if (!dense(a[5], t_f32, D, &qw) || !dense(a[6], t_f32, D, &kw)) return decline();
    if (!handle(a[8], &rope) || !handle(a[9], &cache)) return decline();
    if (rope != NULL) {
        PyObject* rt = PyObject_GetAttr(a[8], s_T);
        if (rt == NULL) return decline();
        if (rt == Py_None) Py_DECREF(rt);
        else if (!as_longlong(rt, &rope_T) || rope_T != T) return decline();
    }
    if (cache != NULL && (!attr_int(a[9], s_S, &S) || a[10] == Py_None || !dense(a[10], t_i32, S + 1, &qs))) return decline();
    if (!status(a[11], &st) || !current_stream(a[0], &stream)) return decline();
    return PyLong_FromLong(p_rope(x, bf ? MOE_DTYPE_BF16 : MOE_DTYPE_F32, ld, (int)T, (int)n_q, (int)n_kv, (int)D, qw, kw, (float)eps, rope,
                                  q, ld_q, k, ld_k, cache, qs, st, stream));
}

/* cache, q_start, k_out, v_out, st */
static PyObject* kv4_read(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void *cache, *qs, *out[2] = {NULL, NULL}, *st, *stream;
    long long S, kv, D, T = -1, Tt, w, ld;
    int i;
    (void)self;
    if (n != 5 || !handle(a[0], &cache) || cache == NULL || !attr_int(a[0], s_S, &S) || !attr_int(a[0], s_n_kv, &kv) ||
        !attr_int(a[0], s_head_dim, &D) || a[1] == Py_None || !dense(a[1], t_i32, S + 1, &qs))
        return decline();
    for (i = 0; i < 2; ++i) {
        if (a[2 + i] == Py_None) continue;
        if (!rows(a[2 + i], t_bf16, &out[i], &Tt, &w, &ld) || w != kv * D || (Tt > 1 && ld != w) || (T >= 0 && T != Tt)) return decline();
        T = Tt;
    }
    if (T < 0 || !fits_int(T) || !status(a[4], &st) || !current_stream(a[1], &stream)) return decline();
    return PyLong_FromLong(p_read(cache, qs, (int)T, out[0], out[1], st, stream));
}

/* q, cache, q_start, out, scale, max_new, window, lse, workspace, st */
static PyObject* attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void *q, *cache, *qs, *out, *lse, *ws, *st, *stream;
    long long T, w, ld, To, wo, ldo, S, D, bytes, n_q;
    (void)self;
    if (n != 10) return decline();
    const double scale = PyFloat_AsDouble(a[4]);
    const long long max_new = PyLong_AsLongLong(a[5]), window = PyLong_AsLongLong(a[6]);
    if (PyErr_Occurred() || !fits_int(max_new) || !fits_int(window)) return decline();
    if (!handle(a[1], &cache) || cache == NULL || !attr_int(a[1], s_S, &S) || !attr_int(a[1], s_head_dim, &D)) return decline();
    if (!rows(a[0], t_bf16, &q, &T, &w, &ld) || D < 1 || w % D != 0 || !fits_int(T) || !fits_int(w)) return decline();
    if (!rows(a[3], t_bf16, &out, &To, &wo, &ldo) || To != T || wo != w) return decline();
    n_q = w / D;
    if (a[2] == Py_None || !dense(a[2], t_i32, S + 1, &qs) || !dense(a[7], t_f32, T * n_q, &lse)) return decline();
    if (a[8] == Py_None || !dense(a[8], t_u8, -1, &ws) || !method_int(a[8], s_numel, &bytes)) return decline();
    if (!status(a[9], &st) || !current_stream(a[0], &stream)) return decline();
    return PyLong_FromLong(p_attention(q, ld, (int)T, (int)n_q, cache, qs, (int)max_new, (float)scale, (int)window, out, ldo, lse, ws,
                                       (size_t)bytes, st, stream));
}

/* pool, vector, workspace or None, st; `vector` may be None where the entry point takes NULL */
static PyObject* pool_call(PyObject* const* a, Py_ssize_t n, int which) {
    void *pool, *v, *ws = NULL, *st, *stream;
    long long S, bytes = 0;
    if (n != 4 || !handle(a[0], &pool) || pool == NULL || !attr_int(a[0], s_S, &S)) return decline();
    if (!dense(a[1], t_i32, which == 2 ? -1 : S, &v)) return decline();
    if (which != 1 && (a[2] == Py_None || !dense(a[2], t_u8, -1, &ws) || !method_int(a[2], s_numel, &bytes))) return decline();
    if (which != 2 && a[1] == Py_None) return decline();
    if (!status(a[3], &st) || !current_stream(which == 2 ? a[2] : a[1], &stream)) return decline();
    if (which == 0) return PyLong_FromLong(p_reserve(pool, v, ws, (size_t)bytes, st, stream));
    if (which == 1) return PyLong_FromLong(p_assign(pool, v, st, stream));
    return PyLong_FromLong(p_compact(pool, v, ws, (size_t)bytes, st, stream));
}
static PyObject* reserve(PyObject* s, PyObject* const* a, Py_ssize_t n) { (void)s; return pool_call(a, n, 0); }
static PyObject* assign(PyObject* s, PyObject* const* a, Py_ssize_t n) { (void)s; return pool_call(a, n, 1); }
static PyObject* compact(PyObject* s, PyObject* const* a, Py_ssize_t n) { (void)s; return pool_call(a, n, 2); }

/* setup(torch.bfloat16, torch.float32, torch.int32, torch.uint8, raw-stream function, six addresses) */
static PyObject* setup(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    uintptr_t p[6];
    int i;
    (void)self;
    if (n != 11) {
        PyErr_SetString(PyExc_TypeError, "setup takes eleven arguments");
        return NULL;
    }
    for (i = 0; i < 6; ++i) p[i] = (uintptr_t)PyLong_AsUnsignedLongLong(a[5 + i]);
    if (PyErr_Occurred()) return NULL;
    t_bf16 = Py_NewRef(a[0]);
    t_f32 = Py_NewRef(a[1]);
    t_i32 = Py_NewRef(a[2]);
    t_u8 = Py_NewRef(a[3]);
    f_stream = Py_NewRef(a[4]);
    memcpy(&p_rope, &p[0], sizeof p[0]);
    memcpy(&p_read, &p[1], sizeof p[0]);
    memcpy(&p_attention, &p[2], sizeof p[0]);
    memcpy(&p_reserve, &p[3], sizeof p[0]);
    memcpy(&p_assign, &p[4], sizeof p[0]);
    memcpy(&p_compact, &p[5], sizeof p[0]);
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, NULL},
    {"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, NULL},
    {"kv4_read", (PyCFunction)(void (*)(void))kv4_read, METH_FASTCALL, NULL},
    {"attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, NULL},
    {"reserve", (PyCFunction)(void (*)(void))reserve, METH_FASTCALL, NULL},
    {"assign", (PyCFunction)(void (*)(void))assign, METH_FASTCALL, NULL},
    {"compact", (PyCFunction)(void (*)(void))compact, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) {
    static const struct {
        PyObject** to;
        const char* name;
    } names[] = {{&s_dtype, "dtype"},       {&s_is_cuda, "is_cuda"},
                 {&s_shape, "shape"},       {&s_stride, "stride"},
                 {&s_data_ptr, "data_ptr"}, {&s_is_contiguous, "is_contiguous"},
                 {&s_numel, "numel"},       {&s_get_device, "get_device"},
                 {&s_ref, "_ref"},          {&s_S, "S"},
                 {&s_n_kv, "n_kv"},         {&s_head_dim, "head_dim"},
                 {&s_T, "T"}};
    size_t i;
    for (i = 0; i < sizeof names / sizeof names[0]; ++i) {
        *names[i].to = PyUnicode_InternFromString(names[i].name);
        if (*names[i].to == NULL) return NULL;
    }
    return PyModule_Create(&module);
}
