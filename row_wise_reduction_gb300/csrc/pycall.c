/*
 * _rowops_call: the Python binding's calls into librowops.so for the entry
 * points whose small, launch-bound calls are dominated by host time. It only
 * marshals arguments: Python ints and floats become the C ABI's pointers,
 * sizes and scalars, the call runs with the GIL released, and its status comes
 * back as an int. The function addresses are handed over once by the ctypes
 * loader (bind), so this module does not link the library itself.
 *
 * A ctypes call with seven typed arguments costs about 2 us of Python time;
 * through this module, about 0.1 us.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

typedef int (*softmax_fn)(const void*, void*, int64_t, int64_t, int64_t, int, void*);
typedef int (*ln_fn)(const void*, void*, const void*, const void*, float, int64_t, int64_t, int64_t, int, void*);

static softmax_fn g_softmax = NULL;
static ln_fn g_ln = NULL;
static ln_fn g_ln_erf = NULL;

static int as_ptr(PyObject* o, void** out) {
    if (o == Py_None) {
        *out = NULL;
        return 0;
    }
    *out = PyLong_AsVoidPtr(o);
    return (*out == NULL && PyErr_Occurred()) ? -1 : 0;
}

static int as_i64(PyObject* o, int64_t* out) {
    long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) return -1;
    *out = (int64_t)v;
    return 0;
}

static int nargs_ok(Py_ssize_t n, Py_ssize_t want, const char* name) {
    if (n == want) return 1;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", name, want, n);
    return 0;
}

/* bind(softmax, layernorm_gelu, layernorm_gelu_erf): function addresses */
static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void *s, *l, *e;
    (void)self;
    if (!nargs_ok(n, 3, "bind") || as_ptr(a[0], &s) || as_ptr(a[1], &l) || as_ptr(a[2], &e)) return NULL;
    g_softmax = (softmax_fn)s;
    g_ln = (ln_fn)l;
    g_ln_erf = (ln_fn)e;
    Py_RETURN_NONE;
}

/* softmax(x, y, M, N, ld, dtype, stream) -> status */
static PyObject* softmax(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void *x, *y, *st;
    int64_t M, N, ld, dt;
    int r;
    (void)self;
    if (!g_softmax) return PyErr_Format(PyExc_RuntimeError, "_rowops_call is not bound");
    if (!nargs_ok(n, 7, "softmax") || as_ptr(a[0], &x) || as_ptr(a[1], &y) || as_i64(a[2], &M) ||
        as_i64(a[3], &N) || as_i64(a[4], &ld) || as_i64(a[5], &dt) || as_ptr(a[6], &st))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    r = g_softmax(x, y, M, N, ld, (int)dt, st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

static PyObject* ln_call(ln_fn f, const char* name, PyObject* const* a, Py_ssize_t n) {
    void *x, *y, *w, *b, *st;
    int64_t M, N, ld, dt;
    double eps;
    int r;
    if (!f) return PyErr_Format(PyExc_RuntimeError, "_rowops_call is not bound");
    if (!nargs_ok(n, 10, name) || as_ptr(a[0], &x) || as_ptr(a[1], &y) || as_ptr(a[2], &w) || as_ptr(a[3], &b))
        return NULL;
    eps = PyFloat_AsDouble(a[4]);
    if (eps == -1.0 && PyErr_Occurred()) return NULL;
    if (as_i64(a[5], &M) || as_i64(a[6], &N) || as_i64(a[7], &ld) || as_i64(a[8], &dt) || as_ptr(a[9], &st))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    r = f(x, y, w, b, (float)eps, M, N, ld, (int)dt, st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
}

/* layernorm_gelu(x, y, w, b, eps, M, N, ld, dtype, stream) -> status (w, b may be None) */
static PyObject* layernorm_gelu(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    return ln_call(g_ln, "layernorm_gelu", a, n);
}

static PyObject* layernorm_gelu_erf(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    return ln_call(g_ln_erf, "layernorm_gelu_erf", a, n);
}

/*
 * The training and serving operators' entry points and workspace queries: the
 * same marshalling, one function each.
 */
static int as_f32(PyObject* o, float* out) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) return -1;
    *out = (float)v;
    return 0;
}

static int as_u64(PyObject* o, uint64_t* out) {
    *out = PyLong_AsUnsignedLongLongMask(o);
    return (*out == (uint64_t)-1 && PyErr_Occurred()) ? -1 : 0;
}

#define MOST_ARGS 26
#define BOUND 14
typedef struct {
    void* p[MOST_ARGS];
    int64_t i[MOST_ARGS];
    uint64_t u[MOST_ARGS];
    float f[MOST_ARGS];
} args_t;

/* Arguments by a form: p pointer or None, i integer, u 64 bits (taken mod 2^64), f float; each
 * lands at its own position of the array of its kind. */
static int take(const char* name, const char* form, PyObject* const* a, Py_ssize_t n, args_t* v) {
    Py_ssize_t k;
    if (!nargs_ok(n, (Py_ssize_t)strlen(form), name)) return -1;
    for (k = 0; k < n; ++k) {
        int bad = form[k] == 'p' ? as_ptr(a[k], &v->p[k])
                : form[k] == 'i' ? as_i64(a[k], &v->i[k])
                : form[k] == 'u' ? as_u64(a[k], &v->u[k]) : as_f32(a[k], &v->f[k]);
        if (bad) return -1;
    }
    return 0;
}

/* the addresses, in the order of bind_operators' arguments */
static void* g_bound[BOUND];

typedef size_t (*gn_bytes_fn)(int64_t, int64_t, int64_t, int64_t, int);
typedef size_t (*rows_bytes_fn)(int64_t, int64_t, int);
typedef int (*gn_fn)(const void*, void*, const void*, const void*, float, int64_t, int64_t, int64_t, int64_t, int64_t,
                     int, float*, int, void*, size_t, void*);
typedef int (*gn_bwd_fn)(const void*, const void*, const void*, const void*, const float*, void*, float*, float*,
                         int64_t, int64_t, int64_t, int64_t, int64_t, int, int, void*, size_t, void*);
typedef int (*drop_fn)(const void*, const void*, const void*, void*, float, uint64_t, uint64_t, const void*, int64_t,
                       int64_t, int64_t, int, void*);
typedef int (*drop_bwd_fn)(const void*, void*, float*, float, uint64_t, uint64_t, const void*, int64_t, int64_t,
                           int64_t, int, void*, size_t, void*);
typedef int (*balance_fn)(const void*, const void*, int, const void*, float, float*, void*, int64_t, int64_t, int64_t,
                          int64_t, int, void*, size_t, void*);
typedef int (*balance_bwd_fn)(const void*, const void*, const float*, const void*, float, void*, int64_t, int64_t,
                              int64_t, int64_t, int, void*);
typedef int (*quant_fn)(const void*, const void*, void*, float*, void*, const void*, float, int64_t, int64_t, int64_t,
                        int64_t, int64_t, int, void*);
typedef size_t (*paged_bytes_fn)(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int);
typedef int (*paged_fn)(const void*, const void*, const void*, const void*, const void*, void*, float*, float, int64_t,
                        int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                        int64_t, int64_t, int64_t, int, void*, size_t, void*);
typedef int (*sample_fn)(const void*, const void*, const void*, float, const void*, int32_t, const void*, float,
                         const void*, float, void*, float*, int64_t, int64_t, int64_t, int, void*);

static PyObject* bind_operators(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    int k;
    (void)self;
    if (!nargs_ok(n, BOUND, "bind_operators")) return NULL;
    for (k = 0; k < BOUND; ++k)
        if (as_ptr(a[k], &g_bound[k])) return NULL;
    Py_RETURN_NONE;
}

#define CALL(name, slot, form, expr)                                                                          \
    static PyObject* name(PyObject* self, PyObject* const* a, Py_ssize_t n) {                                 \
        args_t v;                                                                                             \
        int r;                                                                                                \
        (void)self;                                                                                           \
        if (!g_bound[slot]) return PyErr_Format(PyExc_RuntimeError, "_rowops_call is not bound");             \
        if (take(#name, form, a, n, &v)) return NULL;                                                         \
        Py_BEGIN_ALLOW_THREADS                                                                                \
        r = (expr);                                                                                           \
        Py_END_ALLOW_THREADS                                                                                  \
        return PyLong_FromLong(r);                                                                            \
    }
#define BYTES(name, slot, form, expr)                                                                         \
    static PyObject* name(PyObject* self, PyObject* const* a, Py_ssize_t n) {                                 \
        args_t v;                                                                                             \
        (void)self;                                                                                           \
        if (!g_bound[slot]) return PyErr_Format(PyExc_RuntimeError, "_rowops_call is not bound");             \
        if (take(#name, form, a, n, &v)) return NULL;                                                         \
        return PyLong_FromSize_t(expr);                                                                       \
    }

BYTES(groupnorm_act_workspace_bytes, 0, "iiiii",
      ((gn_bytes_fn)g_bound[0])(v.i[0], v.i[1], v.i[2], v.i[3], (int)v.i[4]))
CALL(groupnorm_act, 1, "ppppfiiiiiipipip",
     ((gn_fn)g_bound[1])(v.p[0], v.p[1], v.p[2], v.p[3], v.f[4], v.i[5], v.i[6], v.i[7], v.i[8], v.i[9],
                         (int)v.i[10], (float*)v.p[11], (int)v.i[12], v.p[13], (size_t)v.i[14], v.p[15]))
BYTES(groupnorm_act_backward_workspace_bytes, 2, "iiiii",
      ((gn_bytes_fn)g_bound[2])(v.i[0], v.i[1], v.i[2], v.i[3], (int)v.i[4]))
CALL(groupnorm_act_backward, 3, "ppppppppiiiiiiipip",
     ((gn_bwd_fn)g_bound[3])(v.p[0], v.p[1], v.p[2], v.p[3], (float*)v.p[4], v.p[5], (float*)v.p[6],
                             (float*)v.p[7], v.i[8], v.i[9], v.i[10], v.i[11], v.i[12], (int)v.i[13],
                             (int)v.i[14], v.p[15], (size_t)v.i[16], v.p[17]))
CALL(bias_dropout_residual, 4, "ppppfuupiiiip",
     ((drop_fn)g_bound[4])(v.p[0], v.p[1], v.p[2], v.p[3], v.f[4], v.u[5], v.u[6], v.p[7], v.i[8], v.i[9],
                           v.i[10], (int)v.i[11], v.p[12]))
BYTES(bias_dropout_residual_backward_workspace_bytes, 5, "iii",
      ((rows_bytes_fn)g_bound[5])(v.i[0], v.i[1], (int)v.i[2]))
CALL(bias_dropout_residual_backward, 6, "pppfuupiiiipip",
     ((drop_bwd_fn)g_bound[6])(v.p[0], v.p[1], (float*)v.p[2], v.f[3], v.u[4], v.u[5], v.p[6], v.i[7], v.i[8],
                               v.i[9], (int)v.i[10], v.p[11], (size_t)v.i[12], v.p[13]))
CALL(router_balance_loss, 7, "ppipfppiiiiipip",
     ((balance_fn)g_bound[7])(v.p[0], v.p[1], (int)v.i[2], v.p[3], v.f[4], (float*)v.p[5], v.p[6], v.i[7],
                              v.i[8], v.i[9], v.i[10], (int)v.i[11], v.p[12], (size_t)v.i[13], v.p[14]))
CALL(router_balance_loss_backward, 8, "ppppfpiiiiip",
     ((balance_bwd_fn)g_bound[8])(v.p[0], v.p[1], (float*)v.p[2], v.p[3], v.f[4], v.p[5], v.i[6], v.i[7], v.i[8],
                                  v.i[9], (int)v.i[10], v.p[11]))
BYTES(router_balance_loss_workspace_bytes, 9, "iii",
      ((rows_bytes_fn)g_bound[9])(v.i[0], v.i[1], (int)v.i[2]))
CALL(rmsnorm_quant, 10, "ppppppfiiiiiip",
     ((quant_fn)g_bound[10])(v.p[0], v.p[1], v.p[2], (float*)v.p[3], v.p[4], v.p[5], v.f[6], v.i[7], v.i[8], v.i[9],
                             v.i[10], v.i[11], (int)v.i[12], v.p[13]))
BYTES(paged_attention_workspace_bytes, 11, "iiiiiiii",
      ((paged_bytes_fn)g_bound[11])(v.i[0], v.i[1], v.i[2], v.i[3], v.i[4], v.i[5], v.i[6], (int)v.i[7]))
CALL(paged_attention, 12, "pppppppfiiiiiiiiiiiiiiipip",
     ((paged_fn)g_bound[12])(v.p[0], v.p[1], v.p[2], v.p[3], v.p[4], v.p[5], (float*)v.p[6], v.f[7], v.i[8], v.i[9],
                             v.i[10], v.i[11], v.i[12], v.i[13], v.i[14], v.i[15], v.i[16], v.i[17], v.i[18], v.i[19],
                             v.i[20], v.i[21], (int)v.i[22], v.p[23], (size_t)v.i[24], v.p[25]))
CALL(sample, 13, "pppfpipfpfppiiiip",
     ((sample_fn)g_bound[13])(v.p[0], v.p[1], v.p[2], v.f[3], v.p[4], (int32_t)v.i[5], v.p[6], v.f[7], v.p[8], v.f[9],
                              v.p[10], (float*)v.p[11], v.i[12], v.i[13], v.i[14], (int)v.i[15], v.p[16]))

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, "rowops_" #name}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, "bind(softmax, layernorm_gelu, layernorm_gelu_erf)"},
    {"softmax", (PyCFunction)(void (*)(void))softmax, METH_FASTCALL, "rowops_softmax"},
    {"layernorm_gelu", (PyCFunction)(void (*)(void))layernorm_gelu, METH_FASTCALL, "rowops_layernorm_gelu"},
    {"layernorm_gelu_erf", (PyCFunction)(void (*)(void))layernorm_gelu_erf, METH_FASTCALL,
     "rowops_layernorm_gelu_erf"},
    {"bind_operators", (PyCFunction)(void (*)(void))bind_operators, METH_FASTCALL, "addresses of the functions below"},
    METHOD(groupnorm_act_workspace_bytes),
    METHOD(groupnorm_act),
    METHOD(groupnorm_act_backward_workspace_bytes),
    METHOD(groupnorm_act_backward),
    METHOD(bias_dropout_residual),
    METHOD(bias_dropout_residual_backward_workspace_bytes),
    METHOD(bias_dropout_residual_backward),
    METHOD(router_balance_loss),
    METHOD(router_balance_loss_backward),
    METHOD(router_balance_loss_workspace_bytes),
    METHOD(rmsnorm_quant),
    METHOD(paged_attention_workspace_bytes),
    METHOD(paged_attention),
    METHOD(sample),
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rowops_call", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__rowops_call(void) { return PyModule_Create(&module); }
