/* gemm_pycall.c -- CPython entry points for the per-call functions of the C ABI:
 * gemm_run, gemm_launch_empty and the calls of gemm_train.h and gemm_ffn.h: one vectorcall with plain integer
 * arguments instead of a ctypes call that converts each argument.  Argument
 * marshalling only: the functions are called through the addresses the Python
 * binding hands over once, after it has loaded libgemm_gb300.so.
 *
 *   set_targets(run_address, empty_address)
 *   run(plan, a, b, c, stream) -> gemm_status_t   (addresses as Python ints)
 *   launch_empty(grid, stream) -> gemm_status_t
 *   Runner(box, general) -> a callable for one plan: runner(A, B, C, stream)
 *       with three objects that have a data_ptr() method (torch tensors) and a
 *       stream object with a cuda_stream attribute calls gemm_run(box[0], ...)
 *       directly; every other call, a box[0] that is None (plan closed) and a
 *       non-zero status go to general(*args, **kwargs), the binding's own path,
 *       which handles the other argument forms and raises the error.
 *   TrainCall(kind, function, plan, elem, weight, types, cols, rows, device, raw_stream, only=-1,
 *             depth=0, square=0)
 *       -> a callable for one call of one plan of gemm_train.h or gemm_ffn.h (only: the index of
 *       the device that tensors have to be on, -1 = not looked at; types: the five dtypes of
 *       gemm_train.h and, for calls with 8-bit matrices, theirs; depth: a product's K; square: its
 *       second operand's scales go by squares; plan 0 for a call without one).  It takes the
 *       call's arguments by position (tensors, numbers, the stream last: an int,
 *       None for the current one, or an object with cuda_stream), checks them as
 *       the binding's general path does and returns the C function's status, or
 *       -1 without having called it where an argument is not what it expects
 *       (the general path then says what is wrong).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stddef.h>
#include <stdint.h>

typedef int (*gemm_run_fn)(void*, const void*, const void*, void*, void*);
typedef int (*gemm_launch_empty_fn)(int, void*);

static gemm_run_fn g_run = NULL;
static gemm_launch_empty_fn g_empty = NULL;

static PyObject* set_targets(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 2) {
        PyErr_SetString(PyExc_TypeError, "set_targets(run_address, empty_address)");
        return NULL;
    }
    void* run = PyLong_AsVoidPtr(args[0]);
    if (run == NULL && PyErr_Occurred()) return NULL;
    void* empty = PyLong_AsVoidPtr(args[1]);
    if (empty == NULL && PyErr_Occurred()) return NULL;
    g_run = (gemm_run_fn)run;
    g_empty = (gemm_launch_empty_fn)empty;
    Py_RETURN_NONE;
}

static PyObject* run(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 5) {
        PyErr_SetString(PyExc_TypeError, "run(plan, a, b, c, stream)");
        return NULL;
    }
    if (g_run == NULL) {
        PyErr_SetString(PyExc_RuntimeError, "gemm_run address not set");
        return NULL;
    }
    void* v[5];
    for (int i = 0; i < 5; ++i) {
        v[i] = PyLong_AsVoidPtr(args[i]);   /* 0 -> NULL without an error */
        if (v[i] == NULL && PyErr_Occurred()) return NULL;
    }
    return PyLong_FromLong(g_run(v[0], v[1], v[2], v[3], v[4]));
}

static PyObject* launch_empty(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 2) {
        PyErr_SetString(PyExc_TypeError, "launch_empty(grid, stream)");
        return NULL;
    }
    if (g_empty == NULL) {
        PyErr_SetString(PyExc_RuntimeError, "gemm_launch_empty address not set");
        return NULL;
    }
    const long grid = PyLong_AsLong(args[0]);
    if (grid == -1 && PyErr_Occurred()) return NULL;
    void* stream = PyLong_AsVoidPtr(args[1]);
    if (stream == NULL && PyErr_Occurred()) return NULL;
    return PyLong_FromLong(g_empty((int)grid, stream));
}

typedef struct {
    PyObject_HEAD
    PyObject* box;       /* list whose item 0 is the plan handle (an int) or None */
    PyObject* general;   /* fallback callable */
    vectorcallfunc vectorcall;
} Runner;

static PyObject* s_data_ptr = NULL;
static PyObject* s_cuda_stream = NULL;

/* The address an object reports, or NULL (error cleared) if it has none. */
static int address_of(PyObject* obj, PyObject* name, int is_method, void** out) {
    PyObject* r = is_method ? PyObject_VectorcallMethod(name, &obj, 1, NULL)
                            : PyObject_GetAttr(obj, name);
    if (r == NULL) {
        PyErr_Clear();
        return 0;
    }
    *out = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    if (*out == NULL && PyErr_Occurred()) {
        PyErr_Clear();
        return 0;
    }
    return 1;
}

static PyObject* runner_call(PyObject* self_, PyObject* const* args, size_t nargsf,
                             PyObject* kwnames) {
    Runner* self = (Runner*)self_;
    const Py_ssize_t nargs = PyVectorcall_NARGS(nargsf);
    if (nargs == 4 && kwnames == NULL && g_run != NULL) {
        PyObject* h = PyList_GET_ITEM(self->box, 0);
        void* plan = h == Py_None ? NULL : PyLong_AsVoidPtr(h);
        if (plan == NULL) PyErr_Clear();
        void* v[4];
        if (plan != NULL && address_of(args[0], s_data_ptr, 1, &v[0]) &&
            address_of(args[1], s_data_ptr, 1, &v[1]) &&
            address_of(args[2], s_data_ptr, 1, &v[2]) &&
            address_of(args[3], s_cuda_stream, 0, &v[3]) &&
            g_run(plan, v[0], v[1], v[2], v[3]) == 0)
            Py_RETURN_NONE;
    }
    return PyObject_Vectorcall(self->general, args, nargsf, kwnames);
}

static PyObject* runner_new(PyTypeObject* type, PyObject* args, PyObject* kwds) {
    PyObject *box, *general;
    if (kwds != NULL && PyDict_GET_SIZE(kwds) != 0) {
        PyErr_SetString(PyExc_TypeError, "Runner(box, general)");
        return NULL;
    }
    if (!PyArg_ParseTuple(args, "O!O:Runner", &PyList_Type, &box, &general)) return NULL;
    if (PyList_GET_SIZE(box) < 1 || !PyCallable_Check(general)) {
        PyErr_SetString(PyExc_TypeError, "Runner(box, general): a non-empty list and a callable");
        return NULL;
    }
    Runner* self = (Runner*)type->tp_alloc(type, 0);
    if (self == NULL) return NULL;
    Py_INCREF(box);
    Py_INCREF(general);
    self->box = box;
    self->general = general;
    self->vectorcall = runner_call;
    return (PyObject*)self;
}

static int runner_traverse(PyObject* self_, visitproc visit, void* arg) {
    Runner* self = (Runner*)self_;
    Py_VISIT(self->box);
    Py_VISIT(self->general);
    return 0;
}

static int runner_clear(PyObject* self_) {
    Runner* self = (Runner*)self_;
    Py_CLEAR(self->box);
    Py_CLEAR(self->general);
    return 0;
}

static void runner_dealloc(PyObject* self) {
    PyObject_GC_UnTrack(self);
    runner_clear(self);
    Py_TYPE(self)->tp_free(self);
}

static PyTypeObject RunnerType = {
    PyVarObject_HEAD_INIT(NULL, 0)
    .tp_name = "_gemm_pycall.Runner",
    .tp_basicsize = sizeof(Runner),
    .tp_flags = Py_TPFLAGS_DEFAULT | Py_TPFLAGS_HAVE_GC | Py_TPFLAGS_HAVE_VECTORCALL,
    .tp_doc = "Runner(box, general): gemm_run for one plan, called as runner(A, B, C, stream)",
    .tp_new = runner_new,
    .tp_dealloc = runner_dealloc,
    .tp_traverse = runner_traverse,
    .tp_clear = runner_clear,
    .tp_call = PyVectorcall_Call,
    .tp_vectorcall_offset = offsetof(Runner, vectorcall),
};

/* ---- the calls of gemm_train.h -------------------------------------------------- */

typedef struct {      /* gemm_teacher_t */
    const void* ids;
    const void* values;
    const float* lse;
    int64_t top, ld_ids, ld_values;
    int32_t id_type, value_elem;
} Teacher;

enum { NORM_FORWARD, NORM_BACKWARD, EMBED_FORWARD, EMBED_BACKWARD, DISTILL_FORWARD,
       DISTILL_BACKWARD, DISTILL_BOTH, RMS_FORWARD, RMS_FORWARD_FP8, RMS_BACKWARD, FP8_RUN,
       GATED_FORWARD, GATED_BACKWARD, QUANTIZE, TRAIN_KINDS };

typedef struct {
    PyObject_HEAD
    int kind;
    void* fn;
    void* plan;
    PyObject* elem;          /* torch dtypes: the plan's elements, */
    PyObject* weight;        /* its weights or table gradients, */
    PyObject* types;         /* and (float16, bfloat16, float32, int32, int64[, float8_e4m3fn]) */
    int64_t cols, rows;      /* of the matrices (rows: of an embedding table, or a product's result) */
    int64_t depth;           /* a product's K */
    int square;              /* its second operand's scales */
    PyObject* device;
    PyObject* raw_stream;    /* callable: device -> the current stream's handle */
    long only;               /* the device that tensors have to be on; -1: there is one, not asked */
    vectorcallfunc vectorcall;
} TrainCall;

static PyObject *s_dtype, *s_is_cuda, *s_get_device, *s_shape, *s_stride, *s_is_contiguous;

/* Whether the tensor is on the plan's device (asked where there are several). */
static int on_device(const TrainCall* call, PyObject* t) {
    if (call->only < 0) return 1;
    PyObject* r = PyObject_CallMethodNoArgs(t, s_get_device);
    const long device = r == NULL ? -1 : PyLong_AsLong(r);
    Py_XDECREF(r);
    return device == call->only;
}

/* Address of a CUDA tensor of `dims` dimensions with its shape and strides; 0 where
 * it is something else. */
static int tensor_of(const TrainCall* call, PyObject* t, int dims, void** ptr, int64_t* shape, int64_t* stride) {
    PyObject* r = PyObject_GetAttr(t, s_is_cuda);
    const int cuda = r == Py_True;
    Py_XDECREF(r);
    if (!cuda || !address_of(t, s_data_ptr, 1, ptr) || !on_device(call, t)) return 0;
    PyObject* a = PyObject_GetAttr(t, s_shape);
    int ok = a != NULL && PyTuple_Check(a) && PyTuple_GET_SIZE(a) == dims;
    for (int i = 0; ok && i < dims; ++i) shape[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(a, i));
    Py_XDECREF(a);
    if (!ok) return 0;
    /* (the usual answer, for less than the strides) */
    PyObject* c = PyObject_VectorcallMethod(s_is_contiguous, &t, 1, NULL);
    Py_XDECREF(c);
    if (c == Py_True) {
        stride[dims - 1] = 1;
        if (dims == 2) stride[0] = shape[1];
        return !PyErr_Occurred();
    }
    PyObject* b = c == NULL ? NULL : PyObject_VectorcallMethod(s_stride, &t, 1, NULL);
    ok = b != NULL && PyTuple_Check(b) && PyTuple_GET_SIZE(b) == dims;
    for (int i = 0; ok && i < dims; ++i) stride[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(b, i));
    Py_XDECREF(b);
    return ok && !PyErr_Occurred();
}

static int has_type(PyObject* t, PyObject* dtype) {
    PyObject* r = PyObject_GetAttr(t, s_dtype);
    Py_XDECREF(r);           /* (dtypes live as long as torch) */
    return r == dtype;
}

/* Which of types[from..to) the tensor has, counted from `from`; -1 for none. */
static int type_among(PyObject* t, PyObject* types, int from, int to) {
    PyObject* r = PyObject_GetAttr(t, s_dtype);
    Py_XDECREF(r);
    for (int i = from; i < to; ++i)
        if (PyTuple_GET_ITEM(types, i) == r) return i - from;
    return -1;
}

/* A rows x cols matrix with contiguous rows (*rows < 0: any number, which is set). */
static int matrix(const TrainCall* call, PyObject* t, int64_t* rows, int64_t cols, void** ptr, int64_t* ld) {
    int64_t shape[2], stride[2];
    if (!tensor_of(call, t, 2, ptr, shape, stride)) return 0;
    if (*rows < 0) *rows = shape[0];
    if (shape[0] != *rows || shape[1] != cols || (cols > 1 && stride[1] != 1)) return 0;
    *ld = *rows > 1 ? stride[0] : cols;
    return 1;
}

/* A rows x cols matrix of the type with contiguous rows; None, a NULL pointer, where that is allowed. */
static int typed(const TrainCall* call, PyObject* t, PyObject* dtype, int64_t* rows, int64_t cols, int none, void** ptr,
                 int64_t* ld) {
    if (t == Py_None) {
        *ptr = NULL;
        *ld = 0;
        return none;
    }
    return has_type(t, dtype) && matrix(call, t, rows, cols, ptr, ld);
}

/* ... all of it contiguous. */
static int whole(const TrainCall* call, PyObject* t, PyObject* dtype, int64_t rows, int64_t cols, int none, void** ptr) {
    int64_t ld;
    return typed(call, t, dtype, &rows, cols, none, ptr, &ld) && (*ptr == NULL || ld == cols || rows * cols == 0);
}

static int64_t groups_of(int64_t n) { return (n + 127) / 128; }

/* A contiguous vector of n values of the type, or None where that is allowed. */
static int vector(const TrainCall* call, PyObject* t, PyObject* dtype, int64_t n, int none, void** ptr) {
    int64_t shape, stride;
    if (t == Py_None) {
        *ptr = NULL;
        return none;
    }
    return (dtype == NULL || has_type(t, dtype)) && tensor_of(call, t, 1, ptr, &shape, &stride) &&
           shape == n && (n < 2 || stride == 1);
}

static int number(PyObject* o, double* v) {
    *v = PyFloat_AsDouble(o);
    return !PyErr_Occurred();
}

static int stream_of(const TrainCall* c, PyObject* o, void** stream) {
    if (o == Py_None) {
        PyObject* r = PyObject_CallOneArg(c->raw_stream, c->device);
        if (r == NULL) return 0;
        *stream = PyLong_AsVoidPtr(r);
        Py_DECREF(r);
        return !PyErr_Occurred();
    }
    if (PyLong_Check(o)) {
        *stream = PyLong_AsVoidPtr(o);
        return !PyErr_Occurred();
    }
    return address_of(o, s_cuda_stream, 0, stream);
}

static int teacher_of(const TrainCall* c, PyObject* ids, PyObject* values, PyObject* lse, int64_t rows,
                      Teacher* t) {
    int64_t shape[2], stride[2], n = rows;
    void *pi, *pv, *pl;
    const int id_type = type_among(ids, c->types, 3, 5), elem = type_among(values, c->types, 0, 3);
    if (id_type < 0 || elem < 0 || !tensor_of(c, ids, 2, &pi, shape, stride)) return 0;
    const int64_t top = shape[1];
    if (shape[0] != rows || (top > 1 && stride[1] != 1)) return 0;
    t->ld_ids = rows > 1 ? stride[0] : top;
    if (!matrix(c, values, &n, top, &pv, &t->ld_values) ||
        !vector(c, lse, PyTuple_GET_ITEM(c->types, 2), rows, 1, &pl))
        return 0;
    t->ids = pi;
    t->values = pv;
    t->lse = (const float*)pl;
    t->top = top;
    t->id_type = id_type;
    t->value_elem = elem;
    return 1;
}

/* The calls of gemm_ffn.h. */
static int ffn_call(const TrainCall* c, PyObject* const* v, Py_ssize_t n) {
    PyObject* const f32 = PyTuple_GET_ITEM(c->types, 2);
    PyObject* const e4m3 = PyTuple_GET_ITEM(c->types, 5);
    void *p[7], *stream;
    int64_t ld[5], rows = -1;
    double x;
    switch (c->kind) {
        case RMS_FORWARD:            /* x, gamma, y, rstd, residual, total, eps, stream */
        case RMS_FORWARD_FP8: {      /* x, gamma, q, scales, rstd, residual, total, eps, stream */
            const int fp8 = c->kind == RMS_FORWARD_FP8;
            PyObject* const* m = v + fp8;
            if (n != 8 + fp8 || !typed(c, v[0], c->elem, &rows, c->cols, 0, &p[0], &ld[0]) ||
                !vector(c, v[1], c->weight, c->cols, 1, &p[1]) ||
                !typed(c, v[2], fp8 ? e4m3 : c->elem, &rows, c->cols, 0, &p[2], &ld[2]) ||
                (fp8 && !typed(c, v[3], f32, &rows, groups_of(c->cols), 0, &p[6], &ld[1])) ||
                !vector(c, m[3], f32, rows, 1, &p[3]) || !typed(c, m[4], c->elem, &rows, c->cols, 1, &p[4], &ld[3]) ||
                !typed(c, m[5], c->elem, &rows, c->cols, 1, &p[5], &ld[4]) || !number(m[6], &x) ||
                !stream_of(c, m[7], &stream))
                return -1;
            if (fp8)
                return ((int (*)(void*, int64_t, const void*, int64_t, const void*, int64_t, const void*, float, void*,
                                 int64_t, void*, int64_t, void*, int64_t, void*, void*))c->fn)(
                    c->plan, rows, p[0], ld[0], p[4], ld[3], p[1], (float)x, p[5], ld[4], p[2], ld[2], p[6], ld[1], p[3],
                    stream);
            return ((int (*)(void*, int64_t, const void*, int64_t, const void*, int64_t, const void*, float, void*,
                             int64_t, void*, int64_t, void*, void*))c->fn)(
                c->plan, rows, p[0], ld[0], p[4], ld[3], p[1], (float)x, p[5], ld[4], p[2], ld[2], p[3], stream);
        }
        case RMS_BACKWARD:           /* total, gamma, rstd, dy, dx, dgamma, dtotal, stream */
            if (n != 8 || !typed(c, v[0], c->elem, &rows, c->cols, 0, &p[0], &ld[0]) ||
                !vector(c, v[1], c->weight, c->cols, 1, &p[1]) || !vector(c, v[2], f32, rows, 0, &p[2]) ||
                !typed(c, v[3], c->elem, &rows, c->cols, 0, &p[3], &ld[1]) ||
                !typed(c, v[4], c->elem, &rows, c->cols, 1, &p[4], &ld[2]) ||
                !vector(c, v[5], c->weight, c->cols, 1, &p[5]) ||
                !typed(c, v[6], c->elem, &rows, c->cols, 1, &p[6], &ld[3]) || !stream_of(c, v[7], &stream))
                return -1;
            return ((int (*)(void*, int64_t, const void*, int64_t, const void*, const void*, const void*, int64_t,
                             const void*, int64_t, void*, int64_t, void*, void*))c->fn)(
                c->plan, rows, p[0], ld[0], p[1], p[2], p[3], ld[1], p[6], ld[3], p[4], ld[2], p[5], stream);
        case FP8_RUN: {              /* A, a_scales, B, b_scales, C, stream */
            const int64_t M = c->rows, N = c->cols, K = c->depth;
            if (n != 6 || !whole(c, v[0], e4m3, M, K, 0, &p[0]) || !whole(c, v[1], f32, M, groups_of(K), 0, &p[1]) ||
                !whole(c, v[2], e4m3, N, K, 0, &p[2]) ||
                !whole(c, v[3], f32, c->square ? groups_of(N) : N, groups_of(K), 0, &p[3]) ||
                !whole(c, v[4], c->elem, M, N, 0, &p[4]) || !stream_of(c, v[5], &stream))
                return -1;
            return ((int (*)(void*, const void*, const void*, const void*, const void*, void*, void*))c->fn)(
                c->plan, p[0], p[1], p[2], p[3], p[4], stream);
        }
        case GATED_FORWARD: {        /* X, W, H, gate_up, stream */
            const int64_t M = c->rows, F = c->cols, K = c->depth;
            if (n != 5 || !whole(c, v[0], c->elem, M, K, 0, &p[0]) || !whole(c, v[1], c->elem, 2 * F, K, 0, &p[1]) ||
                !whole(c, v[2], c->elem, M, F, 0, &p[2]) || !whole(c, v[3], c->elem, M, 2 * F, 1, &p[3]) ||
                !stream_of(c, v[4], &stream))
                return -1;
            return ((int (*)(void*, const void*, const void*, void*, void*, void*))c->fn)(c->plan, p[0], p[1], p[2], p[3],
                                                                                         stream);
        }
        case GATED_BACKWARD: {       /* X, W, gate_up, dH, dgate_up, dX, dW, stream */
            const int64_t M = c->rows, F = c->cols, K = c->depth;
            if (n != 8 || !whole(c, v[0], c->elem, M, K, v[6] == Py_None, &p[0]) ||
                !whole(c, v[1], c->elem, 2 * F, K, v[5] == Py_None, &p[1]) ||
                !whole(c, v[2], c->elem, M, 2 * F, 0, &p[2]) || !whole(c, v[3], c->elem, M, F, 0, &p[3]) ||
                !whole(c, v[4], c->elem, M, 2 * F, 0, &p[4]) || !whole(c, v[5], c->elem, M, K, 1, &p[5]) ||
                !whole(c, v[6], c->elem, 2 * F, K, 1, &p[6]) || !stream_of(c, v[7], &stream))
                return -1;
            return ((int (*)(void*, const void*, const void*, const void*, const void*, void*, void*, void*, void*))c->fn)(
                c->plan, p[0], p[1], p[2], p[3], p[4], p[5], p[6], stream);
        }
        default: {                   /* QUANTIZE: x, q, scales, kind of scales, transpose, stream */
            int64_t shape[2], stride[2];
            const int elem = n == 6 ? type_among(v[0], c->types, 0, 3) : -1;
            if (elem < 0 || !tensor_of(c, v[0], 2, &p[0], shape, stride) || (shape[1] > 1 && stride[1] != 1)) return -1;
            const int kind = (int)PyLong_AsLong(v[3]), turned = PyObject_IsTrue(v[4]);
            if (turned < 0 || PyErr_Occurred()) return -1;
            int64_t out = shape[turned ? 1 : 0], down = kind == 1 ? groups_of(out) : out;
            const int64_t across = shape[turned ? 0 : 1];
            if (!typed(c, v[1], e4m3, &out, across, 0, &p[1], &ld[1]) ||
                !typed(c, v[2], f32, &down, groups_of(across), 0, &p[2], &ld[2]) || !stream_of(c, v[5], &stream))
                return -1;
            ld[0] = shape[0] > 1 ? stride[0] : shape[1];
            return ((int (*)(int64_t, int64_t, int, const void*, int64_t, int, int, void*, int64_t, void*, int64_t,
                             void*))c->fn)(shape[0], shape[1], elem, p[0], ld[0], kind, turned, p[1], ld[1], p[2], ld[2],
                                           stream);
        }
    }
}

/* The status of the call, or -1 where an argument does not fit. */
static int train_call(const TrainCall* c, PyObject* const* v, Py_ssize_t n) {
    PyObject* const f32 = PyTuple_GET_ITEM(c->types, 2);
    void *p[8], *stream;
    int64_t ld[3], rows = -1;
    double x;
    switch (c->kind) {
        case NORM_FORWARD:
            if (n != 8 || !has_type(v[0], c->elem) || !matrix(c, v[0], &rows, c->cols, &p[0], &ld[0]) ||
                !vector(c, v[1], c->weight, c->cols, 1, &p[1]) || !vector(c, v[2], c->weight, c->cols, 1, &p[2]) ||
                !has_type(v[3], c->elem) || !matrix(c, v[3], &rows, c->cols, &p[3], &ld[1]) ||
                !vector(c, v[4], f32, rows, 1, &p[4]) || !vector(c, v[5], f32, rows, 1, &p[5]) ||
                !number(v[6], &x) || !stream_of(c, v[7], &stream))
                return -1;
            return ((int (*)(void*, int64_t, const void*, int64_t, const void*, const void*, float, void*,
                             int64_t, void*, void*, void*))c->fn)(
                c->plan, rows, p[0], ld[0], p[1], p[2], (float)x, p[3], ld[1], p[4], p[5], stream);
        case NORM_BACKWARD:
            p[5] = NULL;
            ld[2] = 0;
            if (n != 9 || !has_type(v[0], c->elem) || !matrix(c, v[0], &rows, c->cols, &p[0], &ld[0]) ||
                !vector(c, v[1], c->weight, c->cols, 1, &p[1]) || !vector(c, v[2], f32, rows, 0, &p[2]) ||
                !vector(c, v[3], f32, rows, 0, &p[3]) || !has_type(v[4], c->elem) ||
                !matrix(c, v[4], &rows, c->cols, &p[4], &ld[1]) ||
                (v[5] != Py_None && (!has_type(v[5], c->elem) || !matrix(c, v[5], &rows, c->cols, &p[5], &ld[2]))) ||
                !vector(c, v[6], c->weight, c->cols, 1, &p[6]) || !vector(c, v[7], c->weight, c->cols, 1, &p[7]) ||
                !stream_of(c, v[8], &stream))
                return -1;
            return ((int (*)(void*, int64_t, const void*, int64_t, const void*, const void*, const void*,
                             const void*, int64_t, void*, int64_t, void*, void*, void*))c->fn)(
                c->plan, rows, p[0], ld[0], p[1], p[2], p[3], p[4], ld[1], p[5], ld[2], p[6], p[7], stream);
        case EMBED_FORWARD:
        case EMBED_BACKWARD: {
            const int back = c->kind == EMBED_BACKWARD;
            int64_t shape, stride, vocab = c->rows;
            const int id_type = n == 6 + back ? type_among(v[0], c->types, 3, 5) : -1;
            if (id_type < 0 || !tensor_of(c, v[0], 1, &p[0], &shape, &stride) || (shape > 1 && stride != 1)) return -1;
            rows = shape;
            PyObject* const by_token = v[back ? 1 : 2];
            PyObject* const table = v[back ? 2 : 1];
            if (!has_type(by_token, c->elem) || !matrix(c, by_token, &rows, c->cols, &p[1], &ld[0]) ||
                !has_type(table, back ? c->weight : c->elem) || !matrix(c, table, &vocab, c->cols, &p[2], &ld[1]) ||
                !number(v[3], &x))
                return -1;
            const int64_t padding = PyLong_AsLongLong(v[4]);
            if (PyErr_Occurred() || !stream_of(c, v[5 + back], &stream)) return -1;
            if (!back)
                return ((int (*)(void*, int64_t, const void*, int, int64_t, const void*, int64_t, float, void*,
                                 int64_t, void*))c->fn)(c->plan, rows, p[0], id_type, padding, p[2], ld[1],
                                                        (float)x, p[1], ld[0], stream);
            const int accumulate = PyObject_IsTrue(v[5]);
            if (accumulate < 0) return -1;
            return ((int (*)(void*, int64_t, const void*, int, int64_t, const void*, int64_t, float, void*,
                             int64_t, int, void*))c->fn)(c->plan, rows, p[0], id_type, padding, p[1], ld[0],
                                                         (float)x, p[2], ld[1], accumulate, stream);
        }
        default: {
            /* logits, ids, values, [loss], lse, [dlogits, dloss], temperature, teacher_lse, stream */
            const int forward = c->kind != DISTILL_BACKWARD, backward = c->kind != DISTILL_FORWARD;
            Teacher t;
            int k = 3;
            if (n != 7 + forward + 2 * backward || !has_type(v[0], c->elem) ||
                !matrix(c, v[0], &rows, c->cols, &p[0], &ld[0]))
                return -1;
            p[1] = p[3] = p[4] = NULL;
            if (forward && !vector(c, v[k++], f32, rows, 0, &p[1])) return -1;
            if (!vector(c, v[k++], f32, rows, 0, &p[2])) return -1;
            if (backward) {
                if (!has_type(v[k], c->elem) || !matrix(c, v[k], &rows, c->cols, &p[3], &ld[1])) return -1;
                if (!vector(c, v[k + 1], f32, rows, 1, &p[4])) return -1;
                k += 2;
            }
            if (!number(v[k], &x) || !teacher_of(c, v[1], v[2], v[k + 1], rows, &t) || !stream_of(c, v[k + 2], &stream))
                return -1;
            if (c->kind == DISTILL_FORWARD)
                return ((int (*)(void*, int64_t, const void*, int64_t, const Teacher*, float, void*, void*,
                                 void*))c->fn)(c->plan, rows, p[0], ld[0], &t, (float)x, p[1], p[2], stream);
            if (c->kind == DISTILL_BACKWARD)
                return ((int (*)(void*, int64_t, const void*, int64_t, const Teacher*, float, const void*,
                                 const void*, void*, int64_t, void*))c->fn)(
                    c->plan, rows, p[0], ld[0], &t, (float)x, p[2], p[4], p[3], ld[1], stream);
            return ((int (*)(void*, int64_t, const void*, int64_t, const Teacher*, float, const void*, void*,
                             void*, void*, int64_t, void*))c->fn)(
                c->plan, rows, p[0], ld[0], &t, (float)x, p[4], p[1], p[2], p[3], ld[1], stream);
        }
    }
}

static PyObject* train_call_vector(PyObject* self, PyObject* const* args, size_t nargsf, PyObject* kwnames) {
    if (kwnames != NULL) {
        PyErr_SetString(PyExc_TypeError, "TrainCall takes its arguments by position");
        return NULL;
    }
    const TrainCall* const call = (const TrainCall*)self;
    const int st = (call->kind < RMS_FORWARD ? train_call : ffn_call)(call, args, PyVectorcall_NARGS(nargsf));
    if (st < 0) PyErr_Clear();
    return PyLong_FromLong(st);
}

static PyObject* train_call_new(PyTypeObject* type, PyObject* args, PyObject* kwds) {
    int kind;
    long long cols, rows, depth = 0;
    long only = -1;
    int square = 0;
    PyObject *fn, *plan, *elem, *weight, *types, *device, *raw_stream;
    if (kwds != NULL && PyDict_GET_SIZE(kwds) != 0) {
        PyErr_SetString(PyExc_TypeError, "TrainCall takes its arguments by position");
        return NULL;
    }
    if (!PyArg_ParseTuple(args, "iOOOOO!LLOO|lLp:TrainCall", &kind, &fn, &plan, &elem, &weight, &PyTuple_Type,
                          &types, &cols, &rows, &device, &raw_stream, &only, &depth, &square))
        return NULL;
    void* f = PyLong_AsVoidPtr(fn);
    void* h = PyErr_Occurred() ? NULL : PyLong_AsVoidPtr(plan);
    if (PyErr_Occurred()) return NULL;
    const Py_ssize_t dtypes = PyTuple_GET_SIZE(types);
    if (kind < 0 || kind >= TRAIN_KINDS || f == NULL || (h == NULL && kind != QUANTIZE) ||
        dtypes != (kind < RMS_FORWARD ? 5 : 6) || !PyCallable_Check(raw_stream)) {
        PyErr_SetString(PyExc_ValueError, "TrainCall: unknown kind, null address, five dtypes (six for gemm_ffn.h) and a callable needed");
        return NULL;
    }
    TrainCall* self = (TrainCall*)type->tp_alloc(type, 0);
    if (self == NULL) return NULL;
    self->kind = kind;
    self->fn = f;
    self->plan = h;
    self->elem = Py_NewRef(elem);
    self->weight = Py_NewRef(weight);
    self->types = Py_NewRef(types);
    self->cols = cols;
    self->rows = rows;
    self->depth = depth;
    self->square = square;
    self->device = Py_NewRef(device);
    self->raw_stream = Py_NewRef(raw_stream);
    self->only = only;
    self->vectorcall = train_call_vector;
    return (PyObject*)self;
}

static int train_call_traverse(PyObject* self_, visitproc visit, void* arg) {
    TrainCall* self = (TrainCall*)self_;
    Py_VISIT(self->elem);
    Py_VISIT(self->weight);
    Py_VISIT(self->types);
    Py_VISIT(self->device);
    Py_VISIT(self->raw_stream);
    return 0;
}

static int train_call_clear(PyObject* self_) {
    TrainCall* self = (TrainCall*)self_;
    Py_CLEAR(self->elem);
    Py_CLEAR(self->weight);
    Py_CLEAR(self->types);
    Py_CLEAR(self->device);
    Py_CLEAR(self->raw_stream);
    return 0;
}

static void train_call_dealloc(PyObject* self) {
    PyObject_GC_UnTrack(self);
    train_call_clear(self);
    Py_TYPE(self)->tp_free(self);
}

static PyTypeObject TrainCallType = {
    PyVarObject_HEAD_INIT(NULL, 0)
    .tp_name = "_gemm_pycall.TrainCall",
    .tp_basicsize = sizeof(TrainCall),
    .tp_flags = Py_TPFLAGS_DEFAULT | Py_TPFLAGS_HAVE_GC | Py_TPFLAGS_HAVE_VECTORCALL,
    .tp_doc = "One call of one plan of gemm_train.h or gemm_ffn.h: its status, or -1 where an argument does not fit",
    .tp_new = train_call_new,
    .tp_dealloc = train_call_dealloc,
    .tp_traverse = train_call_traverse,
    .tp_clear = train_call_clear,
    .tp_call = PyVectorcall_Call,
    .tp_vectorcall_offset = offsetof(TrainCall, vectorcall),
};

static PyMethodDef methods[] = {
    {"set_targets", (PyCFunction)(void (*)(void))set_targets, METH_FASTCALL,
     "set_targets(run_address, empty_address)"},
    {"run", (PyCFunction)(void (*)(void))run, METH_FASTCALL,
     "run(plan, a, b, c, stream) -> status of gemm_run"},
    {"launch_empty", (PyCFunction)(void (*)(void))launch_empty, METH_FASTCALL,
     "launch_empty(grid, stream) -> status of gemm_launch_empty"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gemm_pycall",
                                    "Vectorcall entry points for gemm_run and gemm_launch_empty, "
                                    "a per-plan runner, and the calls of gemm_train.h and gemm_ffn.h.",
                                    -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__gemm_pycall(void) {
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_is_cuda = PyUnicode_InternFromString("is_cuda");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    if (s_data_ptr == NULL || s_cuda_stream == NULL || s_dtype == NULL || s_is_cuda == NULL ||
        s_get_device == NULL || s_shape == NULL ||        s_stride == NULL || s_is_contiguous == NULL || PyType_Ready(&RunnerType) < 0 || PyType_Ready(&TrainCallType) < 0)
        return NULL;
    PyObject* m = PyModule_Create(&module);
    if (m == NULL) return NULL;
    if (PyModule_AddObjectRef(m, "Runner", (PyObject*)&RunnerType) < 0 ||
        PyModule_AddObjectRef(m, "TrainCall", (PyObject*)&TrainCallType) < 0) {
        Py_DECREF(m);
        return NULL;
    }
    return m;
}
