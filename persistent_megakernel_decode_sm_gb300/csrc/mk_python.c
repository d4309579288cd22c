/* The Python module _mk_call: linear() and attend() of the package for the calls that need no more than their
 * operands' addresses, shapes and strides.  Kernels of a few microseconds leave the interpreter as the larger part of
 * a call (one token's attention over 8192 positions, back to back in four processes: 16.4 to 21 us with the checks in
 * Python, 12.0 to 14.4 here, of which 5 in mk_attend; one token's linear map 8.7 to 13.6 and 6.5 to 10).  Each function
 * makes the checks of its Python namesake and then the call; where one fails, or the call is of another kind (another
 * current device, lengths that are not lists of ints), it returns None with nothing done, and the Python function,
 * which checks the same and says what is wrong, takes over. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "mk.h"

static mk_status (*linear_fn)(const mk_linear_args*, void*);
static mk_status (*attend_fn)(const mk_attend_args*, void*, size_t, void*);
static size_t (*attend_workspace_fn)(const mk_attend_args*);
/* torch's objects, held for the life of the process */
static PyObject *bf16, *f32, *i32, *empty, *raw_stream, *current_device, *raw_alloc, *raw_delete;
static PyObject *s_dtype, *s_shape, *s_stride, *s_device, *s_get_device, *s_data_ptr, *s_is_contiguous, *s_numel, *s_element_size;
static PyObject* empty_names;   /* ("dtype", "device") */

typedef struct {
    int64_t shape[5], stride[5];
    uintptr_t ptr;
    int is_f32;
} View;

static int integer(PyObject* o, int64_t* out) {   /* takes the reference */
    if (!o) return 0;
    const int ok = PyLong_Check(o);
    if (ok) *out = PyLong_AsLongLong(o);
    Py_DECREF(o);
    return ok && !(*out == -1 && PyErr_Occurred());
}
static int method(PyObject* t, PyObject* name, int64_t* out) { return integer(PyObject_CallMethodNoArgs(t, name), out); }
static int sizes(PyObject* o, int dim, int64_t* out) {   /* takes the reference */
    int ok = o && PyTuple_Check(o) && PyTuple_GET_SIZE(o) == dim;
    for (int i = 0; ok && i < dim; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
        ok = !(out[i] == -1 && PyErr_Occurred());
    }
    Py_XDECREF(o);
    return ok;
}
/* An operand of type `type` (or fp32, where allowed) on the device, `dim` dimensions, the last one contiguous */
static int view(PyObject* t, PyObject* type, int or_f32, int64_t device, int dim, View* v) {
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    if (!d) return 0;
    v->is_f32 = d == f32;
    const int typed = d == type || (or_f32 && v->is_f32);
    Py_DECREF(d);
    int64_t at, ptr;
    if (!typed || !method(t, s_get_device, &at) || at != device || !sizes(PyObject_GetAttr(t, s_shape), dim, v->shape) ||
        !sizes(PyObject_CallMethodNoArgs(t, s_stride), dim, v->stride) || !method(t, s_data_ptr, &ptr))
        return 0;
    v->ptr = (uintptr_t)ptr;
    return v->stride[dim - 1] == 1 || v->shape[dim - 1] <= 1;
}
static int fits(int64_t x) { return x >= INT32_MIN && x <= INT32_MAX; }
static int small(PyObject* o, int32_t* out) {   /* a Python int of 32 bits */
    if (!PyLong_Check(o)) return 0;
    const long long x = PyLong_AsLongLong(o);
    if ((x == -1 && PyErr_Occurred()) || !fits(x)) return 0;
    *out = (int32_t)x;
    return 1;
}
static PyObject* new_tensor(PyObject* like, const int64_t* shape, int dim, PyObject* type) {
    PyObject* device = PyObject_GetAttr(like, s_device);
    PyObject* size = device ? PyTuple_New(dim) : NULL;
    PyObject* r = NULL;
    if (size) {
        int ok = 1;
        for (int i = 0; i < dim; ++i) {
            PyObject* n = PyLong_FromLongLong(shape[i]);
            if (n) PyTuple_SET_ITEM(size, i, n);
            else ok = 0;
        }
        PyObject* args[3] = {size, type, device};
        if (ok) r = PyObject_Vectorcall(empty, args, 1, empty_names);
    }
    Py_XDECREF(size);
    Py_XDECREF(device);
    return r;
}
static int stream_of(int64_t device, void** out) {
    int64_t s;
    PyObject* d = PyLong_FromLongLong(device);
    if (!d) return 0;
    const int ok = integer(PyObject_CallOneArg(raw_stream, d), &s);
    Py_DECREF(d);
    if (ok) *out = (void*)(uintptr_t)s;
    return ok;
}
/* The operand's device, where it is the current one */
static int device_of(PyObject* t, int64_t* device) {
    int64_t now;
    return method(t, s_get_device, device) && *device >= 0 && integer(PyObject_CallNoArgs(current_device), &now) && now == *device;
}
static int status_of(PyObject* t, int64_t device, int32_t** out) {
    View v;
    *out = NULL;
    if (t == Py_None) return 1;
    if (!view(t, i32, 0, device, 1, &v) || v.shape[0] < 1) return 0;
    *out = (int32_t*)v.ptr;
    return 1;
}
static PyObject* leave(PyObject* out) {   /* None: the Python function takes over */
    Py_XDECREF(out);
    PyErr_Clear();
    Py_RETURN_NONE;
}

/* linear(x, weight, bias, activation, residual, out, out_dtype, status) */
static PyObject* call_linear(PyObject* self, PyObject* const* arg, Py_ssize_t n_arg) {
    (void)self;
    if (n_arg != 8) return leave(NULL);
    PyObject *x = arg[0], *w = arg[1], *bias = arg[2], *act = arg[3], *res = arg[4], *out = arg[5], *type = arg[6];
    mk_linear_args a = {0};
    int64_t device;
    View vx, vw, v;
    if (!device_of(x, &device) || !view(x, bf16, 0, device, 2, &vx) || !view(w, bf16, 0, device, 2, &vw)) return leave(NULL);
    int64_t rows = vx.shape[0], k = vx.shape[1], n = vw.shape[0];
    if (vw.shape[1] != k || (vw.stride[0] != k && n > 1)) return leave(NULL);
    a.activation = -1;
    if (act == Py_None) a.activation = MK_ACT_NONE;
    else if (PyUnicode_Check(act)) {
        if (PyUnicode_CompareWithASCIIString(act, "silu") == 0) a.activation = MK_ACT_SILU;
        else if (PyUnicode_CompareWithASCIIString(act, "gelu") == 0) a.activation = MK_ACT_GELU;
        else if (PyUnicode_CompareWithASCIIString(act, "swiglu") == 0) a.activation = MK_ACT_SWIGLU;
    }
    if (a.activation < 0) return leave(NULL);
    if (bias != Py_None) {
        if (!view(bias, bf16, 0, device, 1, &v) || v.shape[0] != n) return leave(NULL);
        a.bias = (const void*)v.ptr;
    }
    if (a.activation == MK_ACT_SWIGLU) {
        if (n % 2) return leave(NULL);
        n /= 2;
    }
    if (!fits(rows) || !fits(n) || !fits(k)) return leave(NULL);
    if (res != Py_None) {
        if (!view(res, bf16, 1, device, 2, &v) || v.shape[0] != rows || v.shape[1] != n) return leave(NULL);
        a.residual = (const void*)v.ptr;
        a.residual_stride = v.stride[0];
        a.residual_dtype = v.is_f32 ? MK_F32 : MK_BF16;
    }
    void* stream;
    if (!status_of(arg[7], device, &a.status) || !stream_of(device, &stream)) return leave(NULL);
    if (out == Py_None) {
        if (type != Py_None && type != bf16 && type != f32) return leave(NULL);
        const int64_t shape[2] = {rows, n};
        int64_t ptr;
        out = new_tensor(x, shape, 2, type == f32 ? f32 : bf16);
        if (!out || !method(out, s_data_ptr, &ptr)) return leave(out);
        a.out = (void*)(uintptr_t)ptr;
        a.out_stride = n;
        a.out_dtype = type == f32 ? MK_F32 : MK_BF16;
    } else {
        if (!view(out, bf16, 1, device, 2, &v) || v.shape[0] != rows || v.shape[1] != n ||
            (type != Py_None && type != (v.is_f32 ? f32 : bf16)))
            return leave(NULL);
        Py_INCREF(out);
        a.out = (void*)v.ptr;
        a.out_stride = v.stride[0];
        a.out_dtype = v.is_f32 ? MK_F32 : MK_BF16;
    }
    a.rows = (int32_t)rows; a.n = (int32_t)n; a.k = (int32_t)k;
    a.x = (const void*)vx.ptr;
    a.x_stride = vx.stride[0];
    a.w = (const void*)vw.ptr;
    mk_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = linear_fn(&a, stream);
    Py_END_ALLOW_THREADS;
    return st == MK_OK ? out : leave(out);
}

static int lengths(PyObject* o, int32_t* out, Py_ssize_t* n) {
    if (!PyList_Check(o) && !PyTuple_Check(o)) return 0;
    *n = PySequence_Fast_GET_SIZE(o);
    if (*n < 1 || *n > MK_ATTEND_MAX_BATCH) return 0;
    for (Py_ssize_t i = 0; i < *n; ++i)
        if (!small(PySequence_Fast_GET_ITEM(o, i), out + i)) return 0;
    return 1;
}

/* attend(q, k, v, q_lens, kv_lens, layer, window, sinks, shared_prefix, scale, pages, out, workspace, status) */
static PyObject* call_attend(PyObject* self, PyObject* const* arg, Py_ssize_t n_arg) {
    (void)self;
    if (n_arg != 14) return leave(NULL);
    PyObject *q = arg[0], *scale = arg[9], *pages = arg[10], *out = arg[11], *workspace = arg[12];
    mk_attend_args a = {0};
    mk_kv kv = {0};
    mk_kv_pages pg = {0};
    int32_t q_lens[MK_ATTEND_MAX_BATCH], kv_lens[MK_ATTEND_MAX_BATCH];
    Py_ssize_t batch, kv_batch;
    int64_t device, sum = 0;
    View vq, vk, vv, v;
    if (!device_of(q, &device) || !view(q, bf16, 0, device, 3, &vq) || !lengths(arg[3], q_lens, &batch) ||
        !lengths(arg[4], kv_lens, &kv_batch) || batch != kv_batch)
        return leave(NULL);
    for (Py_ssize_t i = 0; i < batch; ++i) sum += q_lens[i];
    const int64_t nq = vq.shape[1], d = vq.shape[2];
    if (sum > vq.shape[0] || !small(arg[5], &a.layer) || !small(arg[6], &a.window) || !small(arg[7], &a.sinks) ||
        !small(arg[8], &a.shared_prefix))
        return leave(NULL);
    if (scale != Py_None) {
        const double s = PyFloat_AsDouble(scale);
        a.scale = (float)s;
        if (!(s > 0) || !(a.scale > 0)) return leave(NULL);
    }
    const int dims = pages == Py_None ? 5 : 4;
    if (!view(arg[1], bf16, 0, device, dims, &vk) || !view(arg[2], bf16, 0, device, dims, &vv)) return leave(NULL);
    for (int i = 0; i < dims; ++i)
        if (vk.shape[i] != vv.shape[i] || vk.stride[i] != vv.stride[i]) return leave(NULL);
    const int64_t *shape = vk.shape + dims - 4, *stride = vk.stride + dims - 4;   /* layer, head, position, element */
    int64_t positions = shape[2];
    if (shape[3] != d || (stride[2] != d && positions > 1) || a.layer < 0 || a.layer >= shape[0]) return leave(NULL);
    kv.k = (void*)vk.ptr;
    kv.v = (void*)vv.ptr;
    kv.layer_stride = stride[0];
    kv.head_stride = stride[1];
    if (pages == Py_None) {
        if (vk.shape[0] < batch) return leave(NULL);
        kv.batch_stride = vk.stride[0];
    } else {
        if (!PyTuple_Check(pages) || PyTuple_GET_SIZE(pages) != 3 || !view(PyTuple_GET_ITEM(pages, 0), i32, 0, device, 2, &v) ||
            !small(PyTuple_GET_ITEM(pages, 1), &pg.block_size) || !small(PyTuple_GET_ITEM(pages, 2), &pg.n_blocks) ||
            v.shape[0] < batch || (v.stride[0] != v.shape[1] && v.shape[0] > 1) || !fits(v.shape[1]) || pg.block_size < 1 ||
            pg.n_blocks < 1 || positions < (int64_t)pg.n_blocks * pg.block_size)
            return leave(NULL);
        pg.block_table = (const int32_t*)v.ptr;
        pg.max_blocks = (int32_t)v.shape[1];
        positions = v.shape[1] * pg.block_size;
        a.pages = &pg;
    }
    void* stream;
    if (!fits(nq) || !fits(d) || !fits(shape[1]) || !status_of(arg[13], device, &a.status) || !stream_of(device, &stream))
        return leave(NULL);
    int64_t ws = 0, ws_bytes = 0, item;
    if (workspace != Py_None) {
        PyObject* c = PyObject_CallMethodNoArgs(workspace, s_is_contiguous);
        const int contiguous = c == Py_True;
        Py_XDECREF(c);
        int64_t at;
        if (!contiguous || !method(workspace, s_get_device, &at) || at != device || !method(workspace, s_data_ptr, &ws) ||
            !method(workspace, s_numel, &ws_bytes) || !method(workspace, s_element_size, &item))
            return leave(NULL);
        ws_bytes *= item;
    }
    int64_t out_row, out_head;
    if (out == Py_None) {
        int64_t ptr;
        out = new_tensor(q, vq.shape, 3, bf16);
        if (!out || !method(out, s_data_ptr, &ptr)) return leave(out);
        a.out = (void*)(uintptr_t)ptr;
        out_row = nq * d;
        out_head = d;
    } else {
        if (!view(out, bf16, 0, device, 3, &v) || v.shape[0] != vq.shape[0] || v.shape[1] != nq || v.shape[2] != d) return leave(NULL);
        Py_INCREF(out);
        a.out = (void*)v.ptr;
        out_row = v.stride[0];
        out_head = v.stride[1];
    }
    if (nq > 1 && (vq.stride[1] != d || out_head != d)) return leave(out);
    a.n_q_heads = (int32_t)nq; a.n_kv_heads = (int32_t)shape[1]; a.head_dim = (int32_t)d; a.batch = (int32_t)batch;
    a.q_lens = q_lens;
    a.kv_lens = kv_lens;
    a.q = (const void*)vq.ptr;
    a.q_stride = vq.stride[0];
    a.out_stride = out_row;
    a.kv = &kv;
    a.max_seq = (int32_t)(positions < (1 << 30) ? positions : 1 << 30);
    PyObject *ptr = NULL;   /* a workspace of torch's allocator, given back behind the call in stream order */
    if (workspace == Py_None && (ws_bytes = (int64_t)attend_workspace_fn(&a)) > 0) {
        PyObject* args[2] = {PyLong_FromLongLong(ws_bytes), PyLong_FromVoidPtr(stream)};
        if (args[0] && args[1]) ptr = PyObject_Vectorcall(raw_alloc, args, 2, NULL);
        Py_XDECREF(args[0]);
        Py_XDECREF(args[1]);
        if (!ptr || !PyLong_Check(ptr)) {
            Py_XDECREF(ptr);
            return leave(out);
        }
        ws = (int64_t)PyLong_AsLongLong(ptr);
    }
    mk_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = attend_fn(&a, (void*)(uintptr_t)ws, (size_t)ws_bytes, stream);
    Py_END_ALLOW_THREADS;
    if (ptr) {
        PyObject* r = PyObject_CallOneArg(raw_delete, ptr);
        Py_DECREF(ptr);
        if (!r) PyErr_Clear();
        Py_XDECREF(r);
    }
    return st == MK_OK ? out : leave(out);
}

/* setup(mk_linear, mk_attend, mk_attend_workspace, bf16, f32, i32, empty, raw_stream, current_device, raw_alloc, raw_delete) */
static PyObject* setup(PyObject* self, PyObject* const* arg, Py_ssize_t n_arg) {
    (void)self;
    if (n_arg != 11) return PyErr_Format(PyExc_TypeError, "setup takes 11 arguments");
    linear_fn = (mk_status (*)(const mk_linear_args*, void*))PyLong_AsVoidPtr(arg[0]);
    attend_fn = (mk_status (*)(const mk_attend_args*, void*, size_t, void*))PyLong_AsVoidPtr(arg[1]);
    attend_workspace_fn = (size_t (*)(const mk_attend_args*))PyLong_AsVoidPtr(arg[2]);
    if (PyErr_Occurred()) return NULL;
    PyObject** held[8] = {&bf16, &f32, &i32, &empty, &raw_stream, &current_device, &raw_alloc, &raw_delete};
    for (int i = 0; i < 8; ++i) {
        Py_INCREF(arg[3 + i]);
        Py_XSETREF(*held[i], arg[3 + i]);
    }
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"linear", (PyCFunction)(void (*)(void))call_linear, METH_FASTCALL, NULL},
    {"attend", (PyCFunction)(void (*)(void))call_attend, METH_FASTCALL, NULL},
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mk_call", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__mk_call(void) {
    struct { PyObject** at; const char* name; } names[] = {
        {&s_dtype, "dtype"}, {&s_shape, "shape"}, {&s_stride, "stride"}, {&s_device, "device"}, {&s_get_device, "get_device"},
        {&s_data_ptr, "data_ptr"}, {&s_is_contiguous, "is_contiguous"}, {&s_numel, "numel"}, {&s_element_size, "element_size"}};
    for (size_t i = 0; i < sizeof names / sizeof names[0]; ++i)
        if (!(*names[i].at = PyUnicode_InternFromString(names[i].name))) return NULL;
    if (!(empty_names = Py_BuildValue("(ss)", "dtype", "device"))) return NULL;
    return PyModule_Create(&module);
}
