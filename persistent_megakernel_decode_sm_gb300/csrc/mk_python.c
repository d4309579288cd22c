/* The Python module _mk_call: linear(), attend(), adapted_linear(), rope_append() and assign_pages() of the package for the
 * calls that need no more than their operands' addresses, shapes and strides.  Kernels of a few microseconds leave the interpreter as the larger part of
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
static mk_status (*adapted_fn)(const mk_linear_args*, const mk_adapters*, void*, size_t, void*);
static size_t (*adapted_workspace_fn)(const mk_linear_args*, const mk_adapters*);
static mk_status (*rope_fn)(const mk_rope_args*, void*);
static mk_status (*pages_fn)(const mk_pages_args*, void*);
/* torch's objects, held for the life of the process */
static PyObject *bf16, *f32, *f64, *i32, *empty, *raw_stream, *current_device, *raw_alloc, *raw_delete;
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

/* The operands x, weight, bias, activation, residual, out, out_dtype and status of a linear map, its output (a new reference) and
 * the stream; 0 where they are not taken */
static int linear_operands(PyObject* const* arg, mk_linear_args* a, int64_t* device, void** stream, PyObject** result) {
    PyObject *x = arg[0], *w = arg[1], *bias = arg[2], *act = arg[3], *res = arg[4], *out = arg[5], *type = arg[6];
    View vx, vw, v;
    *result = NULL;
    if (!device_of(x, device) || !view(x, bf16, 0, *device, 2, &vx) || !view(w, bf16, 0, *device, 2, &vw)) return 0;
    int64_t rows = vx.shape[0], k = vx.shape[1], n = vw.shape[0];
    if (vw.shape[1] != k || (vw.stride[0] != k && n > 1)) return 0;
    a->activation = -1;
    if (act == Py_None) a->activation = MK_ACT_NONE;
    else if (PyUnicode_Check(act)) {
        if (PyUnicode_CompareWithASCIIString(act, "silu") == 0) a->activation = MK_ACT_SILU;
        else if (PyUnicode_CompareWithASCIIString(act, "gelu") == 0) a->activation = MK_ACT_GELU;
        else if (PyUnicode_CompareWithASCIIString(act, "swiglu") == 0) a->activation = MK_ACT_SWIGLU;
    }
    if (a->activation < 0) return 0;
    if (bias != Py_None) {
        if (!view(bias, bf16, 0, *device, 1, &v) || v.shape[0] != n) return 0;
        a->bias = (const void*)v.ptr;
    }
    if (a->activation == MK_ACT_SWIGLU) {
        if (n % 2) return 0;
        n /= 2;
    }
    if (!fits(rows) || !fits(n) || !fits(k)) return 0;
    if (res != Py_None) {
        if (!view(res, bf16, 1, *device, 2, &v) || v.shape[0] != rows || v.shape[1] != n) return 0;
        a->residual = (const void*)v.ptr;
        a->residual_stride = v.stride[0];
        a->residual_dtype = v.is_f32 ? MK_F32 : MK_BF16;
    }
    if (!status_of(arg[7], *device, &a->status) || !stream_of(*device, stream)) return 0;
    if (out == Py_None) {
        if (type != Py_None && type != bf16 && type != f32) return 0;
        const int64_t shape[2] = {rows, n};
        int64_t ptr;
        *result = out = new_tensor(x, shape, 2, type == f32 ? f32 : bf16);
        if (!out || !method(out, s_data_ptr, &ptr)) return 0;
        a->out = (void*)(uintptr_t)ptr;
        a->out_stride = n;
        a->out_dtype = type == f32 ? MK_F32 : MK_BF16;
    } else {
        if (!view(out, bf16, 1, *device, 2, &v) || v.shape[0] != rows || v.shape[1] != n ||
            (type != Py_None && type != (v.is_f32 ? f32 : bf16)))
            return 0;
        Py_INCREF(out);
        *result = out;
        a->out = (void*)v.ptr;
        a->out_stride = v.stride[0];
        a->out_dtype = v.is_f32 ? MK_F32 : MK_BF16;
    }
    a->rows = (int32_t)rows; a->n = (int32_t)n; a->k = (int32_t)k;
    a->x = (const void*)vx.ptr;
    a->x_stride = vx.stride[0];
    a->w = (const void*)vw.ptr;
    return 1;
}

/* linear(x, weight, bias, activation, residual, out, out_dtype, status) */
static PyObject* call_linear(PyObject* self, PyObject* const* arg, Py_ssize_t n_arg) {
    (void)self;
    if (n_arg != 8) return leave(NULL);
    mk_linear_args a = {0};
    int64_t device;
    void* stream;
    PyObject* out;
    if (!linear_operands(arg, &a, &device, &stream, &out)) return leave(out);
    mk_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = linear_fn(&a, stream);
    Py_END_ALLOW_THREADS;
    return st == MK_OK ? out : leave(out);
}

/* A caller's workspace, contiguous on the device: its address and bytes */
static int workspace_of(PyObject* t, int64_t device, int64_t* ws, int64_t* bytes) {
    int64_t at, item;
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    const int contiguous = c == Py_True;
    Py_XDECREF(c);
    if (!contiguous || !method(t, s_get_device, &at) || at != device || !method(t, s_data_ptr, ws) || !method(t, s_numel, bytes) ||
        !method(t, s_element_size, &item))
        return 0;
    *bytes *= item;
    return 1;
}
/* A workspace of torch's allocator (*held: what gives it back behind the call, in stream order) */
static int workspace_new(int64_t bytes, void* stream, int64_t* ws, PyObject** held) {
    PyObject* args[2] = {PyLong_FromLongLong(bytes), PyLong_FromVoidPtr(stream)};
    if (args[0] && args[1]) *held = PyObject_Vectorcall(raw_alloc, args, 2, NULL);
    Py_XDECREF(args[0]);
    Py_XDECREF(args[1]);
    if (!*held || !PyLong_Check(*held)) {
        Py_CLEAR(*held);
        return 0;
    }
    *ws = (int64_t)PyLong_AsLongLong(*held);
    return 1;
}
static void workspace_back(PyObject* held) {
    if (!held) return;
    PyObject* r = PyObject_CallOneArg(raw_delete, held);
    Py_DECREF(held);
    if (!r) PyErr_Clear();
    Py_XDECREF(r);
}

/* adapted_linear(x, weight, bias, activation, residual, out, out_dtype, status, down, up, scale, index, workspace) */
static PyObject* call_adapted(PyObject* self, PyObject* const* arg, Py_ssize_t n_arg) {
    (void)self;
    if (n_arg != 13) return leave(NULL);
    mk_linear_args a = {0};
    mk_adapters ad = {0};
    int64_t device, ws = 0, bytes = 0;
    void* stream;
    PyObject *out, *held = NULL;
    View vd, vu, v;
    if (!linear_operands(arg, &a, &device, &stream, &out)) return leave(out);
    const int64_t n = (int64_t)a.n * (a.activation == MK_ACT_SWIGLU ? 2 : 1);
    if (!view(arg[8], bf16, 0, device, 3, &vd) || !view(arg[9], bf16, 0, device, 3, &vu)) return leave(out);
    const int64_t count = vd.shape[0], rank = vd.shape[1];
    if (!fits(count) || !fits(rank) || vd.shape[2] != a.k || (vd.stride[1] != a.k && rank > 1) || (vd.stride[0] != rank * a.k && count > 1) ||
        vu.shape[0] != count || vu.shape[1] != n || vu.shape[2] != rank || (vu.stride[1] != rank && n > 1) ||
        (vu.stride[0] != n * rank && count > 1))
        return leave(out);
    if (arg[10] != Py_None) {
        if (!view(arg[10], f32, 0, device, 1, &v) || v.shape[0] != count) return leave(out);
        ad.scale = (const float*)v.ptr;
    }
    if (!view(arg[11], i32, 0, device, 1, &v) || v.shape[0] != a.rows) return leave(out);
    ad.index = (const int32_t*)v.ptr;
    ad.n_adapters = (int32_t)count;
    ad.rank = (int32_t)rank;
    ad.down = (const void*)vd.ptr;
    ad.up = (const void*)vu.ptr;
    if (arg[12] != Py_None) {
        if (!workspace_of(arg[12], device, &ws, &bytes)) return leave(out);
    } else if ((bytes = (int64_t)adapted_workspace_fn(&a, &ad)) > 0 && !workspace_new(bytes, stream, &ws, &held)) {
        return leave(out);
    }
    mk_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = adapted_fn(&a, &ad, (void*)(uintptr_t)ws, (size_t)bytes, stream);
    Py_END_ALLOW_THREADS;
    workspace_back(held);
    return st == MK_OK ? out : leave(out);
}

/* rope_append(qkv, k, v, positions, slots, freqs, layer, sections, neighbours, q_gain, k_gain, eps, out, status) */
static PyObject* call_rope(PyObject* self, PyObject* const* arg, Py_ssize_t n_arg) {
    (void)self;
    if (n_arg != 14) return leave(NULL);
    PyObject *qkv = arg[0], *sections = arg[7], *out = arg[12];
    mk_rope_args a = {0};
    mk_kv kv = {0};
    int32_t parts[4];
    int64_t device;
    View vx, vk, vv, v;
    if (!device_of(qkv, &device) || !view(qkv, bf16, 1, device, 2, &vx)) return leave(NULL);
    int dims = 5;
    if (!view(arg[1], bf16, 0, device, 5, &vk)) {
        PyErr_Clear();
        dims = 4;
        if (!view(arg[1], bf16, 0, device, 4, &vk)) return leave(NULL);
    }
    if (!view(arg[2], bf16, 0, device, dims, &vv)) return leave(NULL);
    for (int i = 0; i < dims; ++i)
        if (vk.shape[i] != vv.shape[i] || vk.stride[i] != vv.stride[i]) return leave(NULL);
    const int64_t *shape = vk.shape + dims - 4, *stride = vk.stride + dims - 4;   /* layer, head, position, element */
    const int64_t tokens = vx.shape[0], nkv = shape[1], positions = shape[2], d = shape[3], sequences = dims == 5 ? vk.shape[0] : 1;
    if (d < 1 || (stride[2] != d && positions > 1) || !small(arg[6], &a.layer) || a.layer < 0 || a.layer >= shape[0]) return leave(NULL);
    const int64_t nq = vx.shape[1] / d - 2 * nkv;
    if (nq < 1 || (nq + 2 * nkv) * d != vx.shape[1] || !fits(tokens) || !fits(nq) || !fits(nkv) || !fits(d) || !fits(positions) || !fits(sequences))
        return leave(NULL);
    if (!view(arg[5], f64, 0, -1, 1, &v) || v.shape[0] > INT32_MAX / 2) return leave(NULL);
    a.freqs = (const double*)v.ptr;
    a.rotary = (int32_t)(2 * v.shape[0]);
    a.n_axes = 1;
    if (sections != Py_None) {
        if (!PyList_Check(sections) && !PyTuple_Check(sections)) return leave(NULL);
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(sections);
        if (n < 1 || n > 4) return leave(NULL);
        for (Py_ssize_t i = 0; i < n; ++i)
            if (!small(PySequence_Fast_GET_ITEM(sections, i), parts + i)) return leave(NULL);
        a.n_axes = (int32_t)n;
        a.sections = parts;
        if (!view(arg[3], i32, 0, device, 2, &v) || v.shape[0] != n || v.shape[1] != tokens) return leave(NULL);
        a.position_stride = v.stride[0];
    } else if (!view(arg[3], i32, 0, device, 1, &v) || v.shape[0] != tokens) {
        return leave(NULL);
    }
    a.positions = (const int32_t*)v.ptr;
    if (!view(arg[4], i32, 0, device, 1, &v) || v.shape[0] != tokens) return leave(NULL);
    a.slots = (const int32_t*)v.ptr;
    if (!PyBool_Check(arg[8])) return leave(NULL);
    a.neighbours = arg[8] == Py_True;
    for (int i = 0; i < 2; ++i)
        if (arg[9 + i] != Py_None) {
            if (!view(arg[9 + i], bf16, 0, device, 1, &v) || v.shape[0] != d) return leave(NULL);
            *(i ? &a.k_gain : &a.q_gain) = (const void*)v.ptr;
        }
    if (!PyFloat_Check(arg[11])) return leave(NULL);
    a.eps = (float)PyFloat_AS_DOUBLE(arg[11]);
    void* stream;
    if (!status_of(arg[13], device, &a.status) || !stream_of(device, &stream)) return leave(NULL);
    if (out == Py_None) {
        const int64_t size[3] = {tokens, nq, d};
        int64_t ptr;
        out = new_tensor(qkv, size, 3, bf16);
        if (!out || !method(out, s_data_ptr, &ptr)) return leave(out);
        a.q = (void*)(uintptr_t)ptr;
        a.q_stride = nq * d;
    } else {
        if (!view(out, bf16, 0, device, 3, &v) || v.shape[0] != tokens || v.shape[1] != nq || v.shape[2] != d || (v.stride[1] != d && nq > 1))
            return leave(NULL);
        Py_INCREF(out);
        a.q = (void*)v.ptr;
        a.q_stride = v.stride[0];
    }
    a.tokens = (int32_t)tokens; a.n_q_heads = (int32_t)nq; a.n_kv_heads = (int32_t)nkv; a.head_dim = (int32_t)d;
    a.qkv = (const void*)vx.ptr;
    a.qkv_stride = vx.stride[0];
    a.qkv_dtype = vx.is_f32 ? MK_F32 : MK_BF16;
    kv.k = (void*)vk.ptr;
    kv.v = (void*)vv.ptr;
    kv.batch_stride = dims == 5 ? vk.stride[0] : 0;
    kv.layer_stride = stride[0];
    kv.head_stride = stride[1];
    a.kv = &kv;
    a.max_seq = (int32_t)positions;
    a.sequences = (int32_t)sequences;
    mk_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = rope_fn(&a, stream);
    Py_END_ALLOW_THREADS;
    return st == MK_OK ? out : leave(out);
}

/* assign_pages(ring, ends, ends_out, table, lens, new_lens, block_size, max_tokens, shared_prefix, out, status) */
static PyObject* call_pages(PyObject* self, PyObject* const* arg, Py_ssize_t n_arg) {
    (void)self;
    if (n_arg != 11) return leave(NULL);
    mk_pages_args a = {0};
    int64_t device;
    View ring, ends, ends_out, table, lens, wanted, v;
    if (!device_of(arg[0], &device) || !view(arg[0], i32, 0, device, 1, &ring) || !view(arg[1], i32, 0, device, 1, &ends) ||
        !view(arg[2], i32, 0, device, 1, &ends_out) || !view(arg[3], i32, 0, device, 2, &table) || !view(arg[4], i32, 0, device, 1, &lens) ||
        !view(arg[5], i32, 0, device, 1, &wanted) || !small(arg[6], &a.block_size) || !small(arg[7], &a.max_tokens) ||
        !small(arg[8], &a.shared_prefix))
        return leave(NULL);
    const int64_t batch = table.shape[0], columns = table.shape[1];
    if (!fits(batch) || !fits(columns) || !fits(ring.shape[0]) || (table.stride[0] != columns && batch > 1) || lens.shape[0] != batch ||
        wanted.shape[0] != batch || ends.shape[0] != 3 || ends_out.shape[0] != 3 || a.max_tokens < 0)
        return leave(NULL);
    void* stream;
    if (!status_of(arg[10], device, &a.status) || !stream_of(device, &stream)) return leave(NULL);
    PyObject* out;
    int32_t** to[4] = {&a.slots, &a.positions, &a.sequences, &a.first};
    if (arg[9] != Py_None) {
        if (!PyTuple_Check(arg[9]) || PyTuple_GET_SIZE(arg[9]) != 4) return leave(NULL);
        out = arg[9];
        Py_INCREF(out);
    } else if (!(out = PyTuple_New(4))) {
        return leave(NULL);
    }
    for (int i = 0; i < 4; ++i) {
        const int64_t n = i < 3 ? a.max_tokens : batch + 1;
        if (arg[9] == Py_None) {
            PyObject* t = new_tensor(arg[0], &n, 1, i32);
            int64_t ptr;
            if (!t) return leave(out);
            PyTuple_SET_ITEM(out, i, t);
            if (!method(t, s_data_ptr, &ptr)) return leave(out);
            *to[i] = (int32_t*)(uintptr_t)ptr;
        } else {
            if (!view(PyTuple_GET_ITEM(out, i), i32, 0, device, 1, &v) || v.shape[0] != n) return leave(out);
            *to[i] = (int32_t*)v.ptr;
        }
    }
    a.batch = (int32_t)batch; a.max_blocks = (int32_t)columns; a.n_blocks = (int32_t)ring.shape[0];
    a.ring = (int32_t*)ring.ptr;
    a.ends = (const int32_t*)ends.ptr;
    a.ends_out = (int32_t*)ends_out.ptr;
    a.table = (int32_t*)table.ptr;
    a.lens = (const int32_t*)lens.ptr;
    a.new_lens = (const int32_t*)wanted.ptr;
    mk_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = pages_fn(&a, stream);
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
    int64_t ws = 0, ws_bytes = 0;
    if (workspace != Py_None && !workspace_of(workspace, device, &ws, &ws_bytes)) return leave(NULL);
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
    PyObject* held = NULL;
    if (workspace == Py_None && (ws_bytes = (int64_t)attend_workspace_fn(&a)) > 0 && !workspace_new(ws_bytes, stream, &ws, &held)) return leave(out);
    mk_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = attend_fn(&a, (void*)(uintptr_t)ws, (size_t)ws_bytes, stream);
    Py_END_ALLOW_THREADS;
    workspace_back(held);
    return st == MK_OK ? out : leave(out);
}

/* setup(mk_linear, mk_attend, mk_attend_workspace, mk_linear_adapted, mk_linear_adapted_workspace, mk_rope_append, mk_assign_pages,
 *       bf16, f32, f64, i32, empty, raw_stream, current_device, raw_alloc, raw_delete) */
static PyObject* setup(PyObject* self, PyObject* const* arg, Py_ssize_t n_arg) {
    (void)self;
    if (n_arg != 16) return PyErr_Format(PyExc_TypeError, "setup takes 16 arguments");
    linear_fn = (mk_status (*)(const mk_linear_args*, void*))PyLong_AsVoidPtr(arg[0]);
    attend_fn = (mk_status (*)(const mk_attend_args*, void*, size_t, void*))PyLong_AsVoidPtr(arg[1]);
    attend_workspace_fn = (size_t (*)(const mk_attend_args*))PyLong_AsVoidPtr(arg[2]);
    adapted_fn = (mk_status (*)(const mk_linear_args*, const mk_adapters*, void*, size_t, void*))PyLong_AsVoidPtr(arg[3]);
    adapted_workspace_fn = (size_t (*)(const mk_linear_args*, const mk_adapters*))PyLong_AsVoidPtr(arg[4]);
    rope_fn = (mk_status (*)(const mk_rope_args*, void*))PyLong_AsVoidPtr(arg[5]);
    pages_fn = (mk_status (*)(const mk_pages_args*, void*))PyLong_AsVoidPtr(arg[6]);
    if (PyErr_Occurred()) return NULL;
    PyObject** held[9] = {&bf16, &f32, &f64, &i32, &empty, &raw_stream, &current_device, &raw_alloc, &raw_delete};
    for (int i = 0; i < 9; ++i) {
        Py_INCREF(arg[7 + i]);
        Py_XSETREF(*held[i], arg[7 + i]);
    }
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"linear", (PyCFunction)(void (*)(void))call_linear, METH_FASTCALL, NULL},
    {"attend", (PyCFunction)(void (*)(void))call_attend, METH_FASTCALL, NULL},
    {"adapted_linear", (PyCFunction)(void (*)(void))call_adapted, METH_FASTCALL, NULL},
    {"rope_append", (PyCFunction)(void (*)(void))call_rope, METH_FASTCALL, NULL},
    {"assign_pages", (PyCFunction)(void (*)(void))call_pages, METH_FASTCALL, NULL},
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
