/* paged_calls.c -- the paged-cache calls of binding.py for the arguments that they mostly
 * get, as a CPython module.
 *
 * A call of a few microseconds on the GPU is bound by what the host does around it, and in
 * Python that is some forty attribute reads, comparisons and argument conversions (one
 * decoded token: 13.4 us a call).  Here the same is read and compared in C and the library
 * is called without ctypes in between (10 us, most of it torch's allocation and the launch).
 *
 * These functions never raise on an argument: where anything is not plain (another type or
 * device, a stride, a missing tensor, an option that is rarely given) they return
 * NotImplemented and have done nothing, and the caller's checks in Python take over, which
 * say what is wrong or handle it.  Nothing of torch is compiled in: tensors are read through
 * their Python attributes.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <math.h>
#include <stdint.h>

#include "../../include/fa.h"

typedef struct {
    void *ptr;
    PyObject *dtype; /* one of torch's dtype objects, which live as long as torch */
    int nd;
    long long size[4], stride[4];
    long device;
} Tensor;

/* set by init() */
static PyObject *t_f16, *t_bf16, *t_f32, *t_i32, *t_empty_like, *t_stream, *t_device, *t_contiguous, *t_error;
static int (*c_append)(const fa_paged_cache *, const void *, const void *, const void *, void *, long long, long long,
                       long long, long long, const int32_t *, int, const int32_t *, const int32_t *, const int32_t *,
                       int, int, int, const float *, int, int, int, void *);
static int (*c_decode)(const fa_paged_cache *, const void *, void *, const int32_t *, int, const int32_t *, int, int,
                       float, fa_dtype, void *, size_t, void *);
static int (*c_prefill)(const fa_paged_cache *, const void *, void *, float *, const int32_t *, int, const int32_t *,
                        const int32_t *, int, int, int, int, int, float, fa_dtype, void *, size_t, void *);
static int (*c_shared)(const fa_paged_cache *, const void *, void *, const int32_t *, int, const int32_t *,
                       const int32_t *, int, const int32_t *, int, int, float, fa_dtype, void *, size_t, void *);
static PyObject *s_shape, *s_stride, *s_dtype, *s_get_device, *s_data_ptr, *s_memory_format, *s_names;

static int longs(PyObject *tuple, long long *out, int *n) {
    if (!tuple || !PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) > 4) return 0;
    *n = (int)PyTuple_GET_SIZE(tuple);
    for (int i = 0; i < *n; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
        if (out[i] == -1 && PyErr_Occurred()) return 0;
    }
    return 1;
}

/* Reads a tensor; 0 (and no exception) for anything that is not one of a CUDA device. */
static int read_tensor(PyObject *o, Tensor *t) {
    int ok = 0, n = 0;
    PyObject *shape = NULL, *stride = NULL, *dtype = NULL, *device = NULL, *ptr = NULL;
    if ((shape = PyObject_GetAttr(o, s_shape)) && longs(shape, t->size, &t->nd) &&
        (stride = PyObject_CallMethodNoArgs(o, s_stride)) && longs(stride, t->stride, &n) && n == t->nd &&
        (dtype = PyObject_GetAttr(o, s_dtype)) && (device = PyObject_CallMethodNoArgs(o, s_get_device)) &&
        (ptr = PyObject_CallMethodNoArgs(o, s_data_ptr))) {
        t->dtype = dtype;
        t->device = PyLong_AsLong(device);
        t->ptr = PyLong_AsVoidPtr(ptr);
        ok = t->device >= 0 && !PyErr_Occurred();
    }
    Py_XDECREF(shape);
    Py_XDECREF(stride);
    Py_XDECREF(dtype);
    Py_XDECREF(device);
    Py_XDECREF(ptr);
    if (!ok) PyErr_Clear();
    return ok;
}

static int contiguous(const Tensor *t) { /* (a tensor without elements is) */
    long long want = 1;
    for (int i = 0; i < t->nd; ++i)
        if (t->size[i] == 0) return 1;
    for (int i = t->nd - 1; i >= 0; --i) {
        if (t->size[i] != 1 && t->stride[i] != want) return 0;
        want *= t->size[i];
    }
    return 1;
}

static int fits(long long n) { return n >= 0 && n <= INT32_MAX; }

/* int32, contiguous, nd dimensions, on the device */
static int ints(PyObject *o, Tensor *t, int nd, long device) {
    if (!read_tensor(o, t) || t->dtype != t_i32 || t->nd != nd || t->device != device || !contiguous(t)) return 0;
    for (int i = 0; i < nd; ++i)
        if (!fits(t->size[i])) return 0;
    return 1;
}

/* [tokens][heads][d] rows of the cache's type, tokens any stride apart */
static int rows(PyObject *o, Tensor *t, const Tensor *k, long long d) {
    return read_tensor(o, t) && t->dtype == k->dtype && t->device == k->device && t->nd == 3 && t->size[2] == d &&
           t->stride[2] == 1 && (t->stride[1] == d || t->size[1] == 1) && fits(t->size[0]) && fits(t->size[1]);
}

static int cache_of(PyObject *k_pages, PyObject *v_pages, fa_paged_cache *c, Tensor *k) {
    Tensor v;
    if (!read_tensor(k_pages, k) || !read_tensor(v_pages, &v)) return 0;
    if (k->nd != 4 || v.nd != 4 || v.dtype != k->dtype || v.device != k->device || k->stride[3] != 1) return 0;
    for (int i = 0; i < 4; ++i)
        if (k->size[i] != v.size[i] || k->stride[i] != v.stride[i] || !fits(k->size[i])) return 0;
    if (k->dtype != t_f16 && k->dtype != t_bf16) return 0;
    c->k_pages = k->ptr;
    c->v_pages = v.ptr;
    c->page_stride = k->stride[0];
    c->head_stride = k->stride[1];
    c->slot_stride = k->stride[2];
    c->num_pages = (int)k->size[0];
    c->num_heads = (int)k->size[1];
    c->page_size = (int)k->size[2];
    c->head_dim = (int)k->size[3];
    c->dtype = k->dtype == t_f16 ? FA_F16 : FA_BF16;
    return 1;
}

/* The current stream of the device; 0 when it is not the current device. */
static int stream_of(long device, void **stream) {
    int ok = 0;
    PyObject *now = PyObject_CallNoArgs(t_device), *s = NULL;
    if (now && PyLong_AsLong(now) == device && (s = PyObject_CallOneArg(t_stream, now))) {
        *stream = PyLong_AsVoidPtr(s);
        ok = !PyErr_Occurred();
    }
    Py_XDECREF(now);
    Py_XDECREF(s);
    if (!ok) PyErr_Clear();
    return ok;
}


static PyObject *result(int status, const char *name, PyObject *out) { /* steals out */
    if (status == FA_OK) return out;
    Py_XDECREF(out);
    PyObject *e = PyObject_CallFunction(t_error, "is", status, name);
    if (e) {
        PyErr_SetObject(t_error, e);
        Py_DECREF(e);
    }
    return NULL;
}

/* out given: the same shape and type as q, contiguous; else new.  A new reference, or NULL with no exception. */
static PyObject *output(PyObject *out, PyObject *q, const Tensor *tq, Tensor *to) {
    if (out == Py_None) { /* torch.empty_like(q, memory_format=torch.contiguous_format) */
        PyObject *args[2] = {q, t_contiguous};
        PyObject *ptr = NULL;
        out = PyObject_Vectorcall(t_empty_like, args, 1, s_names);
        if (out && (ptr = PyObject_CallMethodNoArgs(out, s_data_ptr))) {
            *to = *tq;
            to->ptr = PyLong_AsVoidPtr(ptr);
            Py_DECREF(ptr);
            long long stride = 1;
            for (int i = tq->nd - 1; i >= 0; --i) {
                to->stride[i] = stride;
                stride *= tq->size[i];
            }
            return out;
        }
        Py_XDECREF(out);
        PyErr_Clear();
        return NULL;
    }
    Py_INCREF(out);
    int ok = read_tensor(out, to) && to->nd == tq->nd && to->dtype == tq->dtype && to->device == tq->device;
    for (int i = 0; ok && i < tq->nd; ++i) ok = to->size[i] == tq->size[i];
    if (ok) return out;
    Py_DECREF(out);
    return NULL;
}

/* scale: None or a float */
static int scale_of(PyObject *o, int d, float *scale) {
    if (o == Py_None) *scale = (float)(1.0 / sqrt((double)d));
    else if (PyFloat_CheckExact(o)) *scale = (float)PyFloat_AS_DOUBLE(o);
    else return 0;
    return 1;
}

#define GIVE_UP Py_RETURN_NOTIMPLEMENTED

/* append(q, k, v, k_pages, v_pages, page_table, seq_lens, cu_seqlens, rope, interleaved, positions, out) */
static PyObject *py_append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    const int keys_alone = n == 12 && a[0] == Py_None;
    if (n != 12 || (keys_alone && a[11] != Py_None)) GIVE_UP;
    fa_paged_cache c;
    Tensor kp, q, k, v, table, lens, cu, pos, rope, to;
    if (!cache_of(a[3], a[4], &c, &kp)) GIVE_UP;
    const long long d = c.head_dim;
    if ((!keys_alone && !rows(a[0], &q, &kp, d)) || !rows(a[1], &k, &kp, d) || !rows(a[2], &v, &kp, d)) GIVE_UP;
    const long long total = k.size[0];
    if (total < 1 || (!keys_alone && q.size[0] != total) || v.size[0] != total || k.size[1] != c.num_heads || v.size[1] != c.num_heads) GIVE_UP;
    if (!ints(a[5], &table, 2, kp.device) || !ints(a[6], &lens, 1, kp.device) || table.size[0] != lens.size[0]) GIVE_UP;
    cu.ptr = pos.ptr = rope.ptr = NULL;
    if (a[7] != Py_None && (!ints(a[7], &cu, 1, kp.device) || cu.size[0] != lens.size[0] + 1)) GIVE_UP;
    rope.size[0] = rope.size[1] = 0;
    if (a[8] != Py_None && (!read_tensor(a[8], &rope) || rope.dtype != t_f32 || rope.nd != 2 || rope.device != kp.device ||
                            !contiguous(&rope) || !fits(rope.size[0]) || !fits(rope.size[1])))
        GIVE_UP;
    if (a[10] != Py_None && (!ints(a[10], &pos, 1, kp.device) || pos.size[0] != total)) GIVE_UP;
    const int inter = PyObject_IsTrue(a[9]);
    if (inter < 0) {
        PyErr_Clear();
        GIVE_UP;
    }
    void *stream;
    if (!stream_of(kp.device, &stream)) GIVE_UP;
    PyObject *out;
    if (keys_alone) {
        q.ptr = to.ptr = NULL;
        q.stride[0] = to.stride[0] = q.size[1] = 0;
        out = Py_NewRef(Py_None);
    } else {
        out = output(a[11], a[0], &q, &to);
        if (!out) GIVE_UP;
        if (to.stride[2] != 1 || (to.stride[1] != d && to.size[1] != 1)) {
            Py_DECREF(out);
            GIVE_UP;
        }
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = c_append(&c, q.ptr, k.ptr, v.ptr, to.ptr, q.stride[0], k.stride[0], v.stride[0], to.stride[0], table.ptr,
                  (int)table.size[1], lens.ptr, cu.ptr, pos.ptr, (int)lens.size[0], (int)q.size[1], (int)total,
                  rope.size[1] ? rope.ptr : NULL, (int)rope.size[0], (int)rope.size[1], inter, stream);
    Py_END_ALLOW_THREADS
    return result(rc, "fa_cache_append", out);
}

/* What the attention calls share; 0 to give up. */
static int attention(PyObject *const *a, PyObject *table_o, PyObject *lens_o, PyObject *scale_o, fa_paged_cache *c,
                     Tensor *q, Tensor *table, Tensor *lens, float *scale, void **stream) {
    Tensor kp;
    return cache_of(a[1], a[2], c, &kp) && read_tensor(a[0], q) && q->dtype == kp.dtype && q->device == kp.device &&
           q->nd >= 3 && q->size[q->nd - 1] == c->head_dim && (q->nd == 3 || q->size[2] == 1) && fits(q->size[0]) &&
           fits(q->size[1]) && contiguous(q) && ints(table_o, table, 2, kp.device) && ints(lens_o, lens, 1, kp.device) &&
           table->size[0] == lens->size[0] && scale_of(scale_o, c->head_dim, scale) && stream_of(kp.device, stream);
}

/* decode(q, k_pages, v_pages, page_table, seq_lens, scale, out) */
static PyObject *py_decode(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    fa_paged_cache c;
    Tensor q, table, lens, to;
    float scale;
    void *stream;
    if (n != 7 || !attention(a, a[3], a[4], a[5], &c, &q, &table, &lens, &scale, &stream) || q.size[0] != lens.size[0]) GIVE_UP;
    PyObject *out = output(a[6], a[0], &q, &to);
    if (!out) GIVE_UP;
    if (!contiguous(&to)) {
        Py_DECREF(out);
        GIVE_UP;
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = c_decode(&c, q.ptr, to.ptr, table.ptr, (int)table.size[1], lens.ptr, (int)q.size[0], (int)q.size[1], scale, c.dtype,
                  NULL, 0, stream);
    Py_END_ALLOW_THREADS
    return result(rc, "fa_decode_paged", out);
}

/* prefill(q, k_pages, v_pages, page_table, seq_lens, cu_seqlens_q, max_seqlen_q, causal, scale, out) */
static PyObject *py_prefill(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    fa_paged_cache c;
    Tensor q, table, lens, cu, to;
    float scale;
    void *stream;
    if (n != 10 || !attention(a, a[3], a[4], a[8], &c, &q, &table, &lens, &scale, &stream) || q.nd != 3 || q.size[0] < 1 ||
        !ints(a[5], &cu, 1, q.device) || cu.size[0] != lens.size[0] + 1 || !PyLong_CheckExact(a[6]))
        GIVE_UP;
    const long long most = PyLong_AsLongLong(a[6]);
    const int causal = PyObject_IsTrue(a[7]);
    if (PyErr_Occurred() || !fits(most) || causal < 0) {
        PyErr_Clear();
        GIVE_UP;
    }
    PyObject *out = output(a[9], a[0], &q, &to);
    if (!out) GIVE_UP;
    if (!contiguous(&to)) {
        Py_DECREF(out);
        GIVE_UP;
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = c_prefill(&c, q.ptr, to.ptr, NULL, table.ptr, (int)table.size[1], lens.ptr, cu.ptr, (int)lens.size[0], (int)q.size[1],
                   (int)q.size[0], (int)most, causal, scale, c.dtype, NULL, 0, stream);
    Py_END_ALLOW_THREADS
    return result(rc, "fa_prefill_paged", out);
}

/* shared(q, k_pages, v_pages, prefix_table, prefix_len, page_table, seq_lens, scale, out) */
static PyObject *py_shared(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    fa_paged_cache c;
    Tensor q, front, front_len, table, lens, to;
    float scale;
    void *stream;
    if (n != 9 || !attention(a, a[5], a[6], a[7], &c, &q, &table, &lens, &scale, &stream) || q.size[0] != lens.size[0] ||
        !ints(a[3], &front, 1, q.device) || !ints(a[4], &front_len, 1, q.device) || front_len.size[0] != 1)
        GIVE_UP;
    PyObject *out = output(a[8], a[0], &q, &to);
    if (!out) GIVE_UP;
    if (!contiguous(&to)) {
        Py_DECREF(out);
        GIVE_UP;
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = c_shared(&c, q.ptr, to.ptr, front.ptr, (int)front.size[0], front_len.ptr, table.ptr, (int)table.size[1], lens.ptr,
                  (int)q.size[0], (int)q.size[1], scale, c.dtype, NULL, 0, stream);
    Py_END_ALLOW_THREADS
    return result(rc, "fa_decode_shared", out);
}

/* init(torch, FaError, addresses of fa_cache_append, fa_decode_paged, fa_prefill_paged, fa_decode_shared) */
static PyObject *py_init(PyObject *self, PyObject *args) {
    (void)self;
    PyObject *torch, *error, *inner;
    unsigned long long f[4];
    if (!PyArg_ParseTuple(args, "OOKKKK", &torch, &error, &f[0], &f[1], &f[2], &f[3])) return NULL;
    struct {
        PyObject **to;
        const char *name;
    } const names[] = {{&s_shape, "shape"}, {&s_stride, "stride"}, {&s_dtype, "dtype"}, {&s_get_device, "get_device"},
                       {&s_data_ptr, "data_ptr"}, {&s_memory_format, "memory_format"}};
    for (size_t i = 0; i < sizeof names / sizeof *names; ++i)
        if (!*names[i].to && !(*names[i].to = PyUnicode_InternFromString(names[i].name))) return NULL;
    if (!s_names && !(s_names = PyTuple_Pack(1, s_memory_format))) return NULL;
    struct {
        PyObject **to;
        const char *name;
    } const of_torch[] = {{&t_f16, "float16"}, {&t_bf16, "bfloat16"}, {&t_f32, "float32"}, {&t_i32, "int32"},
                          {&t_empty_like, "empty_like"}, {&t_contiguous, "contiguous_format"}};
    for (size_t i = 0; i < sizeof of_torch / sizeof *of_torch; ++i)
        if (!(*of_torch[i].to = PyObject_GetAttrString(torch, of_torch[i].name))) return NULL;
    if (!(inner = PyObject_GetAttrString(torch, "_C"))) return NULL;
    t_stream = PyObject_GetAttrString(inner, "_cuda_getCurrentRawStream");
    t_device = PyObject_GetAttrString(inner, "_cuda_getDevice");
    Py_DECREF(inner);
    if (!t_stream || !t_device) return NULL;
    Py_INCREF(error);
    t_error = error;
    c_append = (void *)(uintptr_t)f[0];
    c_decode = (void *)(uintptr_t)f[1];
    c_prefill = (void *)(uintptr_t)f[2];
    c_shared = (void *)(uintptr_t)f[3];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"init", py_init, METH_VARARGS, NULL},
                                {"append", (PyCFunction)(void *)py_append, METH_FASTCALL, NULL},
                                {"decode", (PyCFunction)(void *)py_decode, METH_FASTCALL, NULL},
                                {"prefill", (PyCFunction)(void *)py_prefill, METH_FASTCALL, NULL},
                                {"shared", (PyCFunction)(void *)py_shared, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__paged_calls(void) { return PyModule_Create(&module); }
