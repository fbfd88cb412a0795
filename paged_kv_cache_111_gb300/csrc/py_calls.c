/* The int8 cache's calls and the combine from Python (module _py_calls, linked to libpagedkv.so): each reads its
 * tensors' properties through their Python methods, refuses what does not do (with the binding's own messages), and
 * makes the C call.
 *
 * These calls stand in a decode step of a few microseconds of GPU time.  Marshalled in Python (ctypes) they take 3.4 to
 * 11.5 us of host time each, of which the launch is 2; here 2.7 to 6.6.  Every call reads its tensors anew.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "pkv.h"

/* names of tensor properties, and what the binding passes to bind() */
static PyObject *s_shape, *s_dtype, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_stride, *s_nbytes;
static PyObject *s_cuda_stream, *s_enter, *s_exit;
static PyObject *t_i8, *t_bf16, *t_f32, *t_i32, *t_i64;
static PyObject *py_refuse, *py_error, *py_device, *py_on_device, *py_raw_stream;

#define MAX_DIMS 5

typedef struct {
    PyObject *object;
    void *ptr;
    long dev;
    int dims;
    int64_t size[MAX_DIMS];
} Tensor;

static int refuse(const char *what, PyObject *x, PyObject *dtype, long dev, const char *form) {
    PyObject *r = PyObject_CallFunction(py_refuse, "sOOls", what, x, dtype ? dtype : Py_None, dev, form);
    if (r) {                                     /* (it always raises) */
        Py_DECREF(r);
        PyErr_Format(PyExc_ValueError, "%s must be %s", what, form);
    }
    return -1;
}

static int get_int(PyObject *v, int64_t *out) {
    *out = PyLong_AsLongLong(v);
    return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int call_int(PyObject *x, PyObject *method, int64_t *out) {
    PyObject *v = PyObject_CallMethodNoArgs(x, method);
    if (!v) return -1;
    const int rc = get_int(v, out);
    Py_DECREF(v);
    return rc;
}

/* Sizes (method NULL) or strides into out; the number of dims, -1 with an exception set, or MAX_DIMS + 1 for more. */
static int get_tuple(PyObject *x, PyObject *method, int64_t *out) {
    PyObject *v = method ? PyObject_CallMethodNoArgs(x, method) : PyObject_GetAttr(x, s_shape);
    if (!v) return -1;
    int n = -1;
    if (!PyTuple_Check(v)) {
        PyErr_SetString(PyExc_TypeError, "a tensor's sizes and strides must be tuples");
    } else if (PyTuple_GET_SIZE(v) > MAX_DIMS) {
        n = MAX_DIMS + 1;
    } else {
        n = (int)PyTuple_GET_SIZE(v);
        for (int i = 0; i < n; ++i)
            if (get_int(PyTuple_GET_ITEM(v, i), out + i)) {
                n = -1;
                break;
            }
    }
    Py_DECREF(v);
    return n;
}

/* Device and sizes of x. */
static int look(PyObject *x, Tensor *t) {
    int64_t dev;
    t->object = x;
    if (call_int(x, s_get_device, &dev)) return -1;
    t->dev = (long)dev;
    t->dims = get_tuple(x, NULL, t->size);
    return t->dims < 0 ? -1 : 0;
}

/* 1 if x is of this type, 0 if not, -1 with an exception set. */
static int of_type(PyObject *x, PyObject *dtype) {
    PyObject *v = PyObject_GetAttr(x, s_dtype);
    if (!v) return -1;
    Py_DECREF(v);
    return v == dtype;
}

static int contiguous(PyObject *x) {
    PyObject *v = PyObject_CallMethodNoArgs(x, s_is_contiguous);
    if (!v) return -1;
    Py_DECREF(v);
    return v == Py_True;
}

static int pointer(Tensor *t) {
    PyObject *v = PyObject_CallMethodNoArgs(t->object, s_data_ptr);
    if (!v) return -1;
    t->ptr = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return !t->ptr && PyErr_Occurred() ? -1 : 0;
}

/* A contiguous tensor of this type, device and number of dims, of the sizes given (-1: any). */
static int full(const char *what, PyObject *x, PyObject *dtype, long dev, int dims, int64_t a, int64_t b, int64_t c,
                const char *form, Tensor *t) {
    if (look(x, t)) return -1;
    const int typed = of_type(x, dtype), whole = contiguous(x);
    if (typed < 0 || whole < 0) return -1;
    const int64_t want[3] = {a, b, c};
    int fits = t->dev == dev && typed && whole && t->dims == dims;
    for (int i = 0; fits && i < dims; ++i) fits = want[i] < 0 || t->size[i] == want[i];
    return fits ? pointer(t) : refuse(what, x, dtype, dev, form);
}

/* The same of a vector, or None (NULL). */
static int maybe(const char *what, PyObject *x, PyObject *dtype, long dev, int64_t size, const char *form, Tensor *t) {
    t->ptr = NULL;
    return x == Py_None ? 0 : full(what, x, dtype, dev, 1, size, 0, 0, form, t);
}

/* bf16 [T, H, width] with contiguous heads side by side, and its token stride (of one token, which means nothing: the
 * least that the call takes). */
static int heads(const char *what, PyObject *x, long dev, int64_t T, int64_t H, int64_t width, Tensor *t,
                 int64_t *step) {
    int64_t strides[MAX_DIMS];
    if (look(x, t)) return -1;
    const int typed = of_type(x, t_bf16), n = get_tuple(x, s_stride, strides);
    if (typed < 0 || n < 0) return -1;
    if (t->dev != dev || !typed || t->dims != 3 || n != 3 || t->size[0] != T || t->size[1] != H ||
        t->size[2] != width || strides[2] != 1 || (H > 1 && strides[1] != width)) {
        char form[96];
        snprintf(form, sizeof form, "[%lld, %lld, %lld] with contiguous heads", (long long)T, (long long)H,
                 (long long)width);
        return refuse(what, x, t_bf16, dev, form);
    }
    *step = T > 1 ? strides[0] : H * width;
    return pointer(t);
}

static int bytes_of(PyObject *x, int64_t *out) {
    PyObject *v = PyObject_GetAttr(x, s_nbytes);
    if (!v) return -1;
    const int rc = get_int(v, out);
    Py_DECREF(v);
    return rc;
}

typedef struct {
    void *cache;
    float *scales;
    long dev;
    int64_t blocks;
    int32_t heads, tokens, width;
} Cache;

static int int32_of(int64_t v, int32_t *out) {
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_Format(PyExc_OverflowError, "%lld does not fit 32 bits", (long long)v);
        return -1;
    }
    *out = (int32_t)v;
    return 0;
}

static int int32_arg(PyObject *v, int32_t *out) {
    int64_t wide;
    return get_int(v, &wide) || int32_of(wide, out) ? -1 : 0;
}

static int int8_cache(PyObject *cache, PyObject *scales, Cache *c) {
    Tensor t, s;
    if (look(cache, &t)) return -1;
    const int typed = of_type(cache, t_i8), whole = contiguous(cache);
    if (typed < 0 || whole < 0) return -1;
    if (t.dev < 0 || !typed || t.dims != 5 || !whole || t.size[2] != 2)
        return refuse("kv_cache", cache, t_i8, t.dev, "a contiguous [NB, Hkv, 2, 16, d]");
    if (pointer(&t) ||
        full("kv_scales", scales, t_f32, t.dev, 3, t.size[0], t.size[1], 2, "a contiguous [NB, Hkv, 2]", &s))
        return -1;
    c->cache = t.ptr, c->scales = s.ptr, c->dev = t.dev, c->blocks = t.size[0];
    return int32_of(t.size[1], &c->heads) || int32_of(t.size[3], &c->tokens) || int32_of(t.size[4], &c->width) ? -1 : 0;
}

static int stream_of(PyObject *stream, long dev, void **out) {
    PyObject *v;
    if (stream == Py_None) {
        PyObject *d = PyLong_FromLong(dev);
        if (!d) return -1;
        v = PyObject_CallOneArg(py_raw_stream, d);
        Py_DECREF(d);
    } else if (PyObject_HasAttr(stream, s_cuda_stream)) {
        v = PyObject_GetAttr(stream, s_cuda_stream);
    } else {
        v = PyNumber_Long(stream);
    }
    if (!v) return -1;
    *out = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return !*out && PyErr_Occurred() ? -1 : 0;
}

/* The tensors' device made current for a call: 0, or -1 with an exception set.  *guard is given to leave(). */
static int enter(long dev, PyObject **guard) {
    *guard = NULL;
    PyObject *now = PyObject_CallNoArgs(py_device);
    if (!now) return -1;
    const long current = PyLong_AsLong(now);
    Py_DECREF(now);
    if (current == -1 && PyErr_Occurred()) return -1;
    if (current == dev) return 0;
    *guard = PyObject_CallFunction(py_on_device, "l", dev);
    PyObject *r = *guard ? PyObject_CallMethodNoArgs(*guard, s_enter) : NULL;
    if (!r) {
        Py_CLEAR(*guard);
        return -1;
    }
    Py_DECREF(r);
    return 0;
}

static PyObject *leave(PyObject *guard, int rc, const char *name) {
    if (guard) {
        PyObject *r = PyObject_CallMethodObjArgs(guard, s_exit, Py_None, Py_None, Py_None, NULL);
        Py_DECREF(guard);
        if (!r) return NULL;
        Py_DECREF(r);
    }
    if (rc == PKV_OK) Py_RETURN_NONE;
    PyObject *e = PyObject_CallFunction(py_error, "is", rc, name);
    if (e) {
        PyErr_SetObject(py_error, e);
        Py_DECREF(e);
    }
    return NULL;
}

static int arity(Py_ssize_t have, Py_ssize_t want) {
    if (have == want) return 0;
    PyErr_Format(PyExc_TypeError, "%zd arguments instead of %zd", have, want);
    return -1;
}

#define CALL(name, dev, ...)                                   \
    PyObject *guard;                                           \
    if (enter(dev, &guard)) return NULL;                       \
    int rc;                                                    \
    Py_BEGIN_ALLOW_THREADS rc = name(__VA_ARGS__);             \
    Py_END_ALLOW_THREADS return leave(guard, rc, #name)

/* kv_cache, kv_scales, key, value, slot_mapping, device_status, stream */
static PyObject *kv_write(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Cache c;
    Tensor slots, key, value, status;
    int64_t k_step, v_step;
    int32_t T = 0;
    void *stream;
    if (arity(n, 7) || int8_cache(a[0], a[1], &c) ||
        full("slot_mapping", a[4], t_i64, c.dev, 1, -1, 0, 0, "a contiguous [T]", &slots) ||
        int32_of(slots.size[0], &T) || heads("key", a[2], c.dev, T, c.heads, c.width, &key, &k_step) ||
        heads("value", a[3], c.dev, T, c.heads, c.width, &value, &v_step) ||
        maybe("device_status", a[5], t_i32, c.dev, -1, "a contiguous vector", &status) ||
        stream_of(a[6], c.dev, &stream))
        return NULL;
    CALL(pkv_kv_write_int8, c.dev, c.cache, c.scales, c.blocks, c.heads, c.width, c.tokens, key.ptr, k_step, value.ptr,
         v_step, slots.ptr, T, status.ptr, stream);
}

/* query_out, kv_cache, kv_scales, query, key, value, q_weight, k_weight, eps, cos_sin, positions, slot_mapping,
 * interleaved, device_status, stream */
static PyObject *qk_norm_rope_kv_write(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Cache c;
    Tensor q, qo, k, v, wq, wk, table, positions, slots, status;
    int64_t qo_step, q_step, k_step, v_step;
    int32_t T = 0, H = 0, rot = 0;
    void *stream;
    if (arity(n, 15) || int8_cache(a[1], a[2], &c) || look(a[3], &q)) return NULL;
    if (q.dims != 3) {
        PyErr_SetString(PyExc_ValueError, "query must be [T, H, d]");
        return NULL;
    }
    const double eps = PyFloat_AsDouble(a[8]);
    if (eps == -1.0 && PyErr_Occurred()) return NULL;
    const int inter = PyObject_IsTrue(a[12]);
    if (inter < 0 || int32_of(q.size[0], &T) || int32_of(q.size[1], &H) ||
        heads("query_out", a[0], c.dev, T, H, c.width, &qo, &qo_step) ||
        heads("query", a[3], c.dev, T, H, c.width, &q, &q_step) ||
        heads("key", a[4], c.dev, T, c.heads, c.width, &k, &k_step) ||
        heads("value", a[5], c.dev, T, c.heads, c.width, &v, &v_step) ||
        full("cos_sin", a[9], t_f32, c.dev, 2, -1, -1, 0, "a contiguous [max_position, rotary_dim]", &table) ||
        int32_of(table.size[1], &rot) || maybe("q_weight", a[6], t_bf16, c.dev, c.width, "[d]", &wq) ||
        maybe("k_weight", a[7], t_bf16, c.dev, c.width, "[d]", &wk) ||
        full("positions", a[10], t_i64, c.dev, 1, T, 0, 0, "a contiguous [T]", &positions) ||
        full("slot_mapping", a[11], t_i64, c.dev, 1, T, 0, 0, "a contiguous [T]", &slots) ||
        maybe("device_status", a[13], t_i32, c.dev, -1, "a contiguous vector", &status) ||
        stream_of(a[14], c.dev, &stream))
        return NULL;
    CALL(pkv_qk_norm_rope_kv_write_int8, c.dev, qo.ptr, qo_step, c.cache, c.scales, c.blocks, H, c.heads, c.width,
         c.tokens, q.ptr, q_step, k.ptr, k_step, v.ptr, v_step, wq.ptr, wk.ptr, (float)eps, table.ptr, table.size[0],
         rot, inter, positions.ptr, slots.ptr, T, status.ptr, stream);
}

/* out, query, kv_cache, kv_scales, block_tables, seq_lens, query_start_loc, max_query_len, max_seq_len, scale,
 * workspace, num_splits, stream */
static PyObject *paged_attn(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Cache c;
    Tensor q, out, tables, lens, starts, ws;
    int64_t q_step, bytes;
    int32_t T = 0, H = 0, S = 0, width = 0, max_q, max_n, splits;
    void *stream;
    if (arity(n, 13) || int8_cache(a[2], a[3], &c) || look(a[1], &q)) return NULL;
    if (q.dims != 3) {
        PyErr_SetString(PyExc_ValueError, "query must be [T, H, d]");
        return NULL;
    }
    const double scale = PyFloat_AsDouble(a[9]);
    if (scale == -1.0 && PyErr_Occurred()) return NULL;
    if (int32_of(q.size[0], &T) || int32_of(q.size[1], &H) || heads("query", a[1], c.dev, T, H, c.width, &q, &q_step) ||
        full("out", a[0], t_bf16, c.dev, 3, T, H, c.width, "a contiguous [T, H, d]", &out) ||
        full("seq_lens", a[5], t_i32, c.dev, 1, -1, 0, 0, "a contiguous [num_seqs]", &lens) ||
        int32_of(lens.size[0], &S) ||
        full("block_tables", a[4], t_i32, c.dev, 2, S, -1, 0, "a contiguous [num_seqs, max_blocks]", &tables) ||
        int32_of(tables.size[1], &width) ||
        full("query_start_loc", a[6], t_i32, c.dev, 1, (int64_t)S + 1, 0, 0, "a contiguous [num_seqs + 1]", &starts) ||
        look(a[10], &ws))
        return NULL;
    const int whole = contiguous(a[10]);
    if (whole < 0) return NULL;
    if (ws.dev != c.dev || !whole) {
        refuse("workspace", a[10], NULL, c.dev, "contiguous");
        return NULL;
    }
    if (bytes_of(a[10], &bytes) || pointer(&ws) || int32_arg(a[7], &max_q) || int32_arg(a[8], &max_n) ||
        int32_arg(a[11], &splits) || stream_of(a[12], c.dev, &stream))
        return NULL;
    CALL(pkv_paged_attn_int8, c.dev, out.ptr, q.ptr, q_step, c.cache, c.scales, c.blocks, tables.ptr, width, lens.ptr,
         starts.ptr, S, T, max_q, max_n, H, c.heads, c.width, c.tokens, (float)scale, splits, ws.ptr,
         (size_t)bytes, NULL, stream);
}

/* key_out, value_out, kv_cache, kv_scales, block_tables, seq_lens, key_start_loc, max_seq_len, device_status, stream */
static PyObject *kv_gather(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Cache c;
    Tensor key, value, tables, lens, starts, status;
    int32_t S = 0, width = 0, max_n;
    void *stream;
    if (arity(n, 10) || int8_cache(a[2], a[3], &c) ||
        full("key_out", a[0], t_bf16, c.dev, 3, -1, c.heads, c.width, "a contiguous [rows, Hkv, d]", &key) ||
        full("value_out", a[1], t_bf16, c.dev, 3, key.size[0], c.heads, c.width, "a contiguous [rows, Hkv, d]",
             &value) ||
        full("seq_lens", a[5], t_i32, c.dev, 1, -1, 0, 0, "a contiguous [num_seqs]", &lens) ||
        int32_of(lens.size[0], &S) ||
        full("block_tables", a[4], t_i32, c.dev, 2, S, -1, 0, "a contiguous [num_seqs, max_blocks]", &tables) ||
        int32_of(tables.size[1], &width) ||
        full("key_start_loc", a[6], t_i32, c.dev, 1, -1, 0, 0, "a contiguous vector", &starts))
        return NULL;
    if (starts.size[0] < S) {
        PyErr_SetString(PyExc_ValueError, "key_start_loc must have an entry per request");
        return NULL;
    }
    if (int32_arg(a[7], &max_n) ||
        maybe("device_status", a[8], t_i32, c.dev, -1, "a contiguous vector", &status) ||
        stream_of(a[9], c.dev, &stream))
        return NULL;
    CALL(pkv_kv_gather_int8, c.dev, key.ptr, value.ptr, key.size[0], c.cache, c.scales, c.blocks, c.heads, c.width,
         c.tokens, tables.ptr, width, lens.ptr, starts.ptr, S, max_n, status.ptr, stream);
}

/* kv_cache, kv_scales, block_mapping, device_status, stream */
static PyObject *copy_blocks(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Cache c;
    Tensor mapping, status;
    int32_t pairs = 0;
    void *stream;
    if (arity(n, 5) || int8_cache(a[0], a[1], &c) ||
        full("block_mapping", a[2], t_i64, c.dev, 2, -1, 2, 0, "a contiguous [num_pairs, 2]", &mapping) ||
        int32_of(mapping.size[0], &pairs) ||
        maybe("device_status", a[3], t_i32, c.dev, -1, "a contiguous vector", &status) ||
        stream_of(a[4], c.dev, &stream))
        return NULL;
    CALL(pkv_copy_blocks_int8, c.dev, c.cache, c.scales, c.blocks, c.heads, c.width, c.tokens, mapping.ptr, pairs,
         status.ptr, stream);
}

/* out, workspace, stream */
static PyObject *combine(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Tensor out, ws;
    int64_t bytes;
    int32_t size[3];
    void *stream;
    if (arity(n, 3) || look(a[0], &out) || look(a[1], &ws)) return NULL;
    if (out.dev < 0 || ws.dev < 0) {
        PyErr_SetString(PyExc_ValueError, "paged KV-cache calls take CUDA tensors only");
        return NULL;
    }
    if (out.dims != 3) {
        PyErr_SetString(PyExc_ValueError, "out must be [T, H, d]");
        return NULL;
    }
    for (int i = 0; i < 3; ++i)
        if (int32_of(out.size[i], size + i)) return NULL;
    if (bytes_of(a[1], &bytes) || pointer(&out) || pointer(&ws) || stream_of(a[2], out.dev, &stream)) return NULL;
    CALL(pkv_paged_attn_combine, out.dev, out.ptr, ws.ptr, (size_t)bytes, size[0], size[1], size[2], stream);
}

/* torch's int8, bfloat16, float32, int32 and int64; the binding's refusal and error; torch's current device, device
 * guard and current stream */
static PyObject *bind(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    PyObject **to[] = {&t_i8, &t_bf16, &t_f32, &t_i32, &t_i64, &py_refuse, &py_error, &py_device, &py_on_device,
                       &py_raw_stream};
    if (arity(n, 10)) return NULL;
    for (int i = 0; i < 10; ++i) {
        Py_INCREF(a[i]);
        Py_XSETREF(*to[i], a[i]);
    }
    Py_RETURN_NONE;
}

#define METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(bind),       METHOD(kv_write),  METHOD(qk_norm_rope_kv_write),
                                METHOD(paged_attn), METHOD(kv_gather), METHOD(copy_blocks),
                                METHOD(combine),    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_py_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__py_calls(void) {
    PyObject **to[] = {&s_shape, &s_dtype, &s_get_device, &s_is_contiguous, &s_data_ptr,
                       &s_stride, &s_nbytes, &s_cuda_stream, &s_enter, &s_exit};
    static const char *const names[] = {"shape", "dtype", "get_device", "is_contiguous", "data_ptr",
                                        "stride", "nbytes", "cuda_stream", "__enter__", "__exit__"};
    for (int i = 0; i < 10; ++i)
        if (!(*to[i] = PyUnicode_InternFromString(names[i]))) return NULL;
    return PyModule_Create(&module);
}
