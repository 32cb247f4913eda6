/* binding.c - the per-call path of the Python binding for the calls that are short on the GPU (rotary
 * positions, the paged cache and its tables, beam selection): argument checks, result allocation and the
 * call into libfa.so.
 *
 * A single token's append or attention takes 3 to 10 us on the GPU; the same checks in Python and
 * ctypes took 15 to 22 us on the host, this module takes about half.  It knows nothing of torch but
 * the names of tensor attributes, and it does not link to libfa.so: api.py hands over the addresses
 * of the entry points it has loaded, with the torch functions used here. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "fa.h"

typedef int (*rope_fn)(const void *, void *, const void *, void *, const long long *,
                       const uint64_t *, const int *, int, int, int, int, int, int, int, int, int,
                       float, void *);
typedef int (*append_fn)(const void *, void *, const void *, const void *, void *, void *,
                         const long long *, const int *, const int *, const int *, const int *,
                         const uint64_t *, int, int, int, int, int, int, int, int, int, int, int,
                         float, void *);
typedef int (*attn_fn)(const void *, const void *, const void *, void *, float *,
                       const long long *, const int *, const int *, const int *, int, int, int, int,
                       int, int, int, int, int, int, float, int, void *, size_t, void *);
typedef size_t (*attn_bytes_fn)(int, int, int, int, int, int, int, int);
typedef int (*reserve_fn)(int *, const int *, const int *, int *, int *, int, int, int, int, int, void *,
                          size_t, void *);
typedef size_t (*reserve_bytes_fn)(int, int, int, int);
typedef int (*fork_fn)(int *, int *, const int *, int *, int, int, int, void *);
typedef int (*free_fn)(int *, const int *, int *, int, int, int, int, void *);
typedef int (*compact_fn)(int *, int *, int *, int *, int *, int, int, int, void *);
typedef int (*copy_fn)(void *, void *, const long long *, const int *, const int *, const int *,
                       const int *, int, int, int, int, int, int, void *);
typedef int (*beam_fn)(const void *, const long long *, const float *, const uint8_t *, float *, int *,
                       int *, uint8_t *, int, int, int, int, int, int, void *, size_t, void *);
typedef size_t (*beam_bytes_fn)(int, int, int, int);

static rope_fn g_rope;
static append_fn g_append;
static attn_fn g_attn;
static attn_bytes_fn g_attn_bytes;
static reserve_fn g_reserve;
static reserve_bytes_fn g_reserve_bytes;
static fork_fn g_fork;
static free_fn g_free;
static compact_fn g_compact;
static copy_fn g_copy;
static beam_fn g_beam;
static beam_bytes_fn g_beam_bytes;
/* torch.empty, the current raw stream of a device, the current device, the dtypes, the error class: set by
 * setup() */
static PyObject *g_empty, *g_stream, *g_current, *g_bf16, *g_fp16, *g_i32, *g_i64, *g_f32, *g_u8, *g_error;
static PyObject *s_get_device, *s_contiguous, *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_device, *s_kwnames;

#define MAX_DIMS 5
typedef struct {
    PyObject *obj; /* borrowed; NULL where the caller gave None */
    const char *name;
    PyObject *dtype; /* borrowed from torch: dtypes live as long as it does */
    int dims;
    long long shape[MAX_DIMS], stride[MAX_DIMS];
    void *ptr;
} Tensor;

static int fail(PyObject *type, const char *text) {
    PyErr_SetString(type, text);
    return -1;
}

static PyObject *call0(PyObject *self, PyObject *name) {
    PyObject *args[1] = {self};
    return PyObject_VectorcallMethod(name, args, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
}

/* A tuple of at most MAX_DIMS integers into out; their number, or -1. */
static int ints_of(PyObject *tuple, long long *out) {
    if (tuple == NULL) return -1;
    int n = -1;
    if (!PyTuple_Check(tuple)) {
        fail(PyExc_TypeError, "expected a tensor");
    } else if (PyTuple_GET_SIZE(tuple) > MAX_DIMS) {
        fail(PyExc_ValueError, "tensors have at most five axes");
    } else {
        n = (int)PyTuple_GET_SIZE(tuple);
        for (int i = 0; i < n; ++i) {
            out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
            if (out[i] == -1 && PyErr_Occurred()) {
                n = -1;
                break;
            }
        }
    }
    Py_DECREF(tuple);
    return n;
}

static long device_of(PyObject *obj) {
    PyObject *x = call0(obj, s_get_device);
    if (x == NULL) return -2;
    const long dev = PyLong_AsLong(x);
    Py_DECREF(x);
    return PyErr_Occurred() ? -2 : dev;
}

/* Reads a tensor that has to be on device dev and have contiguous rows. */
static int take(PyObject *obj, const char *name, long dev, Tensor *t) {
    t->name = name;
    t->obj = obj == Py_None ? NULL : obj;
    t->ptr = NULL;
    t->dims = 0;
    t->dtype = NULL;
    if (t->obj == NULL) return 0;
    const long where = device_of(obj);
    if (where == -2) return -1;
    if (where != dev) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor on the same device as the others",
                     name);
        return -1;
    }
    t->dtype = PyObject_GetAttr(obj, s_dtype);
    if (t->dtype == NULL) return -1;
    Py_DECREF(t->dtype);
    t->dims = ints_of(PyObject_GetAttr(obj, s_shape), t->shape);
    if (t->dims < 0) return -1;
    if (t->dims == 1) { /* dense or not is all that is asked of index arrays */
        PyObject *dense = call0(obj, s_contiguous);
        if (dense == NULL) return -1;
        t->stride[0] = dense == Py_True ? 1 : 2;
        Py_DECREF(dense);
    } else if (ints_of(call0(obj, s_stride), t->stride) < 0) {
        return -1;
    }
    PyObject *p = call0(obj, s_data_ptr);
    if (p == NULL) return -1;
    t->ptr = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    if (t->ptr == NULL && PyErr_Occurred()) return -1;
    if (t->dims > 0 && t->stride[t->dims - 1] != 1 && t->shape[t->dims - 1] != 1) {
        PyErr_Format(PyExc_ValueError, "%s must have contiguous rows", name);
        return -1;
    }
    return 0;
}

static int is_dense(const Tensor *t) {
    long long want = 1;
    for (int i = t->dims - 1; i >= 0; --i) {
        if (t->shape[i] != 1 && t->stride[i] != want) return 0;
        want *= t->shape[i];
    }
    return 1;
}

static int same_shape(const Tensor *a, const Tensor *b) {
    if (a->dims != b->dims) return 0;
    for (int i = 0; i < a->dims; ++i)
        if (a->shape[i] != b->shape[i]) return 0;
    return 1;
}

/* An index array: contiguous int32 of the given extents (n1 < 0: one axis). */
static int check_index(const Tensor *t, long long n0, long long n1) {
    if (t->obj == NULL) return 0;
    if (t->dtype == g_i32 && is_dense(t) &&
        (n1 < 0 ? t->dims == 1 && t->shape[0] == n0
                : t->dims == 2 && t->shape[0] == n0 && t->shape[1] == n1))
        return 0;
    if (n1 < 0)
        PyErr_Format(PyExc_ValueError, "%s must be contiguous int32 [%lld]", t->name, n0);
    else
        PyErr_Format(PyExc_ValueError, "%s must be contiguous int32 [%lld, %lld]", t->name, n0, n1);
    return -1;
}

static int dtype_code(const Tensor *t) {
    if (t->dtype == g_bf16) return FA_BF16;
    if (t->dtype == g_fp16) return FA_FP16;
    PyErr_Format(PyExc_TypeError, "unsupported dtype %R: use torch.bfloat16 or torch.float16",
                 t->dtype);
    return -1;
}

/* The number of rotated elements of a frequency table. */
static long long freq_rot(const Tensor *f) {
    if (f->dtype != g_i64 || f->dims != 1 || !is_dense(f))
        return fail(PyExc_ValueError, "freq must be a contiguous int64 table of rope_frequencies()");
    return 2 * f->shape[0];
}

/* C's int arguments: every extent handed to the library has to be one. */
static int fits(const long long *v, int n) {
    for (int i = 0; i < n; ++i)
        if (v[i] < 0 || v[i] > 0x7fffffff) return fail(PyExc_ValueError, "an extent exceeds 2^31 - 1");
    return 0;
}

/* torch.empty(shape, dtype=, device=): a new reference, with its address; its strides are dense. */
static PyObject *new_tensor(const long long *shape, int dims, PyObject *dtype, PyObject *device,
                            void **ptr) {
    PyObject *size = PyTuple_New(dims);
    if (size == NULL) return NULL;
    for (int i = 0; i < dims; ++i) {
        PyObject *n = PyLong_FromLongLong(shape[i]);
        if (n == NULL) {
            Py_DECREF(size);
            return NULL;
        }
        PyTuple_SET_ITEM(size, i, n);
    }
    PyObject *args[4] = {NULL, size, dtype, device};
    PyObject *t = PyObject_Vectorcall(g_empty, args + 1, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, s_kwnames);
    Py_DECREF(size);
    if (t == NULL) return NULL;
    PyObject *p = call0(t, s_data_ptr);
    if (p == NULL) {
        Py_DECREF(t);
        return NULL;
    }
    *ptr = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    return t;
}

static void dense_strides(const long long *shape, int dims, long long *stride) {
    long long n = 1;
    for (int i = dims - 1; i >= 0; --i) {
        stride[i] = n;
        n *= shape[i];
    }
}

/* The result tensor: the caller's, checked, or a new dense one.  Returns a new reference. */
static PyObject *result(const Tensor *given, const Tensor *like, PyObject *device, void **ptr,
                        long long *stride) {
    if (given->obj == NULL) {
        dense_strides(like->shape, like->dims, stride);
        return new_tensor(like->shape, like->dims, like->dtype, device, ptr);
    }
    if (!same_shape(given, like) || given->dtype != like->dtype) {
        PyErr_Format(PyExc_ValueError, "%s must match %s in shape and dtype", given->name, like->name);
        return NULL;
    }
    for (int i = 0; i < given->dims; ++i) stride[i] = given->stride[i];
    *ptr = given->ptr;
    Py_INCREF(given->obj);
    return given->obj;
}

static int stream_of(long dev, void **stream) {
    PyObject *d = PyLong_FromLong(dev);
    if (d == NULL) return -1;
    PyObject *s = PyObject_CallOneArg(g_stream, d);
    Py_DECREF(d);
    if (s == NULL) return -1;
    *stream = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    return *stream == NULL && PyErr_Occurred() ? -1 : 0;
}

static int check_rc(int rc, const char *where) {
    if (rc == FA_OK) return 0;
    PyObject *e = PyObject_CallFunction(g_error, "is", rc, where);
    if (e != NULL) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return -1;
}

static int first_device(PyObject *obj, const char *name, long *dev) {
    *dev = device_of(obj);
    if (*dev == -2) return -1;
    if (*dev < 0) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
        return -1;
    }
    return 0;
}

/* Whether another device than dev is current: 0, 1, or -1 for an error. */
static int is_away(long dev) {
    PyObject *d = PyObject_CallNoArgs(g_current);
    if (d == NULL) return -1;
    const long now = PyLong_AsLong(d);
    Py_DECREF(d);
    return PyErr_Occurred() ? -1 : now != dev;
}
/* The calls below leave a tensor of another device to their Python wrapper: they return NotImplemented. */
#define LEAVE_IF_AWAY(dev)                       \
    do {                                         \
        const int away_ = is_away(dev);          \
        if (away_ < 0) return NULL;              \
        if (away_) Py_RETURN_NOTIMPLEMENTED;     \
    } while (0)

static int count_args(Py_ssize_t got, Py_ssize_t want) {
    return got == want ? 0 : fail(PyExc_TypeError, "wrong number of arguments");
}

/* rope(q, k, freq, positions, interleaved, mscale, out_q, out_k, inverse) */
static PyObject *py_rope(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Tensor q, k, freq, pos, oq, ok;
    long dev;
    if (count_args(n, 9) || first_device(a[0], "q", &dev) || take(a[0], "q", dev, &q) ||
        take(a[1], "k", dev, &k) || take(a[2], "freq", dev, &freq) ||
        take(a[3], "positions", dev, &pos) || take(a[6], "out_q", dev, &oq) ||
        take(a[7], "out_k", dev, &ok))
        return NULL;
    const int inter = PyObject_IsTrue(a[4]), inverse = PyObject_IsTrue(a[8]);
    const double mscale = PyFloat_AsDouble(a[5]);
    if (inter < 0 || inverse < 0 || (mscale == -1.0 && PyErr_Occurred())) return NULL;
    if (freq.obj == NULL) {
        fail(PyExc_ValueError, "freq must be a table of rope_frequencies()");
        return NULL;
    }
    if (q.dims != 4) {
        fail(PyExc_ValueError, "q, k must be [B, heads, N, d]");
        return NULL;
    }
    const int code = dtype_code(&q);
    const long long rot = code < 0 ? -1 : freq_rot(&freq);
    if (rot < 0) return NULL;
    if (k.obj != NULL && (k.dims != 4 || k.shape[0] != q.shape[0] || k.shape[2] != q.shape[2] ||
                          k.shape[3] != q.shape[3] || k.dtype != q.dtype)) {
        fail(PyExc_ValueError, "k must be [B, H_kv, N, d] with the dtype of q");
        return NULL;
    }
    if (k.obj == NULL && ok.obj != NULL) {
        fail(PyExc_ValueError, "out_k needs k");
        return NULL;
    }
    if (check_index(&pos, q.shape[0], q.shape[2])) return NULL;
    const long long ext[6] = {q.shape[0], q.shape[1], k.obj ? k.shape[1] : 0, q.shape[2], q.shape[3],
                              rot};
    if (fits(ext, 6)) return NULL;
    PyObject *device = PyObject_GetAttr(q.obj, s_device), *rq = NULL, *rk = NULL, *out = NULL;
    void *pq, *pk = NULL, *stream;
    long long sq[MAX_DIMS], sk[MAX_DIMS] = {0};
    if (device == NULL) return NULL;
    if ((rq = result(&oq, &q, device, &pq, sq)) == NULL) goto done;
    if (k.obj != NULL && (rk = result(&ok, &k, device, &pk, sk)) == NULL) goto done;
    if (stream_of(dev, &stream)) goto done;
    {
        const long long st[12] = {q.stride[0], q.stride[1], q.stride[2], sq[0], sq[1], sq[2],
                                  k.obj ? k.stride[0] : 0, k.obj ? k.stride[1] : 0,
                                  k.obj ? k.stride[2] : 0, sk[0], sk[1], sk[2]};
        int rc;
        Py_BEGIN_ALLOW_THREADS
        rc = g_rope(q.ptr, pq, k.ptr, pk, st, freq.ptr, pos.ptr, (int)ext[0], (int)ext[1],
                    (int)ext[2], (int)ext[3], (int)ext[4], (int)rot, code, inter, inverse,
                    (float)mscale, stream);
        Py_END_ALLOW_THREADS
        if (check_rc(rc, "fa_rope")) goto done;
    }
    if (rk != NULL) {
        out = PyTuple_Pack(2, rq, rk);
    } else {
        Py_INCREF(rq);
        out = rq;
    }
done:
    Py_DECREF(device);
    Py_XDECREF(rq);
    Py_XDECREF(rk);
    return out;
}

/* The pages and index arrays of a paged batch. */
typedef struct {
    Tensor kp, vp, table, len, start;
    long long T, heads, d, num_pages, Hkv, page_size, B, max_pages;
    int code;
} Batch;

static int take_batch(PyObject *const *a, const Tensor *tok, long dev, Batch *b) {
    if (take(a[0], "k_pages", dev, &b->kp) || take(a[1], "v_pages", dev, &b->vp) ||
        take(a[2], "block_table", dev, &b->table) || take(a[3], "kv_len", dev, &b->len) ||
        take(a[4], "q_start", dev, &b->start))
        return -1;
    if (b->kp.obj == NULL || b->vp.obj == NULL || b->table.obj == NULL || b->len.obj == NULL)
        return fail(PyExc_ValueError, "k_pages, v_pages, block_table and kv_len are needed");
    b->code = dtype_code(tok);
    if (b->code < 0) return -1;
    if (tok->dims != 3) return fail(PyExc_ValueError, "tokens must be [T, heads, d]");
    b->T = tok->shape[0];
    b->heads = tok->shape[1];
    b->d = tok->shape[2];
    if (b->kp.dims != 4 || !same_shape(&b->kp, &b->vp) || b->kp.shape[3] != b->d ||
        b->kp.dtype != tok->dtype || b->vp.dtype != tok->dtype)
        return fail(PyExc_ValueError, "k_pages and v_pages must be [num_pages, H_kv, page_size, d] with "
                                      "the dtype of the tokens");
    b->num_pages = b->kp.shape[0];
    b->Hkv = b->kp.shape[1];
    b->page_size = b->kp.shape[2];
    if (b->table.dims != 2 || b->table.dtype != g_i32 || !is_dense(&b->table))
        return fail(PyExc_ValueError, "block_table must be contiguous int32 [B, max_pages]");
    b->B = b->table.shape[0];
    b->max_pages = b->table.shape[1];
    if (check_index(&b->len, b->B, -1) || check_index(&b->start, b->B + 1, -1)) return -1;
    const long long ext[8] = {b->T, b->heads, b->d, b->num_pages, b->Hkv, b->page_size, b->B,
                              b->max_pages};
    return fits(ext, 8);
}

/* paged_append(k, v, k_pages, v_pages, block_table, kv_len, q_start, q, out_q, freq, positions,
 *              interleaved, mscale) */
static PyObject *py_append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Tensor k, v, q, oq, freq, pos;
    Batch b;
    long dev;
    if (count_args(n, 13) || first_device(a[0], "k", &dev) || take(a[0], "k", dev, &k) ||
        take(a[1], "v", dev, &v) || take(a[7], "q", dev, &q) || take(a[8], "out_q", dev, &oq) ||
        take(a[9], "freq", dev, &freq) || take(a[10], "positions", dev, &pos) ||
        take_batch(a + 2, &k, dev, &b))
        return NULL;
    const int inter = PyObject_IsTrue(a[11]);
    const double mscale = PyFloat_AsDouble(a[12]);
    if (inter < 0 || (mscale == -1.0 && PyErr_Occurred())) return NULL;
    if (b.heads != b.Hkv || v.obj == NULL || !same_shape(&k, &v) || v.dtype != k.dtype) {
        fail(PyExc_ValueError, "k and v must be [T, H_kv, d] with the H_kv and dtype of the pages");
        return NULL;
    }
    if (check_index(&pos, b.T, -1)) return NULL;
    if (q.obj != NULL &&
        (q.dims != 3 || q.shape[0] != b.T || q.shape[2] != b.d || q.dtype != k.dtype)) {
        fail(PyExc_ValueError, "q must be [T, H, d] with the dtype of k");
        return NULL;
    }
    if (q.obj == NULL && oq.obj != NULL) {
        fail(PyExc_ValueError, "out_q needs q");
        return NULL;
    }
    const long long rot = freq.obj != NULL ? freq_rot(&freq) : 0;
    const long long H = q.obj != NULL ? q.shape[1] : b.Hkv;
    const long long ext[2] = {H, rot};
    if (rot < 0 || fits(ext, 2)) return NULL;
    PyObject *rq = NULL;
    void *pq = NULL, *stream;
    long long sq[MAX_DIMS] = {8, 8, 1};
    if (q.obj != NULL) {
        PyObject *device = PyObject_GetAttr(q.obj, s_device);
        if (device == NULL) return NULL;
        rq = result(&oq, &q, device, &pq, sq);
        Py_DECREF(device);
        if (rq == NULL) return NULL;
    }
    if (stream_of(dev, &stream)) goto fail;
    {
        const long long st[14] = {q.obj ? q.stride[0] : 8, q.obj ? q.stride[1] : 8, sq[0], sq[1],
                                  k.stride[0], k.stride[1], v.stride[0], v.stride[1],
                                  b.kp.stride[0], b.kp.stride[1], b.kp.stride[2],
                                  b.vp.stride[0], b.vp.stride[1], b.vp.stride[2]};
        int rc;
        Py_BEGIN_ALLOW_THREADS
        rc = g_append(q.ptr, pq, k.ptr, v.ptr, b.kp.ptr, b.vp.ptr, st, b.table.ptr, b.len.ptr,
                      b.start.ptr, pos.ptr, freq.ptr, (int)b.T, (int)b.B, (int)H, (int)b.Hkv,
                      (int)b.d, (int)b.num_pages, (int)b.page_size, (int)b.max_pages, (int)rot,
                      b.code, inter, (float)mscale, stream);
        Py_END_ALLOW_THREADS
        if (check_rc(rc, "fa_paged_append")) goto fail;
    }
    if (rq == NULL) Py_RETURN_NONE;
    return rq;
fail:
    Py_XDECREF(rq);
    return NULL;
}

/* paged_attention(q, k_pages, v_pages, block_table, kv_len, q_start, max_q, scale, causal, out, lse,
 *                 workspace) */
static PyObject *py_attention(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Tensor q, out, lse, ws;
    Batch b;
    long dev;
    if (count_args(n, 12) || first_device(a[0], "q", &dev) || take(a[0], "q", dev, &q) ||
        take(a[9], "out", dev, &out) || take(a[10], "lse", dev, &lse) ||
        take(a[11], "workspace", dev, &ws) || take_batch(a + 1, &q, dev, &b))
        return NULL;
    const int causal = PyObject_IsTrue(a[8]);
    if (causal < 0) return NULL;
    long long max_q = b.start.obj != NULL ? b.T : b.B > 0 && b.T / b.B > 1 ? b.T / b.B : 1;
    if (a[6] != Py_None) {
        max_q = PyLong_AsLongLong(a[6]);
        if (max_q == -1 && PyErr_Occurred()) return NULL;
        if (max_q > b.T) max_q = b.T;
        if (max_q < 0) max_q = 0; /* refused by the library */
    }
    double scale = 1.0 / sqrt((double)(b.d > 0 ? b.d : 1));
    if (a[7] != Py_None) {
        scale = PyFloat_AsDouble(a[7]);
        if (scale == -1.0 && PyErr_Occurred()) return NULL;
    }
    if (lse.obj != NULL && (lse.dtype != g_f32 || lse.dims != 2 || lse.shape[0] != b.T ||
                            lse.shape[1] != b.heads || !is_dense(&lse))) {
        fail(PyExc_ValueError, "lse must be contiguous fp32 [T, H]");
        return NULL;
    }
    if (ws.obj != NULL && !is_dense(&ws)) {
        fail(PyExc_ValueError, "workspace must be contiguous");
        return NULL;
    }
    const size_t need = max_q < 1 ? 0
                                  : g_attn_bytes((int)b.T, (int)b.B, (int)b.heads, (int)b.Hkv, (int)b.d,
                                                 (int)max_q, (int)b.page_size, (int)b.max_pages);
    PyObject *device = PyObject_GetAttr(q.obj, s_device), *ro = NULL, *rl = NULL, *rw = NULL, *res = NULL;
    void *po, *pl = lse.ptr, *pw = ws.ptr, *stream;
    long long so[MAX_DIMS];
    if (device == NULL) return NULL;
    if ((ro = result(&out, &q, device, &po, so)) == NULL) goto done;
    if (lse.obj != NULL) {
        Py_INCREF(lse.obj);
        rl = lse.obj;
    } else {
        const long long shape[2] = {b.T, b.heads};
        if ((rl = new_tensor(shape, 2, g_f32, device, &pl)) == NULL) goto done;
    }
    if (ws.obj != NULL) {
        PyObject *bytes = PyObject_GetAttrString(ws.obj, "nbytes");
        const long long have = bytes ? PyLong_AsLongLong(bytes) : -1;
        Py_XDECREF(bytes);
        if (have < 0) goto done;
        if ((size_t)have < need) {
            fail(PyExc_ValueError, "workspace must be of paged_workspace_bytes() bytes");
            goto done;
        }
    } else if (need > 0) {
        const long long shape[1] = {(long long)need};
        if ((rw = new_tensor(shape, 1, g_u8, device, &pw)) == NULL) goto done;
    }
    if (stream_of(dev, &stream)) goto done;
    {
        const long long st[10] = {q.stride[0], q.stride[1], so[0], so[1], b.kp.stride[0],
                                  b.kp.stride[1], b.kp.stride[2], b.vp.stride[0], b.vp.stride[1],
                                  b.vp.stride[2]};
        int rc;
        Py_BEGIN_ALLOW_THREADS
        rc = g_attn(q.ptr, b.kp.ptr, b.vp.ptr, po, pl, st, b.table.ptr, b.len.ptr, b.start.ptr,
                    (int)b.T, (int)b.B, (int)b.heads, (int)b.Hkv, (int)b.d, (int)b.num_pages,
                    (int)b.page_size, (int)b.max_pages, (int)max_q, b.code, (float)scale, causal, pw,
                    need, stream);
        Py_END_ALLOW_THREADS
        if (check_rc(rc, "fa_paged_attn")) goto done;
    }
    res = PyTuple_Pack(2, ro, rl);
done:
    Py_DECREF(device);
    Py_XDECREF(ro);
    Py_XDECREF(rl);
    Py_XDECREF(rw);
    return res;
}

/* An integer argument that the library takes as an int. */
static int int_arg(PyObject *obj, const char *name, long long *out) {
    *out = PyLong_AsLongLong(obj);
    if (*out == -1 && PyErr_Occurred()) return -1;
    if (*out < -0x7fffffffLL || *out > 0x7fffffffLL) {
        PyErr_Format(PyExc_ValueError, "%s is out of range", name);
        return -1;
    }
    return 0;
}

/* The caller's workspace of at least `need` bytes, or a new one (*made: to be released). */
static int workspace(const Tensor *given, size_t need, PyObject *like, void **ptr, PyObject **made) {
    *made = NULL;
    if (given->obj != NULL) {
        if (!is_dense(given)) return fail(PyExc_ValueError, "workspace must be contiguous");
        PyObject *bytes = PyObject_GetAttrString(given->obj, "nbytes");
        const long long have = bytes ? PyLong_AsLongLong(bytes) : -1;
        Py_XDECREF(bytes);
        if (have < 0) return -1;
        if ((size_t)have < need)
            return fail(PyExc_ValueError, "workspace is smaller than its *_workspace_bytes()");
        *ptr = given->ptr;
        return 0;
    }
    *ptr = NULL;
    if (need == 0) return 0;
    const long long shape[1] = {(long long)need};
    PyObject *device = PyObject_GetAttr(like, s_device);
    if (device == NULL) return -1;
    *made = new_tensor(shape, 1, g_u8, device, ptr);
    Py_DECREF(device);
    return *made == NULL ? -1 : 0;
}

/* A result of the given shape: the caller's, which has to be contiguous, or a new one. */
static PyObject *dense_result(const Tensor *given, PyObject *dtype, const long long *shape, int dims,
                              PyObject *device, void **ptr) {
    if (given->obj == NULL) return new_tensor(shape, dims, dtype, device, ptr);
    int same = given->dtype == dtype && given->dims == dims && is_dense(given);
    for (int i = 0; same && i < dims; ++i) same = given->shape[i] == shape[i];
    if (!same) {
        PyErr_Format(PyExc_ValueError, "%s has the wrong shape or type, or is not contiguous", given->name);
        return NULL;
    }
    *ptr = given->ptr;
    Py_INCREF(given->obj);
    return given->obj;
}

/* block_table [B, max_pages] and refs [num_pages]. */
static int take_tables(PyObject *table, PyObject *refs, long dev, Tensor *t, Tensor *r) {
    if (take(table, "block_table", dev, t) || take(refs, "refs", dev, r)) return -1;
    if (t->dims != 2 || t->dtype != g_i32 || !is_dense(t))
        return fail(PyExc_ValueError, "block_table must be contiguous int32 [B, max_pages]");
    if (r->obj == NULL || r->dims != 1 || r->dtype != g_i32 || !is_dense(r))
        return fail(PyExc_ValueError, "refs must be contiguous int32 [num_pages]");
    const long long ext[3] = {t->shape[0], t->shape[1], r->shape[0]};
    return fits(ext, 3);
}

/* An index array that has to be there. */
static int need_index(const Tensor *t, long long n) {
    if (t->obj == NULL) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous int32 [%lld]", t->name, n);
        return -1;
    }
    return check_index(t, n, -1);
}

/* paged_reserve(block_table, kv_len, refs, page_size, q_start, tokens, copies, workspace) */
static PyObject *py_reserve(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Tensor table, refs, len, start, copies, ws;
    long dev;
    long long page, T;
    if (count_args(n, 8) || first_device(a[0], "block_table", &dev)) return NULL;
    LEAVE_IF_AWAY(dev);
    if (take_tables(a[0], a[2], dev, &table, &refs) || take(a[1], "kv_len", dev, &len) ||
        take(a[4], "q_start", dev, &start) || take(a[6], "copies", dev, &copies) || take(a[7], "workspace", dev, &ws) ||
        int_arg(a[3], "page_size", &page))
        return NULL;
    const long long B = table.shape[0];
    if (need_index(&len, B) || check_index(&start, B + 1, -1)) return NULL;
    if (a[5] != Py_None) {
        if (int_arg(a[5], "tokens", &T)) return NULL;
    } else if (start.obj != NULL) {
        fail(PyExc_ValueError, "q_start needs tokens, the number of the batch's tokens");
        return NULL;
    } else {
        T = B;
    }
    PyObject *device = PyObject_GetAttr(table.obj, s_device), *rc = NULL, *rw = NULL;
    void *pc, *pw, *stream;
    if (device == NULL) return NULL;
    const long long shape[2] = {3, B};
    rc = dense_result(&copies, g_i32, shape, 2, device, &pc);
    Py_DECREF(device);
    if (rc == NULL) return NULL;
    const size_t need = T < 1 || page < 1 ? 0 : g_reserve_bytes((int)T, (int)B, (int)refs.shape[0], (int)page);
    if (workspace(&ws, need, table.obj, &pw, &rw) || stream_of(dev, &stream)) goto fail;
    {
        int code;
        Py_BEGIN_ALLOW_THREADS
        code = g_reserve(table.ptr, len.ptr, start.ptr, refs.ptr, pc, (int)T, (int)B, (int)refs.shape[0],
                         (int)page, (int)table.shape[1], pw, need, stream);
        Py_END_ALLOW_THREADS
        if (check_rc(code, "fa_paged_reserve")) goto fail;
    }
    Py_XDECREF(rw);
    return rc;
fail:
    Py_XDECREF(rc);
    Py_XDECREF(rw);
    return NULL;
}

/* paged_fork(block_table, parents, refs, kv_len) */
static PyObject *py_fork(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Tensor table, refs, parents, len;
    long dev;
    void *stream;
    if (count_args(n, 4) || first_device(a[0], "block_table", &dev)) return NULL;
    LEAVE_IF_AWAY(dev);
    if (take_tables(a[0], a[2], dev, &table, &refs) || take(a[1], "parents", dev, &parents) ||
        take(a[3], "kv_len", dev, &len) || check_index(&len, table.shape[0], -1))
        return NULL;
    /* [B], or the [requests, beams] of a selection */
    if (parents.obj == NULL || parents.dtype != g_i32 || !is_dense(&parents) || parents.dims < 1 ||
        parents.dims > 2 || parents.shape[0] * (parents.dims == 2 ? parents.shape[1] : 1) != table.shape[0]) {
        PyErr_Format(PyExc_ValueError, "parents must be contiguous int32 of %lld values", table.shape[0]);
        return NULL;
    }
    if (stream_of(dev, &stream)) return NULL;
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = g_fork(table.ptr, len.ptr, parents.ptr, refs.ptr, (int)table.shape[0], (int)refs.shape[0],
                  (int)table.shape[1], stream);
    Py_END_ALLOW_THREADS
    if (check_rc(code, "fa_paged_fork")) return NULL;
    Py_RETURN_NONE;
}

/* paged_free(block_table, keep_len, refs, page_size) */
static PyObject *py_free(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Tensor table, refs, keep;
    long dev;
    long long page;
    void *stream;
    if (count_args(n, 4) || first_device(a[0], "block_table", &dev)) return NULL;
    LEAVE_IF_AWAY(dev);
    if (take_tables(a[0], a[2], dev, &table, &refs) || take(a[1], "keep_len", dev, &keep) ||
        need_index(&keep, table.shape[0]) ||
        int_arg(a[3], "page_size", &page) || stream_of(dev, &stream))
        return NULL;
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = g_free(table.ptr, keep.ptr, refs.ptr, (int)table.shape[0], (int)refs.shape[0], (int)page,
                  (int)table.shape[1], stream);
    Py_END_ALLOW_THREADS
    if (check_rc(code, "fa_paged_free")) return NULL;
    Py_RETURN_NONE;
}

/* paged_compact(block_table, refs, moves, count) */
static PyObject *py_compact(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Tensor table, refs, moves, count;
    long dev;
    if (count_args(n, 4) || first_device(a[0], "block_table", &dev)) return NULL;
    LEAVE_IF_AWAY(dev);
    if (take_tables(a[0], a[1], dev, &table, &refs) || take(a[2], "moves", dev, &moves) ||
        take(a[3], "count", dev, &count))
        return NULL;
    const long long pages = refs.shape[0], one[1] = {1};
    long long shape[2] = {2, pages > 1 ? pages / 2 : 1};
    if (moves.obj != NULL && moves.dims == 2 && moves.shape[1] > shape[1]) shape[1] = moves.shape[1];
    PyObject *device = PyObject_GetAttr(table.obj, s_device), *rm = NULL, *rc = NULL, *out = NULL;
    void *pm, *pc, *stream;
    if (device == NULL) return NULL;
    if ((rm = dense_result(&moves, g_i32, shape, 2, device, &pm)) == NULL ||
        (rc = dense_result(&count, g_i32, one, 1, device, &pc)) == NULL || stream_of(dev, &stream))
        goto done;
    {
        int code;
        Py_BEGIN_ALLOW_THREADS
        code = g_compact(table.ptr, refs.ptr, pm, (int *)pm + shape[1], pc, (int)table.shape[0], (int)pages,
                         (int)table.shape[1], stream);
        Py_END_ALLOW_THREADS
        if (check_rc(code, "fa_paged_compact")) goto done;
    }
    out = PyTuple_Pack(2, rm, rc);
done:
    Py_DECREF(device);
    Py_XDECREF(rm);
    Py_XDECREF(rc);
    return out;
}

/* paged_copy(k_pages, v_pages, src, dst, rows, count) */
static PyObject *py_copy(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Tensor k, v, src, dst, rows, count;
    long dev;
    void *stream;
    if (count_args(n, 6) || first_device(a[0], "k_pages", &dev)) return NULL;
    LEAVE_IF_AWAY(dev);
    if (take(a[0], "k_pages", dev, &k) || take(a[1], "v_pages", dev, &v) || take(a[2], "src", dev, &src) ||
        take(a[3], "dst", dev, &dst) || take(a[4], "rows", dev, &rows) || take(a[5], "count", dev, &count))
        return NULL;
    if (v.obj == NULL || (k.dims != 4 && k.dims != 5) || !same_shape(&k, &v) || k.dtype != v.dtype) {
        fail(PyExc_ValueError, "k_pages and v_pages must be [num_pages, H_kv, page_size, d] or [L, num_pages, "
                               "H_kv, page_size, d] of one type");
        return NULL;
    }
    if (dtype_code(&k) < 0) return NULL;
    if (src.obj == NULL || src.dims != 1) {
        fail(PyExc_ValueError, "src must be contiguous int32 [n]");
        return NULL;
    }
    if (need_index(&src, src.shape[0]) || need_index(&dst, src.shape[0]) ||
        check_index(&rows, src.shape[0], -1) || check_index(&count, 1, -1))
        return NULL;
    const int at = k.dims - 4; /* the axis of pages */
    const long long L = at ? k.shape[0] : 1;
    const long long ext[6] = {src.shape[0], L, k.shape[at + 1], k.shape[at + 3], k.shape[at],
                              k.shape[at + 2]};
    if (fits(ext, 6) || stream_of(dev, &stream)) return NULL;
    const long long st[8] = {at ? k.stride[0] : 8, k.stride[at], k.stride[at + 1], k.stride[at + 2],
                             at ? v.stride[0] : 8, v.stride[at], v.stride[at + 1], v.stride[at + 2]};
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = g_copy(k.ptr, v.ptr, st, src.ptr, dst.ptr, rows.ptr, count.ptr, (int)ext[0], (int)ext[1],
                  (int)ext[2], (int)ext[3], (int)ext[4], (int)ext[5], stream);
    Py_END_ALLOW_THREADS
    if (check_rc(code, "fa_paged_copy")) return NULL;
    Py_RETURN_NONE;
}

/* beam_select(logits, scores, k, finished, end_token, out_scores, out_parents, out_tokens, out_finished,
 *             workspace) */
static PyObject *py_beam(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Tensor x, scores, fin, out[4], ws;
    static const char *names[4] = {"out_scores", "out_parents", "out_tokens", "out_finished"};
    long dev;
    if (count_args(n, 10) || first_device(a[0], "logits", &dev)) return NULL;
    LEAVE_IF_AWAY(dev);
    if (take(a[0], "logits", dev, &x) || take(a[1], "scores", dev, &scores) || take(a[3], "finished", dev, &fin) ||
        take(a[9], "workspace", dev, &ws))
        return NULL;
    for (int i = 0; i < 4; ++i)
        if (take(a[5 + i], names[i], dev, &out[i])) return NULL;
    if (x.dims != 3) {
        fail(PyExc_ValueError, "logits must be [B, W, V]");
        return NULL;
    }
    int code = x.dtype == g_f32 ? FA_FP32 : x.dtype == g_bf16 ? FA_BF16 : x.dtype == g_fp16 ? FA_FP16 : -1;
    if (code < 0) {
        PyErr_Format(PyExc_TypeError,
                     "unsupported dtype %R: use torch.bfloat16, torch.float16 or torch.float32", x.dtype);
        return NULL;
    }
    const long long B = x.shape[0], W = x.shape[1], V = x.shape[2];
    const Tensor *small[2] = {&scores, &fin};
    for (int i = 0; i < 2; ++i) {
        const Tensor *s = small[i];
        if (i == 1 && s->obj == NULL) continue;
        if (s->obj == NULL || s->dims != 2 || s->shape[0] != B || s->shape[1] != W || !is_dense(s) ||
            s->dtype != (i ? g_u8 : g_f32)) {
            fail(PyExc_ValueError, i ? "finished must be contiguous uint8 [B, W]"
                                     : "scores must be contiguous fp32 [B, W]");
            return NULL;
        }
    }
    long long K = W, end = -1;
    if ((a[2] != Py_None && int_arg(a[2], "k", &K)) || (a[4] != Py_None && int_arg(a[4], "end_token", &end)))
        return NULL;
    if (K < 1) {
        fail(PyExc_ValueError, "k must be at least 1");
        return NULL;
    }
    const long long ext[4] = {B, W, V, K}, shape[2] = {B, K};
    if (fits(ext, 4)) return NULL;
    PyObject *types[4] = {g_f32, g_i32, g_i32, g_u8}, *made[4] = {NULL, NULL, NULL, NULL}, *rw = NULL;
    PyObject *device = PyObject_GetAttr(x.obj, s_device), *res = NULL;
    void *ptr[4], *pw, *stream;
    if (device == NULL) return NULL;
    for (int i = 0; i < 4; ++i)
        if ((made[i] = dense_result(&out[i], types[i], shape, 2, device, &ptr[i])) == NULL) goto done;
    const size_t need = g_beam_bytes((int)B, (int)W, (int)V, (int)K);
    if (workspace(&ws, need, x.obj, &pw, &rw) || stream_of(dev, &stream)) goto done;
    {
        const long long st[2] = {x.stride[0], x.stride[1]};
        Py_BEGIN_ALLOW_THREADS
        code = g_beam(x.ptr, st, scores.ptr, fin.ptr, ptr[0], ptr[1], ptr[2], ptr[3], (int)B, (int)W, (int)V,
                      (int)K, code, (int)end, pw, need, stream);
        Py_END_ALLOW_THREADS
        if (check_rc(code, "fa_beam_select")) goto done;
    }
    res = PyTuple_Pack(4, made[0], made[1], made[2], made[3]);
done:
    Py_DECREF(device);
    for (int i = 0; i < 4; ++i) Py_XDECREF(made[i]);
    Py_XDECREF(rw);
    return res;
}

/* setup(addresses of the entry points in the order below, torch.empty, raw stream of a device, current device,
 *       bfloat16, float16, int32, int64, float32, uint8, error class) */
static PyObject *py_setup(PyObject *self, PyObject *args) {
    (void)self;
    unsigned long long f[12];
    PyObject *o[10];
    if (!PyArg_ParseTuple(args, "(KKKKKKKKKKKK)OOOOOOOOOO", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6],
                          &f[7], &f[8], &f[9], &f[10], &f[11], &o[0], &o[1], &o[2], &o[3], &o[4],
                          &o[5], &o[6], &o[7], &o[8], &o[9]))
        return NULL;
    g_rope = (rope_fn)(uintptr_t)f[0];
    g_append = (append_fn)(uintptr_t)f[1];
    g_attn = (attn_fn)(uintptr_t)f[2];
    g_attn_bytes = (attn_bytes_fn)(uintptr_t)f[3];
    g_reserve = (reserve_fn)(uintptr_t)f[4];
    g_reserve_bytes = (reserve_bytes_fn)(uintptr_t)f[5];
    g_fork = (fork_fn)(uintptr_t)f[6];
    g_free = (free_fn)(uintptr_t)f[7];
    g_compact = (compact_fn)(uintptr_t)f[8];
    g_copy = (copy_fn)(uintptr_t)f[9];
    g_beam = (beam_fn)(uintptr_t)f[10];
    g_beam_bytes = (beam_bytes_fn)(uintptr_t)f[11];
    PyObject **slots[10] = {&g_empty, &g_stream, &g_current, &g_bf16, &g_fp16, &g_i32, &g_i64, &g_f32, &g_u8, &g_error};
    for (int i = 0; i < 10; ++i) {
        Py_INCREF(o[i]);
        Py_XSETREF(*slots[i], o[i]);
    }
    Py_RETURN_NONE;
}

static PyMethodDef kMethods[] = {
    {"setup", py_setup, METH_VARARGS, NULL},
    {"rope", (PyCFunction)(void (*)(void))py_rope, METH_FASTCALL, NULL},
    {"paged_append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, NULL},
    {"paged_attention", (PyCFunction)(void (*)(void))py_attention, METH_FASTCALL, NULL},
    {"paged_reserve", (PyCFunction)(void (*)(void))py_reserve, METH_FASTCALL, NULL},
    {"paged_fork", (PyCFunction)(void (*)(void))py_fork, METH_FASTCALL, NULL},
    {"paged_free", (PyCFunction)(void (*)(void))py_free, METH_FASTCALL, NULL},
    {"paged_compact", (PyCFunction)(void (*)(void))py_compact, METH_FASTCALL, NULL},
    {"paged_copy", (PyCFunction)(void (*)(void))py_copy, METH_FASTCALL, NULL},
    {"beam_select", (PyCFunction)(void (*)(void))py_beam, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, kMethods,
                                     NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
    s_get_device = PyUnicode_InternFromString("get_device");
    s_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_device = PyUnicode_InternFromString("device");
    s_kwnames = Py_BuildValue("(ss)", "dtype", "device");
    if (!s_get_device || !s_contiguous || !s_dtype || !s_shape || !s_stride || !s_data_ptr || !s_device || !s_kwnames)
        return NULL;
    return PyModule_Create(&kModule);
}
