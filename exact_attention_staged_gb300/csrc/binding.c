/* binding.c - the per-call path of the Python binding for the calls that are short on the GPU (rotary
 * positions and the paged cache): argument checks, result allocation and the call into libfa.so.
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

static rope_fn g_rope;
static append_fn g_append;
static attn_fn g_attn;
static attn_bytes_fn g_attn_bytes;
/* torch.empty, the current raw stream of a device, the dtypes, the error class: set by setup() */
static PyObject *g_empty, *g_stream, *g_bf16, *g_fp16, *g_i32, *g_i64, *g_f32, *g_u8, *g_error;
static PyObject *s_get_device, *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_device, *s_kwnames;

#define MAX_DIMS 4
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
        fail(PyExc_ValueError, "tensors have at most four axes");
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
    if (ints_of(call0(obj, s_stride), t->stride) < 0) return -1;
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
    long long sq[4], sk[4] = {0, 0, 0, 0};
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
    long long sq[4] = {8, 8, 1, 0};
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
    long long so[4];
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

/* setup((fa_rope, fa_paged_append, fa_paged_attn, fa_paged_attn_workspace_bytes addresses), torch.empty,
 *       raw stream of a device, bfloat16, float16, int32, int64, float32, uint8, error class) */
static PyObject *py_setup(PyObject *self, PyObject *args) {
    (void)self;
    unsigned long long rope, append, attn, bytes;
    PyObject *o[9];
    if (!PyArg_ParseTuple(args, "(KKKK)OOOOOOOOO", &rope, &append, &attn, &bytes, &o[0], &o[1], &o[2],
                          &o[3], &o[4], &o[5], &o[6], &o[7], &o[8]))
        return NULL;
    g_rope = (rope_fn)(uintptr_t)rope;
    g_append = (append_fn)(uintptr_t)append;
    g_attn = (attn_fn)(uintptr_t)attn;
    g_attn_bytes = (attn_bytes_fn)(uintptr_t)bytes;
    PyObject **slots[9] = {&g_empty, &g_stream, &g_bf16, &g_fp16, &g_i32, &g_i64, &g_f32, &g_u8, &g_error};
    for (int i = 0; i < 9; ++i) {
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
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, kMethods,
                                     NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
    s_get_device = PyUnicode_InternFromString("get_device");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_device = PyUnicode_InternFromString("device");
    s_kwnames = Py_BuildValue("(ss)", "dtype", "device");
    if (!s_get_device || !s_dtype || !s_shape || !s_stride || !s_data_ptr || !s_device || !s_kwnames)
        return NULL;
    return PyModule_Create(&kModule);
}
