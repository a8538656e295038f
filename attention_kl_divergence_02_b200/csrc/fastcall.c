/*
 * fastcall.c -- the everyday case of the paged-cache calls of binding.py, as a CPython extension.
 *
 * These calls are made once per token and layer, and the interpreter's share of one (a dozen attribute
 * checks, fifteen converted arguments) is as long as a small kernel: a paged_attn call takes the host 8.6 us
 * with this and 11.7 without, a paged_kl 10.6 and 15.  Each function here checks the same as its namesake in binding.py and makes the same library
 * call; where anything is out of the ordinary (another device or stream, no workspace, tensors given
 * for the outputs, a check that fails) it returns NotImplemented and binding.py goes on, with its
 * own checks and messages.  It keeps nothing between calls but what setup() gave it.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "streamkl.h"

static PyObject *s_dtype, *s_shape, *s_is_contiguous, *s_get_device, *s_data_ptr, *s_numel, *s_new_empty, *s_unbind;
static PyObject *g_bf16, *g_int32, *g_fp32, *g_empty_like, *g_get_device, *g_raw_stream, *g_zero;

typedef int (*attn_fn)(const streamkl_cache*, const uint16_t*, const int*, int, const int*, int, int, int, float, int, uint16_t*,
                       float*, void*, size_t, void*);
typedef int (*kl_fn)(const streamkl_cache*, const uint16_t*, const streamkl_cache*, const uint16_t*, const int*, int, const int*,
                     int, int, int, float, int, float*, float*, float*, void*, size_t, void*);
typedef int (*append_fn)(const streamkl_cache*, const uint16_t*, const uint16_t*, const int*, int, const int*, const int*, int, int,
                         void*);
typedef int (*gather_fn)(const streamkl_cache*, const int*, int, const int*, const int*, int, int, uint16_t*, uint16_t*, void*);
static attn_fn g_attn;
static kl_fn g_kl;
static append_fn g_append;
static gather_fn g_gather;

/* setup(bf16, int32, fp32, empty_like, get_device, raw_stream, addresses of attn, kl, append, gather) */
static PyObject* setup(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    if (n != 10) {
        PyErr_SetString(PyExc_TypeError, "setup takes 10 arguments");
        return NULL;
    }
    void *attn = PyLong_AsVoidPtr(a[6]), *kl = PyLong_AsVoidPtr(a[7]);
    void *append = PyLong_AsVoidPtr(a[8]), *gather = PyLong_AsVoidPtr(a[9]);
    if (PyErr_Occurred()) return NULL;
    PyObject** to[6] = {&g_bf16, &g_int32, &g_fp32, &g_empty_like, &g_get_device, &g_raw_stream};
    for (int i = 0; i < 6; ++i) {
        Py_INCREF(a[i]);
        Py_XSETREF(*to[i], a[i]);
    }
    g_attn = (attn_fn)attn;
    g_kl = (kl_fn)kl;
    g_append = (append_fn)append;
    g_gather = (gather_fn)gather;
    Py_RETURN_NONE;
}

/* An integer that a method without arguments returns; -1 with an exception set on failure. */
static long long call_int(PyObject* o, PyObject* name) {
    PyObject* r = PyObject_CallMethodNoArgs(o, name);
    if (!r) return -1;
    const long long v = PyLong_AsLongLong(r);
    Py_DECREF(r);
    return v;
}

/* Whether t is a contiguous tensor of this type on this device; -1 on an exception. */
static int is_plain(PyObject* t, PyObject* dtype, long long device) {
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    if (!d) return -1;
    Py_DECREF(d);
    if (d != dtype) return 0;
    const long long at = call_int(t, s_get_device);
    if (at == -1 && PyErr_Occurred()) return -1;
    if (at != device) return 0;
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!c) return -1;
    Py_DECREF(c);
    return c == Py_True;
}

/* The sizes of t, which has `n` dimensions: 1, 0 if it has not, -1 on an exception. */
static int sizes(PyObject* t, int n, long long* to) {
    PyObject* s = PyObject_GetAttr(t, s_shape);
    if (!s) return -1;
    int rc = PyTuple_Check(s) && PyTuple_GET_SIZE(s) == n;
    for (int i = 0; rc == 1 && i < n; ++i) {
        to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(s, i));
        if (to[i] == -1 && PyErr_Occurred()) rc = -1;
    }
    Py_DECREF(s);
    return rc;
}

/* data_ptr(); sets *failed on an exception. */
static void* data_ptr(PyObject* t, int* failed) {
    PyObject* r = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!r) {
        *failed = 1;
        return NULL;
    }
    void* p = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    if (!p && PyErr_Occurred()) *failed = 1;
    return p;
}

/* What a failed step does: an exception (an object that is no tensor, say) is dropped too, so that binding.py
 * meets it and words it. */
static PyObject* go_on(void) {
    PyErr_Clear();
    Py_RETURN_NOTIMPLEMENTED;
}

/* The current stream of the device, if that is the current device: 1, else 0. */
static int on_device(PyObject* index, long long device, void** stream) {
    PyObject* now = PyObject_CallNoArgs(g_get_device);
    if (!now) return 0;
    const long long current = PyLong_AsLongLong(now);
    Py_DECREF(now);
    if (current != device || PyErr_Occurred()) return 0;
    PyObject* s = PyObject_CallOneArg(g_raw_stream, index);
    if (!s) return 0;
    *stream = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    return PyErr_Occurred() == NULL;
}

/* int32 [B] on the device: 1 and its address, else 0. */
static int ints(PyObject* t, long long B, long long device, void** to) {
    long long n[1];
    int failed = 0;
    if (sizes(t, 1, n) != 1 || n[0] != B || is_plain(t, g_int32, device) != 1) return 0;
    *to = data_ptr(t, &failed);
    return !failed;
}

/* int32 [B, width] on the device: the width and its address, else 0. */
static int table_width(PyObject* t, long long B, long long device, void** to) {
    long long n[2];
    int failed = 0;
    if (sizes(t, 2, n) != 1 || n[0] != B || n[1] < 1 || n[1] > 0x7fffffff || is_plain(t, g_int32, device) != 1) return 0;
    *to = data_ptr(t, &failed);
    return failed ? 0 : (int)n[1];
}

typedef struct {
    const streamkl_cache* cache;
    long long device, q[4], width, ws_bytes;
    float scale;
    void *stream, *table, *lengths, *ws, *qp;
} common;

/* q, table, lengths, workspace against the cache: 1 if all is ordinary. */
static int check(common* c, PyObject* address, PyObject* index, PyObject* q, PyObject* table, PyObject* lengths, PyObject* scale,
                 PyObject* workspace) {
    c->cache = (const streamkl_cache*)PyLong_AsVoidPtr(address);
    c->device = PyLong_AsLongLong(index);
    if (!c->cache || PyErr_Occurred() || workspace == Py_None) return 0;
    if (sizes(q, 4, c->q) != 1 || is_plain(q, g_bf16, c->device) != 1) return 0;
    for (int i = 0; i < 4; ++i)
        if (c->q[i] < 1 || c->q[i] > 0x7fffffff) return 0;
    if (c->q[3] != c->cache->d || c->q[1] % c->cache->Hkv) return 0;
    c->width = table_width(table, c->q[0], c->device, &c->table);
    if (!c->width || !ints(lengths, c->q[0], c->device, &c->lengths)) return 0;
    if (is_plain(workspace, g_fp32, c->device) != 1) return 0;
    c->ws_bytes = call_int(workspace, s_numel);
    if (c->ws_bytes < 0) return 0;
    c->ws_bytes *= 4;
    c->scale = (float)PyFloat_AsDouble(scale);
    if (PyErr_Occurred() || !on_device(index, c->device, &c->stream)) return 0;
    int failed = 0;
    c->qp = data_ptr(q, &failed);
    c->ws = data_ptr(workspace, &failed);
    return !failed;
}

/* An fp32 tensor [n, B, Hq, NQ] (n = 0: [B, Hq, NQ]) beside the workspace. */
static PyObject* rows_like(PyObject* workspace, const long long* q, int n) {
    PyObject* shape = n ? Py_BuildValue("(iLLL)", n, q[0], q[1], q[2]) : Py_BuildValue("(LLL)", q[0], q[1], q[2]);
    if (!shape) return NULL;
    PyObject* r = PyObject_CallMethodOneArg(workspace, s_new_empty, shape);
    Py_DECREF(shape);
    return r;
}

/* attn(q, cache address, device, table, lengths, scale, causal, workspace): (status, out, lse) or NotImplemented */
static PyObject* attn(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    common c;
    if (n != 8 || !g_attn || !check(&c, a[1], a[2], a[0], a[3], a[4], a[5], a[7])) return go_on();
    const int causal = PyObject_IsTrue(a[6]);
    if (causal < 0 || !c.cache->v) return go_on();
    PyObject* out = PyObject_CallOneArg(g_empty_like, a[0]);
    if (!out) return NULL;
    PyObject* lse = rows_like(a[7], c.q, 0);
    if (!lse) {
        Py_DECREF(out);
        return NULL;
    }
    int failed = 0;
    void *op = data_ptr(out, &failed), *lp = data_ptr(lse, &failed);
    if (failed) {
        Py_DECREF(out);
        Py_DECREF(lse);
        return NULL;
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_attn(c.cache, (const uint16_t*)c.qp, (const int*)c.table, (int)c.width, (const int*)c.lengths, (int)c.q[0], (int)c.q[1],
                (int)c.q[2], c.scale, causal, (uint16_t*)op, (float*)lp, c.ws, (size_t)c.ws_bytes, c.stream);
    Py_END_ALLOW_THREADS
    return Py_BuildValue("(iNN)", rc, out, lse);
}

/* kl(q1, cache1 address, q2, cache2 address, device, table, lengths, scale, causal, workspace):
 * (status, (kl, lse1, lse2)) or NotImplemented */
static PyObject* kl(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    common c;
    long long q2[4];
    if (n != 10 || !g_kl || !check(&c, a[1], a[4], a[0], a[5], a[6], a[7], a[9])) return go_on();
    const streamkl_cache* cache2 = (const streamkl_cache*)PyLong_AsVoidPtr(a[3]);
    if (!cache2 || sizes(a[2], 4, q2) != 1 || is_plain(a[2], g_bf16, c.device) != 1) return go_on();
    for (int i = 0; i < 4; ++i)
        if (q2[i] != c.q[i]) return go_on();
    const int causal = PyObject_IsTrue(a[8]);
    int failed = 0;
    void* q2p = data_ptr(a[2], &failed);
    if (causal < 0 || failed) return go_on();
    PyObject* all = rows_like(a[9], c.q, 3);
    if (!all) return NULL;
    char* p = (char*)data_ptr(all, &failed);
    PyObject* out = failed ? NULL : PyObject_CallMethodOneArg(all, s_unbind, g_zero);
    Py_DECREF(all);
    if (!out) return NULL;
    const long long rows = c.q[0] * c.q[1] * c.q[2] * 4;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_kl(c.cache, (const uint16_t*)c.qp, cache2, (const uint16_t*)q2p, (const int*)c.table, (int)c.width, (const int*)c.lengths,
              (int)c.q[0], (int)c.q[1], (int)c.q[2], c.scale, causal, (float*)p, (float*)(p + rows), (float*)(p + 2 * rows), c.ws,
              (size_t)c.ws_bytes, c.stream);
    Py_END_ALLOW_THREADS
    return Py_BuildValue("(iN)", rc, out);
}

/* move(cache address, device, append, k, v, table, start or None, count or None): status or NotImplemented */
static PyObject* move(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    if (n != 8 || !g_append || !g_gather) return go_on();
    const streamkl_cache* cache = (const streamkl_cache*)PyLong_AsVoidPtr(a[0]);
    const long long device = PyLong_AsLongLong(a[1]);
    const int append = PyObject_IsTrue(a[2]);
    if (!cache || append < 0 || PyErr_Occurred() || !cache->v) return go_on();
    long long k[4], v[4];
    if (sizes(a[3], 4, k) != 1 || is_plain(a[3], g_bf16, device) != 1) return go_on();
    if (sizes(a[4], 4, v) != 1 || is_plain(a[4], g_bf16, device) != 1) return go_on();
    for (int i = 0; i < 4; ++i)
        if (k[i] < 1 || k[i] > 0x7fffffff || k[i] != v[i]) return go_on();
    if (k[1] != cache->Hkv || k[3] != cache->d) return go_on();
    void *table, *start = NULL, *count = NULL, *stream;
    const int width = table_width(a[5], k[0], device, &table);
    if (!width || (a[6] != Py_None && !ints(a[6], k[0], device, &start)) || (a[7] != Py_None && !ints(a[7], k[0], device, &count)))
        return go_on();
    int failed = 0;
    uint16_t *kp = (uint16_t*)data_ptr(a[3], &failed), *vp = (uint16_t*)data_ptr(a[4], &failed);
    if (failed || !on_device(a[1], device, &stream)) return go_on();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = append ? g_append(cache, kp, vp, (const int*)table, width, (const int*)start, (const int*)count, (int)k[0], (int)k[2], stream)
                : g_gather(cache, (const int*)table, width, (const int*)start, (const int*)count, (int)k[0], (int)k[2], kp, vp, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

static PyMethodDef methods[] = {
    {"move", (PyCFunction)(void (*)(void))move, METH_FASTCALL, NULL},
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, NULL},
    {"attn", (PyCFunction)(void (*)(void))attn, METH_FASTCALL, NULL},
    {"kl", (PyCFunction)(void (*)(void))kl, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) {
    static const struct {
        PyObject** to;
        const char* name;
    } names[] = {{&s_dtype, "dtype"}, {&s_shape, "shape"}, {&s_is_contiguous, "is_contiguous"}, {&s_get_device, "get_device"},
                 {&s_data_ptr, "data_ptr"}, {&s_numel, "numel"}, {&s_new_empty, "new_empty"}, {&s_unbind, "unbind"}};
    for (unsigned i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
        if (!(*names[i].to = PyUnicode_InternFromString(names[i].name))) return NULL;
    if (!(g_zero = PyLong_FromLong(0))) return NULL;
    return PyModule_Create(&module);
}
