/* calls.c -- Python's way into the four calls around the block, argument marshalling only.
 *
 * A single token's call is a few microseconds on the device, and forming its sixteen arguments
 * through ctypes took 3.0 us of the host's time, half of what the whole call took; here it
 * takes 1.0.  The library's functions are handed over as addresses once it is loaded, so that
 * this module links against nothing.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "hs2.h"

typedef hs2_status (*rope_fn)(const hs2_rope_desc*, const void*, const void*, const void*, const float*, const float*,
                              const double*, const int32_t*, const int32_t*, const int32_t*, void*, void*, void*, float*,
                              float*, hs2_stream_t);
typedef hs2_status (*window_fn)(const hs2_attn_desc*, int32_t, const void*, const void*, const void*, const float*,
                                const float*, const int32_t*, const int32_t*, void*, float*, void*, size_t, hs2_stream_t);
typedef hs2_status (*accum_fn)(const hs2_attn_desc*, const void*, const void*, const float*, const float*, const int32_t*,
                               const int32_t*, float, const float*, float*, void*, size_t, hs2_stream_t);
typedef hs2_status (*evict_fn)(const hs2_evict_desc*, const int32_t*, const float*, const void*, const void*, const float*,
                               const float*, void*, void*, float*, float*, float*, int32_t*, int32_t*, hs2_stream_t);

static rope_fn rope;
static window_fn window;
static accum_fn accum;
static evict_fn evict;
static PyObject* name_data_ptr;

/* The addresses of n tensors; None is NULL.  0: an error is set. */
static int addresses(PyObject* const* a, int n, void** p) {
    for (int i = 0; i < n; ++i) {
        p[i] = NULL;
        if (a[i] == Py_None) continue;
        PyObject* x = PyObject_CallMethodNoArgs(a[i], name_data_ptr);
        if (!x) return 0;
        p[i] = PyLong_AsVoidPtr(x);
        Py_DECREF(x);
        if (!p[i] && PyErr_Occurred()) return 0;
    }
    return 1;
}

/* A description (a ctypes structure of this size). */
static int description(PyObject* o, Py_buffer* view, size_t bytes) {
    if (PyObject_GetBuffer(o, view, PyBUF_SIMPLE)) return 0;
    if ((size_t)view->len == bytes) return 1;
    PyBuffer_Release(view);
    PyErr_SetString(PyExc_TypeError, "not this call's description");
    return 0;
}

static int count(Py_ssize_t n, Py_ssize_t want, const void* fn) {
    if (!fn) PyErr_SetString(PyExc_RuntimeError, "the library is not loaded");
    else if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
    return fn && n == want;
}

static int whole(PyObject* o, int32_t* x) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) return 0;
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "not a 32-bit integer");
        return 0;
    }
    *x = (int32_t)v;
    return 1;
}

static int size(PyObject* o, size_t* x) {
    *x = PyLong_AsSize_t(o);
    return *x != (size_t)-1 || !PyErr_Occurred();
}

static int handle(PyObject* o, hs2_stream_t* x) {
    *x = (hs2_stream_t)PyLong_AsVoidPtr(o);
    return *x || !PyErr_Occurred();
}

/* bind(rope, window, accum, evict): the functions' addresses */
static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void* p[4];
    (void)self;
    if (n != 4) return PyErr_Format(PyExc_TypeError, "four addresses, not %zd", n);
    for (int i = 0; i < 4; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is zero");
            return NULL;
        }
    rope = (rope_fn)p[0];
    window = (window_fn)p[1];
    accum = (accum_fn)p[2];
    evict = (evict_fn)p[3];
    Py_RETURN_NONE;
}

/* desc, 14 tensors, stream */
static PyObject* qk_norm_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void* p[14];
    hs2_stream_t st;
    Py_buffer d;
    hs2_status s;
    (void)self;
    if (!count(n, 16, (const void*)rope) || !addresses(a + 1, 14, p) || !handle(a[15], &st)) return NULL;
    if (!description(a[0], &d, sizeof(hs2_rope_desc))) return NULL;
    Py_BEGIN_ALLOW_THREADS;
    s = rope(d.buf, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11], p[12], p[13], st);
    Py_END_ALLOW_THREADS;
    PyBuffer_Release(&d);
    return PyLong_FromLong(s);
}

/* desc, sinks, 10 tensors (the last the workspace), its bytes, stream */
static PyObject* window_attn(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void* p[10];
    int32_t sinks;
    size_t bytes;
    hs2_stream_t st;
    Py_buffer d;
    hs2_status s;
    (void)self;
    if (!count(n, 14, (const void*)window) || !whole(a[1], &sinks) || !addresses(a + 2, 10, p) || !size(a[12], &bytes) ||
        !handle(a[13], &st))
        return NULL;
    if (!description(a[0], &d, sizeof(hs2_attn_desc))) return NULL;
    Py_BEGIN_ALLOW_THREADS;
    s = window(d.buf, sinks, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], bytes, st);
    Py_END_ALLOW_THREADS;
    PyBuffer_Release(&d);
    return PyLong_FromLong(s);
}

/* desc, 6 tensors, decay, 3 tensors (the last the workspace), its bytes, stream */
static PyObject* weight_accum(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void* p[9];
    size_t bytes;
    hs2_stream_t st;
    Py_buffer d;
    hs2_status s;
    (void)self;
    if (!count(n, 13, (const void*)accum) || !addresses(a + 1, 6, p) || !addresses(a + 8, 3, p + 6) || !size(a[11], &bytes) ||
        !handle(a[12], &st))
        return NULL;
    const double decay = PyFloat_AsDouble(a[7]);
    if (decay == -1.0 && PyErr_Occurred()) return NULL;
    if (!description(a[0], &d, sizeof(hs2_attn_desc))) return NULL;
    Py_BEGIN_ALLOW_THREADS;
    s = accum(d.buf, p[0], p[1], p[2], p[3], p[4], p[5], (float)decay, p[6], p[7], p[8], bytes, st);
    Py_END_ALLOW_THREADS;
    PyBuffer_Release(&d);
    return PyLong_FromLong(s);
}

/* desc, 13 tensors, stream */
static PyObject* kv_evict(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void* p[13];
    hs2_stream_t st;
    Py_buffer d;
    hs2_status s;
    (void)self;
    if (!count(n, 15, (const void*)evict) || !addresses(a + 1, 13, p) || !handle(a[14], &st)) return NULL;
    if (!description(a[0], &d, sizeof(hs2_evict_desc))) return NULL;
    Py_BEGIN_ALLOW_THREADS;
    s = evict(d.buf, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11], p[12], st);
    Py_END_ALLOW_THREADS;
    PyBuffer_Release(&d);
    return PyLong_FromLong(s);
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST(bind), FAST(qk_norm_rope), FAST(window_attn), FAST(weight_accum), FAST(kv_evict),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void) {
    name_data_ptr = PyUnicode_InternFromString("data_ptr");
    return name_data_ptr ? PyModule_Create(&module) : NULL;
}
