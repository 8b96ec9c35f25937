/*
 * Argument marshalling of the FP8 entry points for Python, in C: the smallest of
 * them run for a few microseconds on the GPU, about as long as checking five
 * tensors and making the call takes through ctypes (4.2 us; 0.7 us here).
 *
 * Only marshalling: tensor -> device pointer, with the same two checks for every
 * tensor (it lives on the given device, and its storage holds the given number of
 * bytes from its first element on), and a call of a libmoe.so entry point, whose
 * arguments are all pointers: structs, buffers, stream. Tensors are looked at
 * through the DLPack C exchange table of their type (one C call per tensor instead
 * of three Python methods: 7 tensors 0.4 us, 1.5 through the methods), subclasses of
 * torch.Tensor other than Parameter through their Python methods; nothing here
 * depends on torch's binary interface. The bytes that each tensor of a call holds
 * are worked out here too (in Python another microsecond). Built without a DLPack
 * header, it looks at every tensor through its methods; marshal_py.py does what
 * this file does where it is not built.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#if __has_include(<ATen/dlpack.h>)
#include <ATen/dlpack.h>
#endif
#if defined(DLPACK_MAJOR_VERSION) && (DLPACK_MAJOR_VERSION > 1 || DLPACK_MINOR_VERSION >= 3)
#define EXCHANGE_TABLE 1
#endif

#include "moe.h"

enum { kMaxStructs = 4, kMaxBufs = 8 };

static PyObject *s_get_device, *s_nbytes, *s_data_ptr, *s_storage, *s_offset, *s_itemsize, *s_contiguous;

#ifdef EXCHANGE_TABLE
static const DLPackExchangeAPI *s_api;  /* of the types below, once bound */
static PyObject *s_types[2];
#endif

/* obj.name() (or the attribute itself when !call) as an integer; -1 with an exception set on failure. */
static long long number(PyObject *obj, PyObject *name, int call) {
    PyObject *r = call ? PyObject_CallMethodNoArgs(obj, name) : PyObject_GetAttr(obj, name);
    if (!r) return -1;
    const long long v = PyLong_AsLongLong(r);
    Py_DECREF(r);
    return v;
}

/* Bytes from x's first element to the end of its storage. */
static long long bytes_behind(PyObject *x) {
    PyObject *st = PyObject_CallMethodNoArgs(x, s_storage);
    if (!st) return -1;
    const long long all = number(st, s_nbytes, 1);
    Py_DECREF(st);
    if (all < 0) return -1;
    const long long off = number(x, s_offset, 1);
    if (off < 0 && PyErr_Occurred()) return -1;
    const long long size = number(x, s_itemsize, 1);
    if (size < 0) return -1;
    return all - off * size;
}

#ifdef EXCHANGE_TABLE
static int bound(PyObject *x) {
    return s_api && ((PyObject *)Py_TYPE(x) == s_types[0] || (PyObject *)Py_TYPE(x) == s_types[1]);
}

/* A tensor's device (-1: host), bytes from its first element to the end of its last, and address, from the
 * exchange table; 0 when the table does not describe it. */
static int describe(PyObject *x, long *dev, long long *bytes, void **p) {
    DLTensor t;
    if (s_api->dltensor_from_py_object_no_sync(x, &t) != 0) {
        PyErr_Clear();
        return 0;
    }
    if (t.device.device_type != kDLCUDA && t.device.device_type != kDLCPU) return 0;
    *dev = t.device.device_type == kDLCUDA ? t.device.device_id : -1;
    long long last = 0, dense = 1;
    int empty = 0;
    for (int i = t.ndim - 1; i >= 0; --i) {
        if (t.shape[i] == 0) empty = 1;
        last += (t.shape[i] - 1) * (t.strides ? t.strides[i] : dense);
        dense *= t.shape[i];
    }
    *bytes = empty ? 0 : (last + 1) * ((t.dtype.bits * t.dtype.lanes + 7) / 8);
    *p = (char *)t.data + t.byte_offset;
    return 1;
}
#else
static int bound(PyObject *x) { (void)x; return 0; }
static int describe(PyObject *x, long *dev, long long *bytes, void **p) {
    (void)x; (void)dev; (void)bytes; (void)p;
    return 0;
}
#endif

/* The pointers of the n objects in tuple `t`, each holding needs[i] bytes on device dev: None -> NULL, an int is
 * an address and passes unchecked. 0, or 2 i + 1 (tensor i on another device), 2 i + 2 (too small), or -1 with
 * an exception set. */
static long take(PyObject *t, int n, const long long *needs, long dev, void **out) {
    if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != n) {
        PyErr_Format(PyExc_TypeError, "expected a tuple of %d tensors", n);
        return -1;
    }
    for (int i = 0; i < n; ++i) {
        PyObject *x = PyTuple_GET_ITEM(t, i);
        if (x == Py_None) {
            out[i] = NULL;
            continue;
        }
        if (PyLong_Check(x)) {
            out[i] = PyLong_AsVoidPtr(x);
            if (!out[i] && PyErr_Occurred()) return -1;
            continue;
        }
        const long long need = needs[i];
        if (bound(x)) {
            long d;
            long long has;
            if (describe(x, &d, &has, &out[i])) {
                if (d != dev) return 2 * i + 1;
                if (has < need) {  /* part of a larger buffer: what lies behind it counts */
                    has = bytes_behind(x);
                    if (has < 0 && PyErr_Occurred()) return -1;
                }
                if (has < need || (need > 0 && !out[i])) return 2 * i + 2;
                continue;
            }
        }
        const long long d = number(x, s_get_device, 1);
        if (d == -1 && PyErr_Occurred()) return -1;
        if (d != dev) return 2 * i + 1;
        /* nbytes counts elements: what memory they take is known for a contiguous tensor only (an expanded one
         * may have many elements and a few bytes) */
        const long long dense = number(x, s_contiguous, 1);
        if (dense < 0) return -1;
        const long long has = dense ? number(x, s_nbytes, 0) : 0;
        if (has < 0) return -1;
        if (!dense || has < need) {
            const long long behind = bytes_behind(x);
            if (behind < 0 && PyErr_Occurred()) return -1;
            if (behind < need) return 2 * i + 2;
        }
        PyObject *p = PyObject_CallMethodNoArgs(x, s_data_ptr);
        if (!p) return -1;
        out[i] = PyLong_AsVoidPtr(p);
        Py_DECREF(p);
        if (!out[i] && PyErr_Occurred()) return -1;
        if (need > 0 && !out[i]) return 2 * i + 2;  /* memory that was given back */
    }
    return 0;
}

/* A tuple of at most kMaxBufs byte counts; their number, or -1 with an exception set. */
static int read_needs(PyObject *t, long long *needs) {
    if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) > kMaxBufs) {
        PyErr_Format(PyExc_TypeError, "needs: a tuple of at most %d byte counts", kMaxBufs);
        return -1;
    }
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(t); ++i) {
        needs[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
        if (needs[i] == -1 && PyErr_Occurred()) return -1;
    }
    return (int)PyTuple_GET_SIZE(t);
}

/* Bytes of a buffer of `rows` rows, `ld` elements of `size` bytes apart and `cols` long; of a table of one float
 * per block. Beyond 63 bits: the largest, which no tensor holds. */
static long long clamp(__int128 v) { return v > INT64_MAX ? INT64_MAX : v < -1 ? -1 : (long long)v; }
static long long rows_of(long long rows, long long cols, long long ld, int size) {
    return clamp(((__int128)(rows - 1) * ld + cols) * size);
}
static long long blocks(long long n) { return (n + 127) / 128; }
static long long table(long long rows, long long cols) { return clamp((__int128)4 * rows * blocks(cols)); }
static int size_of(int32_t type) { return type == MOE_T_BF16 ? 2 : 4; }

enum { kNorm, kQuantize, kGemm, kFfn, kOps };
enum { kFfnWeights = 6 };

/* What the buffers of an entry point hold for these structs (and the FFN's weights); the number of buffers, or -1
 * with an exception set when a struct is not the one it takes. */
static int sizes(long op, void *const *p, const Py_ssize_t *len, int n, long long *need, long long *weights) {
    static const size_t desc_size[kOps] = {sizeof(moe_norm_desc), sizeof(moe_fp8_quant_desc), sizeof(moe_fp8_gemm_desc),
                                           sizeof(moe_fp8_ffn_desc)};
    if (op < 0 || op >= kOps || n != (op == kFfn ? 2 : 1) || !p[0] || (size_t)len[0] != desc_size[op] ||
        (op == kFfn && p[1] && (size_t)len[1] != sizeof(moe_fp8_ffn_weights))) {
        PyErr_SetString(PyExc_TypeError, "not the descriptor of this entry point");
        return -1;
    }
    if (op == kNorm) {
        const moe_norm_desc *d = p[0];
        need[0] = rows_of(d->T, d->d, d->ldx, size_of(d->x_type));
        need[1] = need[3] = rows_of(d->T, d->d, d->ldr, size_of(d->res_type));
        need[2] = rows_of(1, d->d, 0, size_of(d->w_type));
        need[4] = rows_of(d->T, d->d, d->ldy, 2);
        need[5] = rows_of(d->T, d->d, d->ldq, 1);
        need[6] = table(d->T, d->d);
        return 7;
    }
    if (op == kQuantize) {
        const moe_fp8_quant_desc *d = p[0];
        need[0] = rows_of(d->rows, d->cols, d->ldv, size_of(d->v_type));
        need[1] = rows_of(d->rows, d->cols, d->ldq, 1);
        need[2] = table(d->block_rows == 1 ? d->rows : blocks(d->rows), d->cols);
        return 3;
    }
    if (op == kGemm) {
        const moe_fp8_gemm_desc *d = p[0];
        need[0] = rows_of(d->T, d->K, d->lda, 1);
        need[1] = table(d->T, d->K);
        need[2] = rows_of(d->N, d->K, d->ldw, 1);
        need[3] = table(blocks(d->N), d->K);
        need[4] = rows_of(d->T, d->N, d->ldy, size_of(d->y_type));
        return 5;
    }
    const moe_fp8_ffn_desc *d = p[0];
    need[0] = rows_of(d->T, d->d_model, d->ldx, 1);
    need[1] = table(d->T, d->d_model);
    need[2] = rows_of(d->T, d->d_model, d->ldy, size_of(d->y_type));
    /* the workspace: codes of h in rows of a multiple of 16, then its scales, each to 256 bytes */
    need[3] = (((int64_t)d->T * (((int64_t)d->d_ff + 15) / 16 * 16) + 255) / 256 * 256 + table(d->T, d->d_ff) + 255) /
              256 * 256;
    weights[0] = weights[2] = rows_of(d->d_ff, d->d_model, d->ld13, 1);
    weights[4] = rows_of(d->d_model, d->d_ff, d->ld2, 1);
    weights[1] = weights[3] = weights[5] = table(blocks(d->d_ff), d->d_model);
    return 4;
}

/* check(dev, tensors, needs) -> 0 or a code of take(). */
static PyObject *check(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n != 3) return PyErr_Format(PyExc_TypeError, "check takes 3 arguments");
    const long dev = PyLong_AsLong(a[0]);
    if (dev == -1 && PyErr_Occurred()) return NULL;
    void *p[kMaxBufs];
    long long needs[kMaxBufs];
    const int k = read_needs(a[2], needs);
    if (k < 0) return NULL;
    const long r = take(a[1], k, needs, dev, p);
    return r < 0 ? NULL : PyLong_FromLong(r);
}

/* addresses(objects) -> their addresses, as a tuple: of tensors, integers (which are addresses) and None. */
static PyObject *addresses(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n != 1 || !PyTuple_Check(a[0])) return PyErr_Format(PyExc_TypeError, "addresses takes a tuple");
    const Py_ssize_t k = PyTuple_GET_SIZE(a[0]);
    PyObject *r = PyTuple_New(k);
    for (Py_ssize_t i = 0; r && i < k; ++i) {
        PyObject *x = PyTuple_GET_ITEM(a[0], i), *v;
        long dev;
        long long bytes;
        void *p;
        if (x == Py_None || PyLong_Check(x)) v = Py_NewRef(x);
        else if (bound(x) && describe(x, &dev, &bytes, &p)) v = PyLong_FromVoidPtr(p);
        else v = PyObject_CallMethodNoArgs(x, s_data_ptr);
        if (v) PyTuple_SET_ITEM(r, i, v);
        else Py_CLEAR(r);
    }
    return r;
}

/* bind(type, type): tensors of exactly these types are looked at through their exchange table. */
static PyObject *bind(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n != 2) return PyErr_Format(PyExc_TypeError, "bind takes 2 arguments");
#ifdef EXCHANGE_TABLE
    PyObject *c = PyObject_GetAttrString(a[0], "__dlpack_c_exchange_api__");
    const DLPackExchangeAPI *api = c ? PyCapsule_GetPointer(c, "dlpack_exchange_api") : NULL;
    Py_XDECREF(c);  /* the type keeps it */
    PyErr_Clear();
    if (!api || api->header.version.major != DLPACK_MAJOR_VERSION || !api->dltensor_from_py_object_no_sync)
        Py_RETURN_FALSE;
    for (int i = 0; i < 2; ++i) Py_XSETREF(s_types[i], Py_NewRef(a[i]));
    s_api = api;
    Py_RETURN_TRUE;
#else
    Py_RETURN_FALSE;
#endif
}

typedef void *P;

/* call(address, dev, stream, structs, tensors, needs, weights=None) -> None, (status, 0, 0), or (0, code of
 * take(), bytes) without a call. structs: ctypes structures or None, passed first. needs: a tuple, or an
 * operator's number (its sizes are worked out from its structs). weights: the tensors of the FFN's weight struct,
 * which are only looked at; their codes start behind the tensors'. */
static PyObject *call(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n != 6 && n != 7) return PyErr_Format(PyExc_TypeError, "call takes 6 or 7 arguments");
    void *fn = PyLong_AsVoidPtr(a[0]);
    const long dev = PyLong_AsLong(a[1]);
    void *stream = PyLong_AsVoidPtr(a[2]);
    if (PyErr_Occurred()) return NULL;
    PyObject *structs = a[3];
    if (!PyTuple_Check(structs) || PyTuple_GET_SIZE(structs) > kMaxStructs)
        return PyErr_Format(PyExc_TypeError, "structs: a tuple of at most %d", kMaxStructs);
    void *p[kMaxStructs + kMaxBufs + 1];
    void *wp[kFfnWeights];
    Py_buffer view[kMaxStructs];
    Py_ssize_t len[kMaxStructs];
    long long needs[kMaxBufs], wneeds[kFfnWeights], at = 0;
    const int ns = (int)PyTuple_GET_SIZE(structs);
    int held = 0, status = 0, nt;
    long code = 0;
    PyObject *result = NULL;
    for (int i = 0; i < ns; ++i) {
        PyObject *o = PyTuple_GET_ITEM(structs, i);
        p[i] = NULL;
        len[i] = 0;
        if (o == Py_None) {
            view[held++].obj = NULL;
            continue;
        }
        if (PyObject_GetBuffer(o, &view[held], PyBUF_SIMPLE) != 0) goto out;
        len[i] = view[held].len;
        p[i] = view[held++].buf;
    }
    if (PyLong_Check(a[5])) nt = sizes(PyLong_AsLong(a[5]), p, len, ns, needs, wneeds);
    else nt = read_needs(a[5], needs);
    if (nt < 0 || (code = take(a[4], nt, needs, dev, p + ns)) < 0) goto out;
    if (code) at = needs[(code - 1) / 2];
    if (!code && n == 7 && a[6] != Py_None) {
        if ((code = take(a[6], kFfnWeights, wneeds, dev, wp)) < 0) goto out;
        if (code) at = wneeds[(code - 1) / 2], code += 2 * nt;
    }
    if (code == 0) {
        const int k = ns + nt;
        p[k] = stream;
        Py_BEGIN_ALLOW_THREADS
        switch (k + 1) {
            case 5: status = ((int (*)(P, P, P, P, P))fn)(p[0], p[1], p[2], p[3], p[4]); break;
            case 7: status = ((int (*)(P, P, P, P, P, P, P))fn)(p[0], p[1], p[2], p[3], p[4], p[5], p[6]); break;
            case 9:
                status = ((int (*)(P, P, P, P, P, P, P, P, P))fn)(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8]);
                break;
            case 12:
                status = ((int (*)(P, P, P, P, P, P, P, P, P, P, P, P))fn)(p[0], p[1], p[2], p[3], p[4], p[5], p[6],
                                                                          p[7], p[8], p[9], p[10], p[11]);
                break;
            default: status = -1;
        }
        Py_END_ALLOW_THREADS
        if (status == -1) {
            PyErr_Format(PyExc_TypeError, "no entry point takes %d arguments", k + 1);
            goto out;
        }
    }
    if (status == 0 && code == 0) result = Py_NewRef(Py_None);
    else result = Py_BuildValue("(ilL)", status, code, at);
out:
    for (int i = 0; i < held; ++i)
        if (view[i].obj) PyBuffer_Release(&view[i]);
    return result;
}

static PyMethodDef methods[] = {
    {"call", (PyCFunction)(void (*)(void))call, METH_FASTCALL, "call(address, dev, stream, structs, tensors, needs, weights=None)"},
    {"addresses", (PyCFunction)(void (*)(void))addresses, METH_FASTCALL, "addresses(objects)"},
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, "bind(type, type)"},
    {"check", (PyCFunction)(void (*)(void))check, METH_FASTCALL, "check(dev, tensors, needs)"},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
    if (!(s_get_device = PyUnicode_InternFromString("get_device")) || !(s_nbytes = PyUnicode_InternFromString("nbytes")) ||
        !(s_data_ptr = PyUnicode_InternFromString("data_ptr")) ||
        !(s_storage = PyUnicode_InternFromString("untyped_storage")) ||
        !(s_offset = PyUnicode_InternFromString("storage_offset")) ||
        !(s_itemsize = PyUnicode_InternFromString("element_size")) ||
        !(s_contiguous = PyUnicode_InternFromString("is_contiguous")))
        return NULL;
    PyObject *m = PyModule_Create(&module);
    if (m && (PyModule_AddIntConstant(m, "NORM", kNorm) || PyModule_AddIntConstant(m, "QUANTIZE", kQuantize) ||
              PyModule_AddIntConstant(m, "GEMM", kGemm) || PyModule_AddIntConstant(m, "FFN", kFfn))) {
        Py_DECREF(m);
        return NULL;
    }
    return m;
}
