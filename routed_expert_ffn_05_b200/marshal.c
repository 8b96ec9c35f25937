/*
 * Argument marshalling of the FP8 entry points for Python, in C: the smallest of
 * them run for a few microseconds on the GPU, about as long as checking five
 * tensors and making the call takes through ctypes (4.2 us; 0.7 us here).
 *
 * Only marshalling: tensor -> device pointer, with the same checks for every tensor
 * (it lives on the given device, its elements are of the type that the call reads
 * or writes, its rows lie where the call looks for them, and it holds that many
 * bytes), and a call of a libmoe.so entry point, whose arguments are all pointers:
 * structs, buffers, stream. Tensors are looked at
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
#include <string.h>

#if __has_include(<ATen/dlpack.h>)
#include <ATen/dlpack.h>
#endif
#if defined(DLPACK_MAJOR_VERSION) && (DLPACK_MAJOR_VERSION > 1 || DLPACK_MINOR_VERSION >= 3)
#define EXCHANGE_TABLE 1
#endif

#include "moe.h"

enum { kMaxStructs = 4, kMaxBufs = 8 };

static PyObject *s_get_device, *s_nbytes, *s_data_ptr, *s_storage, *s_offset, *s_itemsize, *s_dtype, *s_shape, *s_stride;

/* What a tensor's elements are, as far as the entry points care. */
enum { kByte, kInt8, kE4m3, kInt16, kBf16Type, kInt32, kF32Type, kOther };

enum { kMaxDims = 16 };
typedef struct {
    long dev;                /* -1: host */
    int type, ndim;
    long long size;          /* bytes of an element */
    long long shape[kMaxDims], stride[kMaxDims];
    void *p;
} Tensor;

/* What a buffer of a call is: `rows` rows of `row` bytes, `ld` bytes apart, of elements that `kind` names. */
enum { kAny, kCodes, kBf16, kF32, kI32 };
typedef struct {
    long long need, row, ld, rows;
    int kind;
} Buffer;

/* int16 and int32 hold the bits of the 16- and 32-bit types (the routed layer's calls take them so), and a uint8
 * tensor is a buffer of bytes. */
static int accepts(int kind, int type) {
    if (kind == kAny || type == kByte) return 1;
    if (kind == kCodes) return type == kInt8 || type == kE4m3;
    if (kind == kBf16) return type == kBf16Type || type == kInt16;
    return type == kInt32 || (kind == kF32 && type == kF32Type);
}

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

/* What x is, from the exchange table; 0 when the table does not describe it. */
static int describe(PyObject *x, Tensor *o) {
    DLTensor t;
    if (s_api->dltensor_from_py_object_no_sync(x, &t) != 0) {
        PyErr_Clear();
        return 0;
    }
    if ((t.device.device_type != kDLCUDA && t.device.device_type != kDLCPU) || t.ndim > kMaxDims || t.dtype.lanes != 1)
        return 0;
    o->dev = t.device.device_type == kDLCUDA ? t.device.device_id : -1;
    o->ndim = t.ndim;
    o->size = (t.dtype.bits + 7) / 8;
    const int c = t.dtype.code, bits = t.dtype.bits, whole = c == kDLInt || c == kDLUInt;
    o->type = whole && bits == 8 ? (c == kDLUInt ? kByte : kInt8) : whole && bits == 16 ? kInt16
              : whole && bits == 32 ? kInt32 : c == kDLBfloat && bits == 16 ? kBf16Type
              : c == kDLFloat && bits == 32 ? kF32Type : c == kDLFloat8_e4m3fn ? kE4m3 : kOther;
    long long dense = 1;
    for (int i = t.ndim - 1; i >= 0; --i) {
        o->shape[i] = t.shape[i];
        o->stride[i] = t.strides ? t.strides[i] : dense;
        dense *= t.shape[i];
    }
    o->p = (char *)t.data + t.byte_offset;
    return 1;
}
#else
static int bound(PyObject *x) { (void)x; return 0; }
static int describe(PyObject *x, Tensor *o) { (void)x; (void)o; return 0; }
#endif

/* A sequence of integers, at most kMaxDims; their number or -1 with an exception set. Steals the reference. */
static int dims_of(PyObject *seq, long long *out) {
    if (!seq) return -1;
    const Py_ssize_t n = PySequence_Size(seq);
    if (n > kMaxDims) PyErr_Format(PyExc_ValueError, "a tensor of more than %d dimensions", kMaxDims);
    for (Py_ssize_t i = 0; n <= kMaxDims && i < n; ++i) {
        PyObject *v = PySequence_GetItem(seq, i);
        out[i] = v ? PyLong_AsLongLong(v) : -1;
        Py_XDECREF(v);
        if (PyErr_Occurred()) break;
    }
    Py_DECREF(seq);
    return PyErr_Occurred() ? -1 : (int)n;
}

/* The same through x's methods; 0 with an exception set on failure. */
static int ask(PyObject *x, Tensor *o) {
    static const struct { const char *name; int type; } names[] = {
        {"torch.uint8", kByte}, {"torch.int8", kInt8}, {"torch.float8_e4m3fn", kE4m3}, {"torch.int16", kInt16},
        {"torch.uint16", kInt16}, {"torch.bfloat16", kBf16Type}, {"torch.int32", kInt32}, {"torch.uint32", kInt32},
        {"torch.float32", kF32Type}};
    o->dev = (long)number(x, s_get_device, 1);
    if (o->dev == -1 && PyErr_Occurred()) return 0;
    if ((o->size = number(x, s_itemsize, 1)) < 0) return 0;
    o->ndim = dims_of(PyObject_GetAttr(x, s_shape), o->shape);
    if (o->ndim < 0 || dims_of(PyObject_CallMethodNoArgs(x, s_stride), o->stride) != o->ndim) return 0;
    PyObject *dtype = PyObject_GetAttr(x, s_dtype), *name = dtype ? PyObject_Str(dtype) : NULL;
    Py_XDECREF(dtype);
    if (!name) return 0;
    const char *text = PyUnicode_AsUTF8(name);
    o->type = kOther;
    for (size_t i = 0; text && i < sizeof names / sizeof *names; ++i)
        if (!strcmp(text, names[i].name)) o->type = names[i].type;
    Py_DECREF(name);
    PyObject *p = text ? PyObject_CallMethodNoArgs(x, s_data_ptr) : NULL;
    if (!p) return 0;
    o->p = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    return o->p || !PyErr_Occurred();
}

/* Bytes from the first element to the end of the last. */
static long long span(const Tensor *t) {
    long long last = 0;
    for (int i = 0; i < t->ndim; ++i) {
        if (t->shape[i] == 0) return 0;
        last += (t->shape[i] - 1) * t->stride[i];
    }
    return (last + 1) * t->size;
}

/* Whether the tensor's memory is laid out as the buffer's rows are: dense, or dense runs that hold a row, b->ld
 * bytes apart. */
static int laid_out(const Tensor *t, const Buffer *b) {
    long long run = t->size;  /* bytes that follow one another */
    int i = t->ndim - 1;
    for (; i >= 0; --i) {
        if (t->shape[i] == 1) continue;
        if (t->stride[i] * t->size != run) break;
        run *= t->shape[i];
    }
    if (i < 0) return 1;
    if (run < b->row) return 0;
    if (b->rows == 1) return 1;
    for (long long step = b->ld; i >= 0; --i) {
        if (t->shape[i] == 1) continue;
        if (t->stride[i] * t->size != step) return 0;
        step *= t->shape[i];
    }
    return 1;
}

/* The pointers of the n objects in tuple `t`, each a buffer b[i] on device dev: None -> NULL, an int is an address
 * and passes unchecked. 0, or 2 i + 1 (tensor i on another device), 2 i + 2 (too small), or -1 with an exception
 * set. `whole`: what the tensor itself holds counts, and its type (kOddType + i) and layout (kOddLayout + i) are
 * looked at; otherwise only device and bytes, those behind it in its storage included. */
enum { kOddType = 1000, kOddLayout = 2000 };
static long take(PyObject *t, int n, const Buffer *b, long dev, void **out, int whole) {
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
        Tensor d;
        if (!(bound(x) && describe(x, &d)) && !ask(x, &d)) return -1;
        if (d.dev != dev) return 2 * i + 1;
        long long has = span(&d);
        if (has < b[i].need && !whole) {  /* part of a larger buffer: what lies behind it counts */
            has = bytes_behind(x);
            if (has < 0 && PyErr_Occurred()) return -1;
        }
        /* (!d.p: memory that was given back) */
        if (has < b[i].need || (b[i].need > 0 && !d.p)) return 2 * i + 2;
        if (whole && b[i].need > 0) {
            if (!accepts(b[i].kind, d.type)) return kOddType + i;
            if (!laid_out(&d, &b[i])) return kOddLayout + i;
        }
        out[i] = d.p;
    }
    return 0;
}

/* A tuple of at most kMaxBufs byte counts; their number, or -1 with an exception set. */
static int read_needs(PyObject *t, Buffer *needs) {
    if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) > kMaxBufs) {
        PyErr_Format(PyExc_TypeError, "needs: a tuple of at most %d byte counts", kMaxBufs);
        return -1;
    }
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(t); ++i) {
        needs[i] = (Buffer){PyLong_AsLongLong(PyTuple_GET_ITEM(t, i)), 0, 0, 1, kAny};
        if (needs[i].need == -1 && PyErr_Occurred()) return -1;
    }
    return (int)PyTuple_GET_SIZE(t);
}

/* `rows` rows of `cols` elements of `size` bytes, `ld` elements apart; a table of one float per block; a workspace.
 * Bytes beyond 63 bits: the largest count, which no tensor holds. */
static long long clamp(__int128 v) { return v > INT64_MAX ? INT64_MAX : v < -1 ? -1 : (long long)v; }
static Buffer rows_of(long long rows, long long cols, long long ld, int size, int kind) {
    return (Buffer){clamp(((__int128)(rows - 1) * ld + cols) * size), clamp((__int128)cols * size),
                    clamp((__int128)ld * size), rows, kind};
}
static long long blocks(long long n) { return (n + 127) / 128; }
static Buffer table(long long rows, long long cols) { return rows_of(rows, blocks(cols), blocks(cols), 4, kF32); }
static Buffer bytes_of(long long n) { return (Buffer){n, n, n, 1, kAny}; }
static Buffer typed(long long rows, long long cols, long long ld, int32_t type) {
    return type == MOE_T_BF16 ? rows_of(rows, cols, ld, 2, kBf16) : rows_of(rows, cols, ld, 4, kF32);
}

enum { kNorm, kQuantize, kGemm, kFfn, kBlock, kOps };
enum { kFfnWeights = 6 };

static void weights_of(long long d, long long F, long long ld13, long long ld2, Buffer *w) {
    w[0] = w[2] = rows_of(F, d, ld13, 1, kCodes);
    w[1] = w[3] = table(blocks(F), d);
    w[4] = rows_of(d, F, ld2, 1, kCodes);
    w[5] = table(blocks(d), F);
}

/* What the buffers of an entry point are for these structs (and the FFN's weights; ws: bytes of moe_block's
 * workspace); the number of buffers, or -1 with an exception set when a struct is not the one it takes. */
static int sizes(long op, void *const *p, const Py_ssize_t *len, int n, long long ws, Buffer *need, Buffer *weights) {
    static const size_t first[kOps] = {sizeof(moe_norm_desc), sizeof(moe_fp8_quant_desc), sizeof(moe_fp8_gemm_desc),
                                       sizeof(moe_fp8_ffn_desc), sizeof(moe_dims)};
    static const int structs[kOps] = {1, 1, 1, 2, 4};
    int ok = op >= 0 && op < kOps && n == structs[op] && p[0] && (size_t)len[0] == first[op];
    if (ok && op == kFfn) ok = !p[1] || (size_t)len[1] == sizeof(moe_fp8_ffn_weights);
    if (ok && op == kBlock)
        ok = (!p[1] || (size_t)len[1] == sizeof(moe_weights)) && p[2] && (size_t)len[2] == sizeof(moe_norm_desc) &&
             (!p[3] || (size_t)len[3] == sizeof(moe_fp8_ffn_weights));
    if (!ok) {
        PyErr_SetString(PyExc_TypeError, "not the descriptor of this entry point");
        return -1;
    }
    if (op == kNorm) {
        const moe_norm_desc *d = p[0];
        need[0] = typed(d->T, d->d, d->ldx, d->x_type);
        need[1] = need[3] = typed(d->T, d->d, d->ldr, d->res_type);
        need[2] = typed(1, d->d, d->d, d->w_type);
        need[4] = typed(d->T, d->d, d->ldy, MOE_T_BF16);
        need[5] = rows_of(d->T, d->d, d->ldq, 1, kCodes);
        need[6] = table(d->T, d->d);
        return 7;
    }
    if (op == kQuantize) {
        const moe_fp8_quant_desc *d = p[0];
        need[0] = typed(d->rows, d->cols, d->ldv, d->v_type);
        need[1] = rows_of(d->rows, d->cols, d->ldq, 1, kCodes);
        need[2] = table(d->block_rows == 1 ? d->rows : blocks(d->rows), d->cols);
        return 3;
    }
    if (op == kGemm) {
        const moe_fp8_gemm_desc *d = p[0];
        need[0] = rows_of(d->T, d->K, d->lda, 1, kCodes);
        need[1] = table(d->T, d->K);
        need[2] = rows_of(d->N, d->K, d->ldw, 1, kCodes);
        need[3] = table(blocks(d->N), d->K);
        need[4] = typed(d->T, d->N, d->ldy, d->y_type);
        return 5;
    }
    if (op == kBlock) {
        const moe_dims *d = p[0];
        const moe_norm_desc *m = p[2];
        need[0] = typed(d->T, d->d_model, m->ldx, m->x_type);
        need[1] = need[3] = typed(d->T, d->d_model, m->ldr, m->res_type);
        need[2] = typed(1, d->d_model, d->d_model, m->w_type);
        need[4] = rows_of(1, d->T, d->T, 4, kI32);
        need[5] = typed(d->T, d->d_model, d->d_model, MOE_T_F32);
        need[6] = bytes_of(ws);
        weights_of(d->d_model, d->d_ff_shared, d->d_model, d->d_ff_shared, weights);
        return 7;
    }
    const moe_fp8_ffn_desc *d = p[0];
    need[0] = rows_of(d->T, d->d_model, d->ldx, 1, kCodes);
    need[1] = table(d->T, d->d_model);
    need[2] = typed(d->T, d->d_model, d->ldy, d->y_type);
    /* the workspace: codes of h in rows of a multiple of 16, then its scales, each to 256 bytes */
    need[3] = bytes_of((((int64_t)d->T * (((int64_t)d->d_ff + 15) / 16 * 16) + 255) / 256 * 256 +
                        table(d->T, d->d_ff).need + 255) / 256 * 256);
    weights_of(d->d_model, d->d_ff, d->ld13, d->ld2, weights);
    return 4;
}

/* check(dev, tensors, needs) -> 0 or a code of take(). */
static PyObject *check(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n != 3) return PyErr_Format(PyExc_TypeError, "check takes 3 arguments");
    const long dev = PyLong_AsLong(a[0]);
    if (dev == -1 && PyErr_Occurred()) return NULL;
    void *p[kMaxBufs];
    Buffer needs[kMaxBufs];
    const int k = read_needs(a[2], needs);
    if (k < 0) return NULL;
    const long r = take(a[1], k, needs, dev, p, 0);
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
        Tensor d;
        if (x == Py_None || PyLong_Check(x)) v = Py_NewRef(x);
        else if (bound(x) && describe(x, &d)) v = PyLong_FromVoidPtr(d.p);
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

/* call(address, dev, stream, structs, tensors, needs, weights=None, ws=0) -> None, (status, 0, 0), or (0, code of
 * take(), bytes) without a call. structs: ctypes structures or None, passed first. needs: a tuple of byte counts, or
 * an operator's number (its buffers are worked out from its structs and ws, moe_block's workspace). weights: the
 * tensors of the FFN's weight struct, which are only looked at; their codes start behind the tensors'. */
static PyObject *call(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n < 6 || n > 8) return PyErr_Format(PyExc_TypeError, "call takes 6 to 8 arguments");
    void *fn = PyLong_AsVoidPtr(a[0]);
    const long dev = PyLong_AsLong(a[1]);
    void *stream = PyLong_AsVoidPtr(a[2]);
    const long long ws = n == 8 ? PyLong_AsLongLong(a[7]) : 0;
    if (PyErr_Occurred()) return NULL;
    PyObject *structs = a[3];
    if (!PyTuple_Check(structs) || PyTuple_GET_SIZE(structs) > kMaxStructs)
        return PyErr_Format(PyExc_TypeError, "structs: a tuple of at most %d", kMaxStructs);
    void *p[kMaxStructs + kMaxBufs + 1];
    void *wp[kFfnWeights];
    Py_buffer view[kMaxStructs];
    Py_ssize_t len[kMaxStructs];
    Buffer needs[kMaxBufs], wneeds[kFfnWeights];
    long long at = 0;
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
    const int whole = PyLong_Check(a[5]);
    if (whole) nt = sizes(PyLong_AsLong(a[5]), p, len, ns, ws, needs, wneeds);
    else nt = read_needs(a[5], needs);
    if (nt < 0 || (code = take(a[4], nt, needs, dev, p + ns, whole)) < 0) goto out;
    if (code) at = code < kOddType ? needs[(code - 1) / 2].need : 0;
    if (!code && n > 6 && a[6] != Py_None) {
        if ((code = take(a[6], kFfnWeights, wneeds, dev, wp, whole)) < 0) goto out;
        if (code) {
            at = code < kOddType ? wneeds[(code - 1) / 2].need : 0;
            code += code < kOddType ? 2 * nt : nt;
        }
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
    {"call", (PyCFunction)(void (*)(void))call, METH_FASTCALL, "call(address, dev, stream, structs, tensors, needs, weights=None, ws=0)"},
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
        !(s_dtype = PyUnicode_InternFromString("dtype")) || !(s_shape = PyUnicode_InternFromString("shape")) ||
        !(s_stride = PyUnicode_InternFromString("stride")))
        return NULL;
    PyObject *m = PyModule_Create(&module);
    if (m && (PyModule_AddIntConstant(m, "NORM", kNorm) || PyModule_AddIntConstant(m, "QUANTIZE", kQuantize) ||
              PyModule_AddIntConstant(m, "GEMM", kGemm) || PyModule_AddIntConstant(m, "FFN", kFfn) ||
              PyModule_AddIntConstant(m, "BLOCK", kBlock))) {
        Py_DECREF(m);
        return NULL;
    }
    return m;
}
