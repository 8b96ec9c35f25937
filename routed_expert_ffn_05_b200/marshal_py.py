"""What marshal.c does, through ctypes: the binding uses it where the C part is not built.

The same calls with the same answers (a test runs the binding's host tests through both);
a call takes about 4 us on the host instead of 0.7.
"""
from __future__ import annotations

import ctypes

NORM, QUANTIZE, GEMM, FFN, BLOCK = range(5)
_INT64_MAX = (1 << 63) - 1
_ANY, _CODES, _BF16, _F32, _I32 = range(5)
# int16 and int32 hold the bits of the 16- and 32-bit types, and a uint8 tensor is a buffer of bytes
_TYPES = {_CODES: ("uint8", "int8", "float8_e4m3fn"), _BF16: ("uint8", "bfloat16", "int16", "uint16"),
          _F32: ("uint8", "float32", "int32", "uint32"), _I32: ("uint8", "int32", "uint32")}


def bind(*types):
    """Nothing to look up: tensors are looked at through their methods."""
    return True


def _behind(x):
    """Bytes from x's first element to the end of its storage."""
    return x.untyped_storage().nbytes() - x.storage_offset() * x.element_size()


def _span(x):
    """Bytes from x's first element to the end of its last."""
    if 0 in x.shape:
        return 0
    return (sum((n - 1) * st for n, st in zip(x.shape, x.stride())) + 1) * x.element_size()


def _laid_out(x, row, ld, rows):
    """Whether x is dense, or dense runs that hold a row, ld bytes apart."""
    size = x.element_size()
    run = size
    dims = [(n, st * size) for n, st in zip(x.shape, x.stride()) if n != 1]
    while dims and dims[-1][1] == run:
        run *= dims.pop()[0]
    if not dims:
        return True
    if run < row:
        return False
    step = ld
    while rows != 1 and dims:
        n, st = dims.pop()
        if st != step:
            return False
        step *= n
    return True


def _take(tensors, needs, dev, whole):
    """(code, pointers): 0, or 2 i + 1 (tensor i on another device), 2 i + 2 (too small), 1000 + i (its type),
    2000 + i (its layout). needs: (bytes, kind, row, ld, rows) each, or bytes alone where not ``whole``."""
    if not isinstance(tensors, tuple) or len(tensors) != len(needs):
        raise TypeError(f"expected a tuple of {len(needs)} tensors")
    out = []
    for i, (x, b) in enumerate(zip(tensors, needs)):
        if x is None or isinstance(x, int):
            out.append(x)
            continue
        need = b[0] if whole else b
        if x.get_device() != dev:
            return 2 * i + 1, out
        if _span(x) < need and (whole or _behind(x) < need):
            return 2 * i + 2, out
        p = x.data_ptr()
        if need > 0 and not p:  # memory that was given back
            return 2 * i + 2, out
        if whole and need > 0:
            if b[1] != _ANY and str(x.dtype).split(".")[-1] not in _TYPES[b[1]]:
                return 1000 + i, out
            if not _laid_out(x, *b[2:]):
                return 2000 + i, out
        out.append(p)
    return 0, out


def _clamp(v):
    return min(max(v, -1), _INT64_MAX)


def _rows(rows, cols, ld, size, kind):
    return _clamp(((rows - 1) * ld + cols) * size), kind, cols * size, ld * size, rows


def _typed(rows, cols, ld, t):
    return _rows(rows, cols, ld, 2, _BF16) if t == 0 else _rows(rows, cols, ld, 4, _F32)


def _blocks(n):
    return (n + 127) // 128


def _table(rows, cols):
    return _rows(rows, _blocks(cols), _blocks(cols), 4, _F32)


def _weights(d, F, ld13, ld2):
    w13, t = _rows(F, d, ld13, 1, _CODES), _table(_blocks(F), d)
    return w13, t, w13, t, _rows(d, F, ld2, 1, _CODES), _table(_blocks(d), F)


def _sizes(op, structs, ws):
    """What the buffers of an entry point are for these structs, and the FFN's weights."""
    import routed_expert_ffn_05_b200 as M
    types = {NORM: (M.moe_norm_desc,), QUANTIZE: (M.moe_fp8_quant_desc,), GEMM: (M.moe_fp8_gemm_desc,),
             FFN: (M.moe_fp8_ffn_desc, M.moe_fp8_ffn_weights),
             BLOCK: (M.moe_dims, M.moe_weights, M.moe_norm_desc, M.moe_fp8_ffn_weights)}.get(op, ())
    may_be_none = {FFN: (1,), BLOCK: (1, 3)}.get(op, ())
    if not types or len(structs) != len(types) or not all(
            type(s) is t or (s is None and i in may_be_none) for i, (s, t) in enumerate(zip(structs, types))):
        raise TypeError("not the descriptor of this entry point")
    d = structs[0]
    if op == NORM:
        res = _typed(d.T, d.d, d.ldr, d.res_type)
        return (_typed(d.T, d.d, d.ldx, d.x_type), res, _typed(1, d.d, d.d, d.w_type), res, _typed(d.T, d.d, d.ldy, 0),
                _rows(d.T, d.d, d.ldq, 1, _CODES), _table(d.T, d.d)), ()
    if op == QUANTIZE:
        return (_typed(d.rows, d.cols, d.ldv, d.v_type), _rows(d.rows, d.cols, d.ldq, 1, _CODES),
                _table(d.rows if d.block_rows == 1 else _blocks(d.rows), d.cols)), ()
    if op == GEMM:
        return (_rows(d.T, d.K, d.lda, 1, _CODES), _table(d.T, d.K), _rows(d.N, d.K, d.ldw, 1, _CODES),
                _table(_blocks(d.N), d.K), _typed(d.T, d.N, d.ldy, d.y_type)), ()
    if op == BLOCK:
        m, D, F = structs[2], d.d_model, d.d_ff_shared
        res = _typed(d.T, D, m.ldr, m.res_type)
        return (_typed(d.T, D, m.ldx, m.x_type), res, _typed(1, D, D, m.w_type), res, _rows(1, d.T, d.T, 4, _I32),
                _typed(d.T, D, D, 1), (ws, _ANY, ws, ws, 1)), _weights(D, F, D, F)
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    ws = up(up(d.T * ((d.d_ff + 15) // 16 * 16)) + _table(d.T, d.d_ff)[0])
    return (_rows(d.T, d.d_model, d.ldx, 1, _CODES), _table(d.T, d.d_model), _typed(d.T, d.d_model, d.ldy, d.y_type),
            (ws, _ANY, ws, ws, 1)), _weights(d.d_model, d.d_ff, d.ld13, d.ld2)


def check(dev, tensors, needs):
    if not isinstance(needs, tuple) or len(needs) > 8:
        raise TypeError("needs: a tuple of at most 8 byte counts")
    return _take(tensors, needs, dev, False)[0]


def addresses(objects):
    if not isinstance(objects, tuple):
        raise TypeError("addresses takes a tuple")
    return tuple(x if x is None or isinstance(x, int) else x.data_ptr() for x in objects)


_calls = {}  # entry point's address -> ctypes function


def call(address, dev, stream, structs, tensors, needs, weights=None, ws=0):
    whole, wneeds = isinstance(needs, int), ()
    if whole:
        needs, wneeds = _sizes(needs, structs, ws)
    n = len(needs)
    code, p = _take(tensors, needs, dev, whole)
    if not code and weights is not None:
        code, _ = _take(weights, wneeds, dev, whole)
        if code:
            needs += wneeds
            code += n if code >= 1000 else 2 * n
    if code:
        b = needs[(code - 1) // 2] if code < 1000 else (0,)
        return 0, code, b[0] if whole else b
    args = [None if s is None else ctypes.addressof(s) for s in structs] + p + [stream]
    if len(args) not in (5, 7, 9, 12):
        raise TypeError(f"no entry point takes {len(args)} arguments")
    key = address, len(args)
    if key not in _calls:
        _calls[key] = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * len(args))(address)
    status = _calls[key](*args)
    return (status, 0, 0) if status else None
