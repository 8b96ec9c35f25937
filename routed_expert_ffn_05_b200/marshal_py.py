"""What marshal.c does, through ctypes: the binding uses it where the C part is not built.

The same calls with the same answers (a test runs the binding's host tests through both);
a call takes about 4 us on the host instead of 0.7.
"""
from __future__ import annotations

import ctypes

NORM, QUANTIZE, GEMM, FFN = range(4)
_INT64_MAX = (1 << 63) - 1


def bind(*types):
    """Nothing to look up: tensors are looked at through their methods."""
    return True


def _behind(x):
    """Bytes from x's first element to the end of its storage."""
    return x.untyped_storage().nbytes() - x.storage_offset() * x.element_size()


def _take(tensors, needs, dev):
    """(code, pointers): 0, or 2 i + 1 (tensor i on another device), 2 i + 2 (too small)."""
    if not isinstance(tensors, tuple) or len(tensors) != len(needs):
        raise TypeError(f"expected a tuple of {len(needs)} tensors")
    out = []
    for i, (x, need) in enumerate(zip(tensors, needs)):
        if x is None or isinstance(x, int):
            out.append(x)
            continue
        if x.get_device() != dev:
            return 2 * i + 1, out
        # nbytes counts elements: what memory they take is known for a contiguous tensor only
        if (not x.is_contiguous() or x.nbytes < need) and _behind(x) < need:
            return 2 * i + 2, out
        p = x.data_ptr()
        if need > 0 and not p:  # memory that was given back
            return 2 * i + 2, out
        out.append(p)
    return 0, out


def _clamp(v):
    return min(max(v, -1), _INT64_MAX)


def _rows(rows, cols, ld, size):
    return _clamp(((rows - 1) * ld + cols) * size)


def _blocks(n):
    return (n + 127) // 128


def _table(rows, cols):
    return _clamp(4 * rows * _blocks(cols))


def _size(t):
    return 2 if t == 0 else 4


def _sizes(op, structs):
    """What the buffers of an entry point hold for these structs, and the FFN's weights."""
    import routed_expert_ffn_05_b200 as M
    desc = (M.moe_norm_desc, M.moe_fp8_quant_desc, M.moe_fp8_gemm_desc, M.moe_fp8_ffn_desc)
    ok = 0 <= op < 4 and len(structs) == (2 if op == FFN else 1) and type(structs[0]) is desc[op]
    if not ok or (op == FFN and structs[1] is not None and type(structs[1]) is not M.moe_fp8_ffn_weights):
        raise TypeError("not the descriptor of this entry point")
    d = structs[0]
    if op == NORM:
        res = _rows(d.T, d.d, d.ldr, _size(d.res_type))
        return (_rows(d.T, d.d, d.ldx, _size(d.x_type)), res, _rows(1, d.d, 0, _size(d.w_type)), res,
                _rows(d.T, d.d, d.ldy, 2), _rows(d.T, d.d, d.ldq, 1), _table(d.T, d.d)), ()
    if op == QUANTIZE:
        return (_rows(d.rows, d.cols, d.ldv, _size(d.v_type)), _rows(d.rows, d.cols, d.ldq, 1),
                _table(d.rows if d.block_rows == 1 else _blocks(d.rows), d.cols)), ()
    if op == GEMM:
        return (_rows(d.T, d.K, d.lda, 1), _table(d.T, d.K), _rows(d.N, d.K, d.ldw, 1), _table(_blocks(d.N), d.K),
                _rows(d.T, d.N, d.ldy, _size(d.y_type))), ()
    w13, t = _rows(d.d_ff, d.d_model, d.ld13, 1), _table(_blocks(d.d_ff), d.d_model)
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    ws = up(up(d.T * ((d.d_ff + 15) // 16 * 16)) + _table(d.T, d.d_ff))
    return (_rows(d.T, d.d_model, d.ldx, 1), _table(d.T, d.d_model), _rows(d.T, d.d_model, d.ldy, _size(d.y_type)),
            ws), (w13, t, w13, t, _rows(d.d_model, d.d_ff, d.ld2, 1), t)


def check(dev, tensors, needs):
    if not isinstance(needs, tuple) or len(needs) > 8:
        raise TypeError("needs: a tuple of at most 8 byte counts")
    return _take(tensors, needs, dev)[0]


def addresses(objects):
    if not isinstance(objects, tuple):
        raise TypeError("addresses takes a tuple")
    return tuple(x if x is None or isinstance(x, int) else x.data_ptr() for x in objects)


_calls = {}  # entry point's address -> ctypes function


def call(address, dev, stream, structs, tensors, needs, weights=None):
    wneeds = ()
    if isinstance(needs, int):
        needs, wneeds = _sizes(needs, structs)
    code, p = _take(tensors, needs, dev)
    at = needs[(code - 1) // 2] if code else 0
    if not code and weights is not None:
        code, _ = _take(weights, wneeds, dev)
        if code:
            at, code = wneeds[(code - 1) // 2], code + 2 * len(needs)
    if code:
        return 0, code, at
    args = [None if s is None else ctypes.addressof(s) for s in structs] + p + [stream]
    if len(args) not in (5, 7, 9, 12):
        raise TypeError(f"no entry point takes {len(args)} arguments")
    key = address, len(args)
    if key not in _calls:
        _calls[key] = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * len(args))(address)
    status = _calls[key](*args)
    return (status, 0, 0) if status else None
