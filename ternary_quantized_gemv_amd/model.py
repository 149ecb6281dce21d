"""Python binding of the operators around the layers (include/bq.h): bq_embed,
bq_gated_q8, bq_matmul and bq_sample.

As in layer.py the functions keep the C names and only marshal arguments:
shapes, types, strides and devices are checked against each other here,
everything else by the library.  A call runs on the device of its tensors,
whichever is current, and on `stream` (default: the current stream of that
device).
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import Act, Weights, bq_act, bq_weights, lib
from .layer import (TYPES, _check, _f32, _first, _flat, _i32, _i64, _Pack, _refuse, _rows, _run, _scratch, _type, _vp)

BQ_NONE, BQ_SILU, BQ_GELU, BQ_RELU2 = 0, 1, 2, 3
BQ_VOCAB_MAX = 1 << 22


class bq_table(ctypes.Structure):
    _fields_ = [("w", bq_weights), ("dense", _vp), ("ld_dense", _i64), ("dense_type", _i32), ("type", _i32),
                ("scale", _f32), ("reserved", _i32), ("tokens", _i64), ("ids", _vp), ("out", _vp), ("ld_out", _i64)]


class bq_gated(ctypes.Structure):
    _fields_ = [("type", _i32), ("act", _i32), ("qa", _i32), ("f16_scale", _i32), ("tokens", _i64), ("n", _i64),
                ("gate", _vp), ("ld_gate", _i64), ("up", _vp), ("ld_up", _i64), ("q", _vp), ("ld_q", _i64), ("d", _vp),
                ("ld_d", _i64), ("y", _vp), ("ld_y", _i64)]


class bq_product(ctypes.Structure):
    _fields_ = [("w", bq_weights), ("a", bq_act), ("type", _i32), ("act", _i32), ("bias", _vp), ("mul", _vp),
                ("ld_mul", _i64), ("res", _vp), ("ld_res", _i64), ("y", _vp), ("ld_y", _i64), ("work", _vp),
                ("work_bytes", _i64)]


class bq_draw(ctypes.Structure):
    _fields_ = [("type", _i32), ("reserved", _i32), ("rows", _i64), ("vocab", _i64), ("logits", _vp),
                ("ld_logits", _i64), ("u", _vp), ("temperature", _vp), ("top_k", _vp), ("top_p", _vp), ("min_p", _vp),
                ("token", _vp), ("logprob", _vp), ("work", _vp), ("work_bytes", _i64)]


_pack_table, _pack_gated, _pack_product, _pack_draw = (_Pack(k).pack for k in (bq_table, bq_gated, bq_product, bq_draw))

for _name in ("bq_embed", "bq_gated_q8", "bq_matmul", "bq_matmul_work_bytes", "bq_sample", "bq_sample_work_bytes"):
    getattr(lib, _name).restype = ctypes.c_int
    getattr(lib, _name).argtypes = [_vp, _vp]


def _matrix(fn: str, what: str, t) -> tuple:
    """Shape of a tensor of rows; a single row may come without its first dimension."""
    if not isinstance(t, torch.Tensor) or t.dim() not in (1, 2):
        _refuse(fn, f"{what} must be a tensor of one or two dimensions")
    return tuple(t.shape) if t.dim() == 2 else (1, t.shape[0])


def _planes(fn: str, w: Weights) -> tuple:
    """The fields of a packed matrix, and its device."""
    dev = w.bits.get_device()
    if w.scales.get_device() != dev:
        _refuse(fn, "the planes of the weights must be on one device")
    return (w.fmt, 0, w.rows, w.cols, w.bits.data_ptr(), w.scales.data_ptr()), dev


def _work_of(fn: str, work, need: int, dev: int, stream) -> tuple:
    """Pointer and bytes of the scratch, and what keeps it: the caller's, one of this call, or none."""
    if work is None and not need:
        return 0, 0, None
    work = _scratch(fn, work, need, dev, stream)
    return work.data_ptr(), work.nbytes, work


def bq_embed(table, ids, out, scale: float = 1.0, stream=None) -> None:
    """out[t] = scale * table[ids[t]].  table: Weights, or a tensor [count, n]
    (float32, float16 or bfloat16); ids: int64 [tokens] (-1: a row of zeros);
    out: [tokens, n] of any of the three types."""
    fn = "bq_embed"
    if isinstance(table, Weights):
        w, dev = _planes(fn, table)
        dense = (0, 0, 0)
        n = table.cols
    else:
        dev = _first(fn, "table", table)
        if table.dim() != 2:
            _refuse(fn, "table must be Weights or [count, n]")
        count, n = table.shape
        kind = _type(fn, "table", table)
        p, ld = _rows(fn, "table", table, table.dtype, dev, (count, n))
        w, dense = (0, 0, count, n, 0, 0), (p, ld, kind)
    if not isinstance(ids, torch.Tensor) or ids.dim() != 1:
        _refuse(fn, "ids must be [tokens]")
    T = ids.shape[0]
    if not isinstance(out, torch.Tensor):
        _refuse(fn, "out must be a tensor")
    a = _pack_table(*w, *dense, _type(fn, "out", out), scale, 0, T, _flat(fn, "ids", ids, torch.int64, dev, T),
                    *_rows(fn, "out", out, out.dtype, dev, (T, n)))
    _run(lib.bq_embed, a, dev, stream)


def bq_gated_q8(gate, up, act: int, qa: int, q, d, y=None, f16_scale: bool = False, stream=None) -> None:
    """act(gate) * up to 8 bits.  gate, up, y: [tokens, n] of one type; q: int8
    [tokens, n]; d: float32 [tokens, n / qa]; act: BQ_NONE, BQ_SILU, BQ_GELU or
    BQ_RELU2.  y receives the values; it may be gate or up."""
    fn = "bq_gated_q8"
    dev = _first(fn, "gate", gate)
    shape = T, n = _matrix(fn, "gate", gate)
    kind, dt = _type(fn, "gate", gate), gate.dtype
    a = _pack_gated(kind, act, qa, int(f16_scale), T, n, *_rows(fn, "gate", gate, dt, dev, shape),
                    *_rows(fn, "up", up, dt, dev, shape), *_rows(fn, "q", q, torch.int8, dev, shape),
                    *_rows(fn, "d", d, torch.float32, dev, (T, n // qa if qa > 0 else 0)),
                    *((0, 0) if y is None else _rows(fn, "y", y, dt, dev, shape)))
    _run(lib.bq_gated_q8, a, dev, stream)


@functools.lru_cache(maxsize=1024)
def _matmul_work(fmt, rows, cols, qa, tokens, kind) -> int:
    need = _i64()
    _check(lib.bq_matmul_work_bytes(_pack_product(fmt, 0, rows, cols, 0, 0, 0, 0, cols, qa, tokens, 0, 0, kind, 0, *[0] * 9),
                                    ctypes.byref(need)))
    return need.value


def bq_matmul(w: Weights, a: Act, y, bias=None, act: int = BQ_NONE, mul=None, res=None, work=None, stream=None) -> None:
    """y = act(W x + bias) * mul + res for the a.ncols tokens of a.  y, mul,
    res: [tokens, rows] of one type; bias: float32 [rows].  y may be mul or
    res.  work: scratch of at least bq_matmul_work_bytes(...) bytes, by default
    a tensor of the call's own (calls that may run at the same time must not
    share one)."""
    fn = "bq_matmul"
    planes, dev = _planes(fn, w)
    if a.q.get_device() != dev or a.d.get_device() != dev:
        _refuse(fn, f"the activations must be on device {dev}")
    dt, kind = (y.dtype, _type(fn, "y", y)) if isinstance(y, torch.Tensor) else (None, 0)
    T = a.ncols
    shape = (T, w.rows)
    yp = _rows(fn, "y", y, dt, dev, shape)
    need = _matmul_work(w.fmt, w.rows, w.cols, a.qa, T, kind)
    wp, size, keep = _work_of(fn, work, need, dev, stream)
    ld_q, ld_d = a._ld()
    p = _pack_product(*planes, a.q.data_ptr(), a.d.data_ptr(), a.n, a.qa, T, ld_q, ld_d, kind, act,
                      0 if bias is None else _flat(fn, "bias", bias, torch.float32, dev, w.rows),
                      *((0, 0) if mul is None else _rows(fn, "mul", mul, dt, dev, shape)),
                      *((0, 0) if res is None else _rows(fn, "res", res, dt, dev, shape)), *yp, wp, size)
    _run(lib.bq_matmul, p, dev, stream)


def bq_matmul_work_bytes(w: Weights, tokens: int, qa: int, y_type=torch.float32) -> int:
    """Bytes of scratch that bq_matmul needs for these sizes."""
    return _matmul_work(w.fmt, w.rows, w.cols, qa, tokens, TYPES[y_type])


@functools.lru_cache(maxsize=1024)
def _sample_work(kind, rows, vocab) -> int:
    need = _i64()
    _check(lib.bq_sample_work_bytes(_pack_draw(kind, 0, rows, vocab, *[0] * 11), ctypes.byref(need)))
    return need.value


def bq_sample(logits, u, token, logprob=None, temperature=None, top_k=None, top_p=None, min_p=None, work=None,
              stream=None) -> None:
    """The next token of each row.  logits: [rows, vocab]; u: float32 [rows] in
    [0, 1); token: int64 [rows]; logprob: float32 [rows]; temperature, top_p,
    min_p: float32 [rows], top_k: int32 [rows] (None: 1, no filter).  work:
    scratch of at least bq_sample_work_bytes(...) bytes, by default a tensor of
    the call's own (calls that may run at the same time must not share one)."""
    fn = "bq_sample"
    dev = _first(fn, "logits", logits)
    B, V = _matrix(fn, "logits", logits)
    kind = _type(fn, "logits", logits)
    p = _rows(fn, "logits", logits, logits.dtype, dev, (B, V))

    def each(what, t, dtype=torch.float32):
        return 0 if t is None else _flat(fn, what, t, dtype, dev, B)

    if u is None or token is None:
        _refuse(fn, "u and token must be tensors")
    wp, size, keep = _work_of(fn, work, _sample_work(kind, B, V), dev, stream)
    a = _pack_draw(kind, 0, B, V, *p, each("u", u), each("temperature", temperature), each("top_k", top_k, torch.int32),
                   each("top_p", top_p), each("min_p", min_p), each("token", token, torch.int64), each("logprob", logprob),
                   wp, size)
    _run(lib.bq_sample, a, dev, stream)


def bq_sample_work_bytes(rows: int, vocab: int, logits_type=torch.float32) -> int:
    """Bytes of scratch that bq_sample needs for these sizes."""
    return _sample_work(TYPES[logits_type], rows, vocab)
