"""Python binding of the operators between the products (include/bq.h):
bq_rmsnorm_q8, bq_kv_append, bq_paged_attn and bq_adapters_add.

As in the rest of the package the functions keep the C names and only marshal
arguments: shapes, types, strides and devices are checked against each other
here (the library takes bare pointers), everything else by the library.  A
call runs on the device of its tensors, whichever is current, and on `stream`
(default: the current stream of that device).
"""
from __future__ import annotations

import ctypes
import functools
import struct as _struct

import torch

from . import BQ_EARG, BQError, lib

BQ_F32, BQ_F16, BQ_BF16 = 0, 1, 2
BQ_NORM_MAX = 65536
TYPES = {torch.float32: BQ_F32, torch.float16: BQ_F16, torch.bfloat16: BQ_BF16}

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class bq_norm(ctypes.Structure):
    _fields_ = [("type", _i32), ("qa", _i32), ("f16_scale", _i32), ("reserved", _i32), ("eps", ctypes.c_double),
                ("tokens", _i64), ("n", _i64),
                ("x", _vp), ("ld_x", _i64), ("res", _vp), ("ld_res", _i64), ("h", _vp), ("ld_h", _i64), ("w", _vp),
                ("q", _vp), ("ld_q", _i64), ("d", _vp), ("ld_d", _i64), ("y", _vp), ("ld_y", _i64)]


class bq_kv_cache(ctypes.Structure):
    _fields_ = [("type", _i32), ("heads", _i32), ("dim", _i32), ("page", _i32), ("pages", _i64), ("k", _vp), ("v", _vp)]


class bq_append(ctypes.Structure):
    _fields_ = [("cache", bq_kv_cache), ("type", _i32), ("q_out_type", _i32), ("q_heads", _i32), ("rot", _i32),
                ("eps", _f32), ("reserved", _i32), ("tokens", _i64), ("q", _vp), ("ld_q", _i64), ("k", _vp),
                ("ld_k", _i64), ("v", _vp), ("ld_v", _i64), ("q_out", _vp), ("ld_qo", _i64), ("pos", _vp),
                ("slot", _vp), ("freq", _vp), ("q_norm", _vp), ("k_norm", _vp)]


class bq_attn(ctypes.Structure):
    _fields_ = [("cache", bq_kv_cache), ("type", _i32), ("q_heads", _i32), ("requests", _i32), ("table_cols", _i32),
                ("ld_table", _i64), ("tokens", _i64), ("max_new", _i64), ("max_keys", _i64), ("q", _vp), ("ld_q", _i64),
                ("out", _vp), ("ld_out", _i64), ("cu", _vp), ("lens", _vp), ("table", _vp), ("scale", _f32),
                ("reserved", _i32), ("work", _vp), ("work_bytes", _i64)]


class bq_adapters(ctypes.Structure):
    _fields_ = [("type", _i32), ("x_type", _i32), ("rank", _i32), ("count", _i32), ("requests", _i32),
                ("reserved", _i32), ("n", _i64), ("rows", _i64), ("tokens", _i64), ("max_new", _i64), ("a", _vp),
                ("b", _vp), ("gain", _vp), ("x", _vp), ("ld_x", _i64), ("cu", _vp), ("ids", _vp), ("y", _vp),
                ("ld_y", _i64), ("out", _vp), ("ld_out", _i64), ("work", _vp), ("work_bytes", _i64)]


def _format(struct) -> str:
    """The struct module's format of a ctypes structure (nested ones flattened)."""
    codes = {_i32: "i", _i64: "q", _f32: "f", ctypes.c_double: "d", _vp: "P"}
    return "".join(codes[t] if t in codes else _format(t) for _, t in struct._fields_)


class _Pack:
    """Packs an argument block in one go: several times faster than filling the
    ctypes structure, whose layout it has (native alignment, eight-byte end)."""

    def __init__(self, struct):
        self.pack = _struct.Struct("@" + _format(struct) + "0q").pack
        assert len(self.pack(*[0] * len(_format(struct)))) == ctypes.sizeof(struct)


_pack_norm, _pack_append, _pack_attn, _pack_adapters = (_Pack(k).pack for k in (bq_norm, bq_append, bq_attn, bq_adapters))

for _name in ("bq_rmsnorm_q8", "bq_kv_append", "bq_paged_attn", "bq_adapters_add"):
    getattr(lib, _name).restype = ctypes.c_int
    getattr(lib, _name).argtypes = [_vp, _vp]
for _name in ("bq_paged_attn_work_bytes", "bq_adapters_work_bytes"):
    getattr(lib, _name).restype = ctypes.c_int
    getattr(lib, _name).argtypes = [_vp, _vp]


# ------------------------------------------------------------------ checks
def _refuse(fn: str, text: str):
    raise BQError(BQ_EARG, f"{fn}: {text}")


def _check(rc: int):
    if rc:
        raise BQError(rc, lib.bq_last_error().decode())


def _first(fn: str, what: str, t) -> int:
    """The index of the device that the call runs on, from the tensor that says so."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _refuse(fn, f"{what} must be a tensor on a ROCm device")
    return t.get_device()


def _type(fn: str, what: str, t) -> int:
    k = TYPES.get(t.dtype)
    if k is None:
        _refuse(fn, f"{what} must be float32, float16 or bfloat16, not {t.dtype}")
    return k


def _tensor(fn: str, what: str, t, dtype, dev: int):
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _refuse(fn, f"{what} must be a tensor on device {dev}")
    if t.dtype is not dtype:
        _refuse(fn, f"{what} must be {dtype}, not {t.dtype}")


def _rows(fn: str, what: str, t, dtype, dev: int, shape):
    """(pointer, elements between rows) of a tensor of this shape whose rows
    (all dimensions but the first) are contiguous; a single row may come
    without its first dimension."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr(), t.stride(0)
    _tensor(fn, what, t, dtype, dev)
    have, stride = t.shape, t.stride()
    if len(have) == len(shape) - 1 and shape[0] == 1:
        have, stride = (1, *have), (0, *stride)
    if tuple(have) != shape:
        _refuse(fn, f"{what} has shape {tuple(t.shape)}, needs {shape}")
    step = 1
    for size, st in zip(reversed(shape[1:]), reversed(stride[1:])):
        if st != step and size != 1:
            _refuse(fn, f"the rows of {what} must be contiguous")
        step *= size
    return t.data_ptr(), stride[0]


def _flat(fn: str, what: str, t, dtype, dev: int, n: int) -> int:
    """Pointer of a contiguous tensor of n values."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == n and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _tensor(fn, what, t, dtype, dev)
    _refuse(fn, f"{what} must be contiguous with {n} values, has shape {tuple(t.shape)}")


def _whole(fn: str, what: str, t, dtype, dev: int, shape) -> int:
    """Pointer of a contiguous tensor of this shape."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _tensor(fn, what, t, dtype, dev)
    _refuse(fn, f"{what} must be contiguous with shape {tuple(shape)}, has {tuple(t.shape)}")


# the stream and device lookups without the objects that torch.cuda makes of them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(call, args: bytes, dev: int, stream):
    stream = _raw_stream(dev) if stream is None else getattr(stream, "cuda_stream", stream)
    if dev == _current_device():
        _check(call(args, stream))
    else:
        with torch.cuda.device(dev):
            _check(call(args, stream))


def _scratch(fn: str, work, need: int, dev: int, stream):
    """The caller's scratch tensor, or one of this call: allocated on the
    stream that the call runs on, so that the allocator reuses it in order."""
    if work is None:
        if stream is None or not need:
            return torch.empty(need, dtype=torch.uint8, device=dev)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream, device=dev)
        with torch.cuda.stream(stream):
            return torch.empty(need, dtype=torch.uint8, device=dev)
    if not isinstance(work, torch.Tensor) or work.get_device() != dev or not work.is_contiguous():
        _refuse(fn, f"work must be a contiguous tensor on device {dev}")
    return work


# -------------------------------------------------------------- the operators
def bq_rmsnorm_q8(x, w, eps: float, qa: int, q, d, res=None, h=None, y=None, f16_scale: bool = False,
                  stream=None) -> None:
    """Residual addition, RMS norm and 8-bit activation in one pass.  x, res,
    h, y: [tokens, n] of one type; w: [n]; q: int8 [tokens, n]; d: float32
    [tokens, n / qa] (Act(q, d, n, qa, tokens) feeds them to the products).
    h receives x + res, y the normed rows; either may be x or res."""
    fn = "bq_rmsnorm_q8"
    dev = _first(fn, "x", x)
    kind, dt, shape = _type(fn, "x", x), x.dtype, x.shape
    if len(shape) == 2:
        T, n = shape
    elif len(shape) == 1:
        T, n = 1, shape[0]
    else:
        _refuse(fn, "x must be [tokens, n] or [n]")
    shape = (T, n)
    none = (0, 0)
    a = _pack_norm(kind, qa, int(f16_scale), 0, eps, T, n, *_rows(fn, "x", x, dt, dev, shape),
                   *(none if res is None else _rows(fn, "res", res, dt, dev, shape)),
                   *(none if h is None else _rows(fn, "h", h, dt, dev, shape)), _flat(fn, "w", w, dt, dev, n),
                   *_rows(fn, "q", q, torch.int8, dev, shape),
                   *_rows(fn, "d", d, torch.float32, dev, (T, n // qa if qa > 0 else 0)),
                   *(none if y is None else _rows(fn, "y", y, dt, dev, shape)))
    _run(lib.bq_rmsnorm_q8, a, dev, stream)


class KVCache:
    """A paged cache of keys [pages, heads, page, dim] and values [pages,
    heads, dim, page] (float16 or bfloat16, contiguous)."""

    def __init__(self, k, v):
        fn = "KVCache"
        self.dev = dev = _first(fn, "k", k)
        if k.dim() != 4:
            _refuse(fn, "k must be [pages, heads, page, dim]")
        self.pages, self.heads, self.page, self.dim = pages, heads, page, dim = k.shape
        dt = k.dtype
        self.k, self.v = k, v
        self.c = (_type(fn, "k", k), heads, dim, page, pages, _whole(fn, "k", k, dt, dev, k.shape),
                  _whole(fn, "v", v, dt, dev, (pages, heads, dim, page)))

    @classmethod
    def empty(cls, pages: int, heads: int, dim: int, page: int = 64, dtype=torch.bfloat16, device="cuda"):
        return cls(torch.empty(pages, heads, page, dim, dtype=dtype, device=device),
                   torch.empty(pages, heads, dim, page, dtype=dtype, device=device))


def bq_kv_append(cache: KVCache, k, v, pos, slot, freq, q=None, q_out=None, q_norm=None, k_norm=None,
                 eps: float = 1e-6, stream=None) -> None:
    """New tokens into the cache.  k, v: [tokens, heads, dim] and q, q_out:
    [tokens, q_heads, dim] (float32 or the cache's type; q_out either); pos:
    int32 [tokens]; slot: int64 [tokens], place of each token in the cache
    (page * page size + offset) or -1; freq: float32 [rot / 2]; q_norm,
    k_norm: float32 [dim].  The rotated queries go to q_out (q itself allowed)."""
    fn = "bq_kv_append"
    dev, c = cache.dev, cache
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        _refuse(fn, "k must be [tokens, heads, dim]")
    dt, T = k.dtype, k.shape[0]
    shape = (T, c.heads, c.dim)
    kind = _type(fn, "k", k)
    Hq = 0
    qp = qo = (0, 0)
    out_kind = kind
    if (q is None) != (q_out is None):
        _refuse(fn, "q and q_out come together")
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3 or not isinstance(q_out, torch.Tensor):
            _refuse(fn, "q and q_out must be [tokens, q_heads, dim]")
        Hq = q.shape[1]
        qp = _rows(fn, "q", q, dt, dev, (T, Hq, c.dim))
        out_kind = _type(fn, "q_out", q_out)
        qo = _rows(fn, "q_out", q_out, q_out.dtype, dev, (T, Hq, c.dim))
    if not isinstance(freq, torch.Tensor):
        _refuse(fn, "freq must be a tensor")
    half = freq.numel()
    a = _pack_append(*c.c, kind, out_kind, Hq, 2 * half, eps, 0, T, *qp, *_rows(fn, "k", k, dt, dev, shape),
                     *_rows(fn, "v", v, dt, dev, shape), *qo, _flat(fn, "pos", pos, torch.int32, dev, T),
                     _flat(fn, "slot", slot, torch.int64, dev, T), _flat(fn, "freq", freq, torch.float32, dev, half),
                     0 if q_norm is None else _flat(fn, "q_norm", q_norm, torch.float32, dev, c.dim),
                     0 if k_norm is None else _flat(fn, "k_norm", k_norm, torch.float32, dev, c.dim))
    _run(lib.bq_kv_append, a, dev, stream)


@functools.lru_cache(maxsize=1024)
def _attn_work(cache_sizes, kind, q_heads, requests, tokens, max_new, max_keys) -> int:
    need = _i64()
    _check(lib.bq_paged_attn_work_bytes(
        _pack_attn(*cache_sizes, 0, 0, kind, q_heads, requests, 1, 1, tokens, max_new, max_keys, *[0] * 7, 0.0, *[0] * 3),
        ctypes.byref(need)))
    return need.value


def bq_paged_attn(cache: KVCache, q, cu, lens, table, scale: float, max_new: int, max_keys: int, out, work=None,
                  stream=None) -> None:
    """Causal attention of the new tokens of several requests over the cache.
    q, out: [tokens, q_heads, dim] (float32 or the cache's type); cu: int32
    [requests + 1], lens: int32 [requests], table: int32 [requests, pages of a
    request]; max_new, max_keys: bounds for any request.  work: scratch of at
    least bq_paged_attn_work_bytes(...) bytes, by default a tensor of the call's
    own (calls that may run at the same time must not share one)."""
    fn = "bq_paged_attn"
    dev, c = cache.dev, cache
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        _refuse(fn, "q must be [tokens, q_heads, dim]")
    if not isinstance(lens, torch.Tensor) or lens.dim() != 1:
        _refuse(fn, "lens must be [requests]")
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        _refuse(fn, "table must be [requests, pages of a request]")
    dt, kind, B = q.dtype, _type(fn, "q", q), lens.shape[0]
    shape = (q.shape[0], q.shape[1], c.dim)
    cols = table.shape[1]
    tp, ld_table = _rows(fn, "table", table, torch.int32, dev, (B, cols))
    need = _attn_work(c.c[:5], kind, shape[1], B, shape[0], max_new, max_keys)
    work = _scratch(fn, work, need, dev, stream)
    a = _pack_attn(*c.c, kind, shape[1], B, cols, ld_table, shape[0], max_new, max_keys,
                   *_rows(fn, "q", q, dt, dev, shape), *_rows(fn, "out", out, dt, dev, shape),
                   _flat(fn, "cu", cu, torch.int32, dev, B + 1), _flat(fn, "lens", lens, torch.int32, dev, B), tp, scale,
                   0, work.data_ptr(), work.nbytes)
    _run(lib.bq_paged_attn, a, dev, stream)


def bq_paged_attn_work_bytes(cache: KVCache, tokens: int, q_heads: int, requests: int, max_new: int, max_keys: int,
                             q_type=torch.float32) -> int:
    """Bytes of scratch that bq_paged_attn needs for these sizes (tables of
    any width)."""
    return _attn_work(cache.c[:5], TYPES[q_type], q_heads, requests, tokens, max_new, max_keys)


class Adapters:
    """Low-rank adapters of one projection: a [count, rank, n], b [count,
    rows, rank] (float16 or bfloat16, contiguous), gain float32 [count]."""

    def __init__(self, a, b, gain):
        fn = "Adapters"
        self.dev = dev = _first(fn, "a", a)
        if a.dim() != 3 or not isinstance(b, torch.Tensor) or b.dim() != 3:
            _refuse(fn, "a must be [count, rank, n] and b [count, rows, rank]")
        self.count, self.rank, self.n = count, rank, n = a.shape
        self.rows = rows = b.shape[1]
        dt = a.dtype
        self.pointers = (_whole(fn, "a", a, dt, dev, a.shape), _whole(fn, "b", b, dt, dev, (count, rows, rank)),
                         _flat(fn, "gain", gain, torch.float32, dev, count))
        self.a, self.b, self.gain = a, b, gain
        self.type = _type(fn, "a", a)


@functools.lru_cache(maxsize=1024)
def _adapters_work(kind, x_kind, rank, count, requests, n, rows, tokens, max_new) -> int:
    need = _i64()
    _check(lib.bq_adapters_work_bytes(
        _pack_adapters(kind, x_kind, rank, count, requests, 0, n, rows, tokens, max_new, *[0] * 13), ctypes.byref(need)))
    return need.value


def bq_adapters_add(adapters: Adapters, x, cu, ids, max_new: int, y, out=None, work=None, stream=None) -> None:
    """out = y + gain B (A x), each request with its adapter.  x: [tokens, n]
    (float32 or the adapters' type); y, out: float32 [tokens, rows] (out
    defaults to y: in place); cu: int32 [requests + 1]; ids: int32 [requests],
    -1 for none; max_new: bound for the tokens of any request.  work: scratch
    of at least bq_adapters_work_bytes(...) bytes, by default a tensor of the
    call's own."""
    fn = "bq_adapters_add"
    p, dev = adapters, adapters.dev
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        _refuse(fn, "x must be [tokens, n]")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 1:
        _refuse(fn, "ids must be [requests]")
    T, B, kind = x.shape[0], ids.shape[0], _type(fn, "x", x)
    sizes = (p.type, kind, p.rank, p.count, B)
    work = _scratch(fn, work, _adapters_work(*sizes, p.n, p.rows, T, max_new), dev, stream)
    yp = _rows(fn, "y", y, torch.float32, dev, (T, p.rows))
    a = _pack_adapters(*sizes, 0, p.n, p.rows, T, max_new, *p.pointers, *_rows(fn, "x", x, x.dtype, dev, (T, p.n)),
                       _flat(fn, "cu", cu, torch.int32, dev, B + 1), _flat(fn, "ids", ids, torch.int32, dev, B), *yp,
                       *(yp if out is None else _rows(fn, "out", out, torch.float32, dev, (T, p.rows))), work.data_ptr(),
                       work.nbytes)
    _run(lib.bq_adapters_add, a, dev, stream)


def bq_adapters_work_bytes(adapters: Adapters, tokens: int, requests: int, max_new: int, x_type=torch.float32) -> int:
    """Bytes of scratch that bq_adapters_add needs for these sizes."""
    p = adapters
    return _adapters_work(p.type, TYPES[x_type], p.rank, p.count, requests, p.n, p.rows, tokens, max_new)
