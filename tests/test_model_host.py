"""Argument checks of the operators around the layers, without a GPU: bad
arguments are refused on the host before anything is launched, scratch sizes
are host arithmetic, and nothing is done for no tokens."""
import ctypes

import pytest
import torch

import ternary_quantized_gemv_amd as bq
from ternary_quantized_gemv_amd import layer as L
from ternary_quantized_gemv_amd import model as M

P = 0x10000
ROOM = 1 << 40  # bytes of scratch, enough for any


def set_all(a, k):
    for name, v in k.items():
        at = a
        *path, last = name.split(".")
        for p in path:
            at = getattr(at, p)
        setattr(at, last, v)
    return a


def packed_table(**k):
    return set_all(M.bq_table(bq.bq_weights(1, 0, 100, 256, P, P), None, 0, 0, L.BQ_F32, 2.0, 0, 3, P, P, 256), k)


def dense_table(**k):
    return set_all(M.bq_table(bq.bq_weights(0, 0, 100, 256, None, None), P, 256, L.BQ_BF16, L.BQ_F32, 2.0, 0, 3, P, P, 256), k)


def gated(**k):
    return set_all(M.bq_gated(L.BQ_F32, bq.BQ_SILU, 128, 0, 3, 256, P, 256, P, 256, P, 256, P, 2, P * 2, 256), k)


def product(**k):
    return set_all(M.bq_product(bq.bq_weights(2, 0, 100, 256, P, P), bq.bq_act(P, P, 256, 128, 300, 256, 2), L.BQ_F32,
                                bq.BQ_GELU, P, P, 100, P, 100, 2 * P, 100, P, ROOM), k)


def draw(**k):
    return set_all(M.bq_draw(L.BQ_F32, 0, 3, 1000, P, 1000, P, P, P, P, P, P, P, P, ROOM), k)


def rc_of(fn, a):
    return getattr(bq.lib, fn)(ctypes.byref(a), None)


CASES = [
    ("bq_embed", packed_table, "tokens", [
        ("type", 3), ("reserved", 1), ("scale", float("inf")), ("scale", float("nan")), ("tokens", -1), ("tokens", 1 << 31),
        ("w.fmt", 3), ("w.fmt", -1), ("w.reserved", 1), ("w.rows", 0), ("w.rows", 1 << 31), ("w.cols", 192), ("w.cols", 0),
        ("w.bits", None), ("w.scales", None), ("dense", P), ("ld_dense", 256), ("dense_type", 1), ("ids", None),
        ("out", None), ("ld_out", 255), ("ld_out", 1 << 41), ("w.fmt", 0)], [
        ("w.bits", P + 8), ("w.scales", P + 2), ("ids", P + 4), ("out", P + 4), ("ld_out", 258)]),
    ("bq_embed", dense_table, "tokens", [
        ("dense_type", 3), ("dense", None), ("ld_dense", 128), ("w.rows", 0), ("w.rows", 1 << 31), ("w.cols", 252),
        ("w.cols", 0), ("w.bits", P), ("w.scales", P), ("w.reserved", 1)], [
        ("dense", P + 2), ("ld_dense", 260)]),
    ("bq_gated_q8", gated, "tokens", [
        ("type", 3), ("act", 4), ("act", -1), ("qa", 48), ("f16_scale", 2), ("tokens", -1), ("tokens", 1 << 31), ("n", 0),
        ("n", 200), ("n", 1 << 31), ("gate", None), ("up", None), ("q", None), ("d", None), ("ld_gate", 255), ("ld_up", 128),
        ("ld_y", 1), ("ld_q", 240), ("ld_d", 1), ("ld_q", 1 << 41)], [
        ("gate", P + 4), ("up", P + 8), ("y", P + 4), ("q", P + 4), ("d", P + 2), ("ld_gate", 258), ("ld_q", 264)]),
    ("bq_matmul", product, "a.ncols", [
        ("w.fmt", 0), ("w.fmt", 3), ("w.reserved", 1), ("w.rows", 0), ("w.rows", 1 << 31), ("w.cols", 128), ("w.cols", 160),
        ("w.bits", None), ("w.scales", None), ("type", 3), ("act", 4), ("act", -1), ("a.ncols", -1),
        ("a.ncols", (1 << 31) - 1), ("a.qa", 48), ("a.q", None), ("a.d", None), ("a.n", 128), ("a.ld_q", 240), ("a.ld_d", 1),
        ("a.ld_q", 1 << 41), ("y", None), ("ld_y", 99), ("ld_mul", 99), ("ld_res", 99), ("ld_y", 1 << 41)], [
        ("w.bits", P + 8), ("a.q", P + 8), ("a.ld_q", 264), ("a.d", P + 2), ("y", P + 2), ("mul", P + 2), ("res", P + 1),
        ("bias", P + 2)]),
    ("bq_sample", draw, "rows", [
        ("type", 3), ("reserved", 1), ("rows", -1), ("rows", 1 << 31), ("vocab", 0), ("vocab", (1 << 22) + 1), ("logits", None),
        ("ld_logits", 999), ("ld_logits", 1 << 41), ("u", None), ("token", None)], [
        ("logits", P + 2), ("u", P + 2), ("temperature", P + 1), ("top_k", P + 2), ("top_p", P + 2), ("min_p", P + 2),
        ("token", P + 4), ("logprob", P + 2)]),
]


@pytest.mark.parametrize("fn,make,count,wrong,misaligned", CASES, ids=[c[1].__name__ for c in CASES])
def test_refused_on_the_host(fn, make, count, wrong, misaligned):
    for code, cases in ((bq.BQ_EARG, wrong), (bq.BQ_EALIGN, misaligned)):
        for name, value in cases:
            assert rc_of(fn, make(**{name: value})) == code, (name, value, bq.bq_last_error())
            assert bq.bq_last_error().startswith(fn + ":"), (name, value)
    assert getattr(bq.lib, fn)(None, None) == bq.BQ_EARG
    assert rc_of(fn, make(**{count: 0})) == bq.BQ_OK  # nothing to do


def test_aliases():
    assert rc_of("bq_gated_q8", gated(y=P, ld_y=512)) == bq.BQ_EARG
    assert rc_of("bq_gated_q8", gated(gate=3 * P, y=P, ld_y=512)) == bq.BQ_EARG
    assert rc_of("bq_matmul", product(y=P, ld_y=128)) == bq.BQ_EARG
    assert rc_of("bq_matmul", product(mul=None, y=P, ld_y=128)) == bq.BQ_EARG


def test_scratch_sizes():
    need = ctypes.c_int64(-1)
    for fn, make, count in (("bq_matmul", product, "a.ncols"), ("bq_sample", draw, "rows")):
        size = getattr(bq.lib, fn + "_work_bytes")
        last = 0
        for n in (0, 1, 16, 100, 1000, 10000):
            a = make(**{count: n})
            assert size(ctypes.byref(a), ctypes.byref(need)) == bq.BQ_OK and need.value >= 0
            assert n or need.value == 0
            if fn == "bq_matmul":  # what serves many tokens serves fewer
                assert need.value >= last
                last = need.value
            if need.value:
                a.work_bytes = need.value - 1
                assert rc_of(fn, a) == bq.BQ_EARG and "work" in bq.bq_last_error()
                a.work_bytes, a.work = need.value, None
                assert rc_of(fn, a) == bq.BQ_EARG and "work" in bq.bq_last_error()
                a.work = P + 8
                assert rc_of(fn, a) == bq.BQ_EALIGN
        assert size(ctypes.byref(make(type=3)), ctypes.byref(need)) == bq.BQ_EARG
        assert size(ctypes.byref(make()), None) == bq.BQ_EARG and size(None, ctypes.byref(need)) == bq.BQ_EARG


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 256)
    one = torch.zeros(2)
    with pytest.raises(bq.BQError):
        bq.bq_embed(x, torch.zeros(2, dtype=torch.int64), x)
    with pytest.raises(bq.BQError):
        bq.bq_gated_q8(x, x, bq.BQ_SILU, 128, x.char(), x[:, :2])
    with pytest.raises(bq.BQError):
        bq.bq_sample(x, one, one.long())


def test_structs_have_the_headers_layout():
    """Sizes of the argument blocks as a C compiler lays them out."""
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = ("bq_table", "bq_gated", "bq_product", "bq_draw")
    body = "".join(f'printf("%zu ", sizeof({n}));' for n in names)
    body += "".join(f'printf("%zu ", offsetof({n}, {f}));' for n in names for f, _ in getattr(M, n)._fields_)
    with tempfile.TemporaryDirectory() as d:
        src = os.path.join(d, "s.c")
        with open(src, "w") as f:
            f.write(f'#include <stdio.h>\n#include "bq.h"\nint main(void) {{ {body} return 0; }}\n')
        exe = os.path.join(d, "s")
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), src, "-o", exe], check=True)
        got = [int(v) for v in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    want = [ctypes.sizeof(getattr(M, n)) for n in names]
    want += [getattr(getattr(M, n), f).offset for n in names for f, _ in getattr(M, n)._fields_]
    assert got == want
