"""Argument checks of the operators between the products, without a GPU: bad
arguments are refused on the host before anything is launched, scratch sizes
are host arithmetic, and nothing is done for no tokens."""
import ctypes

import pytest
import torch

import ternary_quantized_gemv_amd as bq
from ternary_quantized_gemv_amd import layer as L

P = 0x10000


def norm(**k):
    a = L.bq_norm(L.BQ_F32, 128, 0, 0, 1e-6, 2, 256, P, 256, P, 256, P, 256, P, P, 256, P, 2, None, 0)
    for n, v in k.items():
        setattr(a, n, v)
    return a


def cache(**k):
    c = L.bq_kv_cache(L.BQ_BF16, 2, 64, 16, 4, P, P)
    for n, v in k.items():
        setattr(c, n, v)
    return c


def append(c=None, **k):
    a = L.bq_append(c or cache(), L.BQ_F32, L.BQ_F32, 4, 64, 1e-6, 0, 3, P, 256, P, 128, P, 128, 2 * P, 256, P, P, P,
                    None, None)
    for n, v in k.items():
        setattr(a, n, v)
    return a


def attn(c=None, **k):
    a = L.bq_attn(c or cache(), L.BQ_F32, 4, 2, 4, 4, 3, 2, 64, P, 256, 2 * P, 256, P, P, P, 0.125, 0, P, 1 << 20)
    for n, v in k.items():
        setattr(a, n, v)
    return a


def adapters(**k):
    a = L.bq_adapters(L.BQ_F16, L.BQ_F32, 16, 2, 2, 0, 256, 100, 3, 2, P, P, P, P, 256, P, P, P, 100, P, 100, P, 1 << 20)
    for n, v in k.items():
        setattr(a, n, v)
    return a


def rc_of(fn, a):
    return getattr(bq.lib, fn)(ctypes.byref(a), None)


CASES = [
    ("bq_rmsnorm_q8", norm, [
        ("type", 3), ("qa", 48), ("f16_scale", 2), ("reserved", 1), ("eps", 0.0), ("eps", 1e-31), ("eps", float("inf")), ("eps", float("nan")),
        ("tokens", -1), ("tokens", 1 << 31), ("n", 0), ("n", 200), ("n", 65536 + 128), ("x", None), ("w", None),
        ("q", None), ("d", None), ("ld_x", 255), ("ld_x", 1 << 41), ("ld_res", 128), ("ld_h", 0), ("ld_q", 240),
        ("ld_d", 1)], [
        ("x", P + 4), ("res", P + 8), ("h", P + 4), ("w", P + 4), ("q", P + 4), ("d", P + 2), ("ld_x", 258),
        ("ld_q", 264)]),
    ("bq_kv_append", append, [
        ("type", L.BQ_F16), ("q_out_type", L.BQ_F16), ("q_heads", -1), ("q_heads", 1025), ("rot", 24), ("rot", 128),
        ("rot", -16), ("reserved", 1), ("tokens", -1), ("tokens", 1 << 31), ("q", None), ("k", None), ("v", None),
        ("q_out", None), ("pos", None), ("slot", None), ("freq", None), ("ld_k", 64), ("ld_q", 128), ("ld_v", 1),
        ("ld_qo", 64), ("q_heads", 0)], [
        ("q", P + 4), ("k", P + 8), ("v", P + 4), ("q_out", P + 4), ("pos", P + 2), ("slot", P + 4), ("freq", P + 1),
        ("q_norm", P + 2), ("ld_k", 130)]),
    ("bq_paged_attn", attn, [
        ("type", L.BQ_F16), ("type", 7), ("q_heads", 3), ("q_heads", 0), ("q_heads", 34), ("requests", -1),
        ("requests", 65536), ("table_cols", 0), ("table_cols", 1 << 28), ("tokens", -1), ("tokens", 1 << 30),
        ("max_new", 0), ("max_new", 1 << 31), ("max_keys", -1), ("max_keys", 1 << 31), ("reserved", 1), ("q", None),
        ("out", None), ("cu", None), ("lens", None), ("table", None), ("ld_table", 3), ("ld_q", 128), ("ld_out", 1),
        ("scale", float("nan"))], [
        ("q", P + 4), ("out", P + 8), ("cu", P + 2), ("lens", P + 1), ("table", P + 2), ("ld_q", 258)]),
    ("bq_adapters_add", adapters, [
        ("type", L.BQ_F32), ("x_type", L.BQ_BF16), ("rank", 0), ("rank", 12), ("rank", 136), ("count", 0),
        ("requests", -1), ("requests", (1 << 30) + 1), ("reserved", 1), ("n", 0), ("n", 12), ("rows", 0), ("rows", 1 << 23), ("tokens", -1),
        ("max_new", 0), ("a", None), ("b", None), ("gain", None), ("x", None), ("cu", None), ("ids", None), ("y", None),
        ("out", None), ("ld_x", 128), ("ld_y", 99), ("ld_out", 99), ("ld_out", 104), ("work", None), ("work_bytes", 16)], [
        ("a", P + 8), ("b", P + 2), ("gain", P + 2), ("x", P + 4), ("cu", P + 1), ("ids", P + 2), ("y", P + 1),
        ("work", P + 4), ("ld_x", 258)]),
]


@pytest.mark.parametrize("fn,make,wrong,misaligned", CASES, ids=[c[0] for c in CASES])
def test_refused_on_the_host(fn, make, wrong, misaligned):
    for code, cases in ((bq.BQ_EARG, wrong), (bq.BQ_EALIGN, misaligned)):
        for name, value in cases:
            assert rc_of(fn, make(**{name: value})) == code, (name, value, bq.bq_last_error())
            assert bq.bq_last_error().startswith(fn + ":"), (name, value)
    assert getattr(bq.lib, fn)(None, None) == bq.BQ_EARG
    assert rc_of(fn, make(tokens=0)) == bq.BQ_OK  # nothing to do


@pytest.mark.parametrize("make,fn", [(append, "bq_kv_append"), (attn, "bq_paged_attn")])
@pytest.mark.parametrize("field,value,code", [
    ("type", L.BQ_F32, 1), ("heads", 0, 1), ("heads", 1025, 1), ("dim", 96, 1), ("page", 8, 1), ("page", 24, 1),
    ("page", 512, 1), ("pages", 0, 1), ("pages", 1 << 27, 1), ("k", None, 1), ("v", None, 1), ("k", P + 8, 2),
    ("v", P + 2, 2)])
def test_bad_caches(make, fn, field, value, code):
    assert rc_of(fn, make(cache(**{field: value}))) == code, bq.bq_last_error()


def test_aliases():
    assert rc_of("bq_rmsnorm_q8", norm(x=P, h=P, ld_h=512)) == bq.BQ_EARG
    assert rc_of("bq_rmsnorm_q8", norm(res=2 * P, y=2 * P, ld_y=512, h=None)) == bq.BQ_EARG
    assert rc_of("bq_rmsnorm_q8", norm(h=3 * P, y=3 * P, ld_y=256)) == bq.BQ_EARG
    assert rc_of("bq_kv_append", append(q_out=P, ld_qo=512)) == bq.BQ_EARG
    assert rc_of("bq_kv_append", append(q_out=P, q_out_type=L.BQ_BF16)) == bq.BQ_EARG
    assert rc_of("bq_paged_attn", attn(out=P)) == bq.BQ_EARG


def test_norm_eps_needed_with_weights_only():
    assert rc_of("bq_kv_append", append(k_norm=P, eps=0.0)) == bq.BQ_EARG
    assert rc_of("bq_kv_append", append(eps=0.0, tokens=0)) == bq.BQ_OK


def test_scratch_sizes():
    need = ctypes.c_int64(-1)
    assert bq.lib.bq_paged_attn_work_bytes(ctypes.byref(attn()), ctypes.byref(need)) == bq.BQ_OK and need.value >= 0
    few = need.value
    # one short row over many keys is split: sums of 64 values, a maximum and a sum per row and piece
    assert bq.lib.bq_paged_attn_work_bytes(ctypes.byref(attn(tokens=1, requests=1, max_new=1, max_keys=100000)), ctypes.byref(need)) == bq.BQ_OK
    assert need.value > 4 * (4 * 64 + 8)
    a = attn(tokens=1, requests=1, max_new=1, max_keys=100000, work=None)
    assert rc_of("bq_paged_attn", a) == bq.BQ_EARG and "work" in bq.bq_last_error()
    a = attn(tokens=1, requests=1, max_new=1, max_keys=100000, work_bytes=need.value - 1)
    assert rc_of("bq_paged_attn", a) == bq.BQ_EARG and "work" in bq.bq_last_error()
    # however many tokens and keys, the pieces are as many as fill the GPU: tens of megabytes at most
    for tokens, requests, new, keys in ((100000, 2, 90000, 90000), (4096, 4096, 1, 1 << 20), (1 << 20, 1, 1 << 20, 1 << 20),
                                        (100000, 300, 20, 5000), (100000, 1, 20, 100000), (60000, 1000, 5000, 8000)):
        big = attn(cache(heads=8, dim=128), tokens=tokens, requests=requests, max_new=new, max_keys=keys, q_heads=32)
        assert bq.lib.bq_paged_attn_work_bytes(ctypes.byref(big), ctypes.byref(need)) == bq.BQ_OK
        assert need.value < 100 << 20, (tokens, requests, new, keys, need.value)
    assert bq.lib.bq_paged_attn_work_bytes(ctypes.byref(attn(tokens=0)), ctypes.byref(need)) == bq.BQ_OK and need.value == 0
    assert bq.lib.bq_paged_attn_work_bytes(ctypes.byref(attn()), None) == bq.BQ_EARG and few >= 0
    assert bq.lib.bq_adapters_work_bytes(ctypes.byref(adapters()), ctypes.byref(need)) == bq.BQ_OK and need.value > 0
    assert bq.lib.bq_adapters_work_bytes(ctypes.byref(adapters(rank=12)), ctypes.byref(need)) == bq.BQ_EARG
    assert bq.lib.bq_adapters_work_bytes(ctypes.byref(adapters()), None) == bq.BQ_EARG


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 256)
    with pytest.raises(bq.BQError):
        bq.bq_rmsnorm_q8(x, x[0], 1e-6, 128, x.char(), x[:, :2])
    with pytest.raises(bq.BQError):
        bq.KVCache(torch.zeros(1, 1, 16, 64, dtype=torch.half), torch.zeros(1, 1, 64, 16, dtype=torch.half))
    with pytest.raises(bq.BQError):
        bq.Adapters(torch.zeros(1, 8, 64).half(), torch.zeros(1, 64, 8).half(), torch.zeros(1))


def test_structs_have_the_headers_layout():
    """Sizes of the argument blocks as a C compiler lays them out."""
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = ("bq_norm", "bq_kv_cache", "bq_append", "bq_attn", "bq_adapters")
    body = "".join(f'printf("%zu ", sizeof({n}));' for n in names)
    body += "".join(f'printf("%zu ", offsetof({n}, {f}));' for n in names for f, _ in getattr(L, n)._fields_)
    with tempfile.TemporaryDirectory() as d:
        src = os.path.join(d, "s.c")
        with open(src, "w") as f:
            f.write(f'#include <stdio.h>\n#include "bq.h"\nint main(void) {{ {body} return 0; }}\n')
        exe = os.path.join(d, "s")
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), src, "-o", exe], check=True)
        got = [int(v) for v in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    want = [ctypes.sizeof(getattr(L, n)) for n in names]
    want += [getattr(getattr(L, n), f).offset for n in names for f, _ in getattr(L, n)._fields_]
    assert got == want
