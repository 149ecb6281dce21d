"""Row lengths past what a tile of 64 packed rows may hold: refused by bq_matmul,
and by the call that sizes its scratch."""
import ctypes

import pytest

import ternary_quantized_gemv_amd as bq
from ternary_quantized_gemv_amd import layer as L
from ternary_quantized_gemv_amd import model as M

P = 0x10000


@pytest.mark.parametrize("fmt,last", [(1, 268435328), (2, 134217664)])
def test_longest_rows(fmt, last):
    need = ctypes.c_int64(-1)
    step = 128 if fmt == 1 else 64
    for cols, fits in ((last, True), (last + step, False), ((1 << 31) - step, False)):
        a = M.bq_product(bq.bq_weights(fmt, 0, 100, cols, P, P), bq.bq_act(P, P, cols, 64, 3, cols, cols // 64), L.BQ_F32,
                         bq.BQ_NONE, None, None, 0, None, 0, P, 100, P, 1 << 40)
        rc = bq.lib.bq_matmul_work_bytes(ctypes.byref(a), ctypes.byref(need))
        assert rc == (bq.BQ_OK if fits else bq.BQ_EARG), (cols, bq.bq_last_error())
        if not fits:
            assert "payload" in bq.bq_last_error()
            assert bq.lib.bq_matmul(ctypes.byref(a), None) == bq.BQ_EARG and "payload" in bq.bq_last_error()
    t = M.bq_table(bq.bq_weights(fmt, 0, 100, last + step, P, P), None, 0, 0, L.BQ_F32, 1.0, 0, 3, P, P, last + step)
    assert bq.lib.bq_embed(ctypes.byref(t), None) == bq.BQ_EARG and "payload" in bq.bq_last_error()
