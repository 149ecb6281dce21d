"""Scratch of bq_matmul for matrices of few rows: none, as their products take the
kernel without laid-out activations, however many tokens there are."""
import ctypes

import pytest

import ternary_quantized_gemv_amd as bq
from ternary_quantized_gemv_amd import layer as L
from ternary_quantized_gemv_amd import model as M


@pytest.mark.parametrize("fmt,qa", [(1, 32), (1, 128), (2, 32), (2, 64), (2, 128)])
def test_few_rows(fmt, qa):
    need = ctypes.c_int64(-1)
    for rows, some in ((1, False), (40, False), (64, False), (257, True), (4096, True)):
        a = M.bq_product(bq.bq_weights(fmt, 0, rows, 4096, None, None), bq.bq_act(None, None, 4096, qa, 100000, 4096, 4096 // qa),
                         L.BQ_F32, bq.BQ_NONE)
        assert bq.lib.bq_matmul_work_bytes(ctypes.byref(a), ctypes.byref(need)) == bq.BQ_OK
        assert (need.value > 0) == some, rows
