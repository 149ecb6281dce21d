"""Sizes at the end of what the operators between the products can count."""
import ctypes

import pytest

import ternary_quantized_gemv_amd as bq
from test_layer_host import L, adapters, rc_of


@pytest.mark.parametrize("tokens,code", [((1 << 31) - 1, bq.BQ_EARG), ((1 << 31) - 32, bq.BQ_EARG), ((1 << 31) - 63, bq.BQ_EARG),
                                         ((1 << 31) - 64, bq.BQ_OK), (1 << 30, bq.BQ_OK)])
def test_adapter_tokens(tokens, code):
    """A tile of 32 rows that starts inside the rows ends below 2^31."""
    need = ctypes.c_int64(-1)
    a = adapters(tokens=tokens, rows=1, n=8, rank=8, ld_x=8, ld_y=1, ld_out=1, type=L.BQ_BF16)
    assert bq.lib.bq_adapters_work_bytes(ctypes.byref(a), ctypes.byref(need)) == code
    if code == bq.BQ_OK:
        assert need.value >= tokens * 8 * 4
    else:
        assert "tokens" in bq.bq_last_error()
        assert rc_of("bq_adapters_add", a) == bq.BQ_EARG and "tokens" in bq.bq_last_error()
