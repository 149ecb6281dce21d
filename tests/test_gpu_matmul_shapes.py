"""bq_matmul at the ends of its range of shapes: a head of many rows for a handful
of tokens, a projection to few rows of many tokens."""
import numpy as np
import pytest

import synth
from gpu_util import bqmod, torch
from layer_util import within
from model_util import matmul_ref
from test_gpu_matmul import acts, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,qa,cols", [(1, 128, 256), (1, 32, 128), (2, 64, 320), (2, 128, 128)])
@pytest.mark.parametrize("T", [17, 32, 33])
def test_many_rows_few_tokens(fmt, qa, cols, T):
    bq, rows = bqmod(), 66001
    canon = synth.blocks(fmt, rows, cols, 3, T)
    q, d = acts(T, cols, qa, T)
    y = run(bq.Weights.upload(fmt, canon, rows, cols), q, d, qa, torch().float32)
    within(y, *matmul_ref(fmt, canon, q, d, qa, torch().float32), (fmt, qa, T))


@pytest.mark.parametrize("fmt,qa,cols", [(1, 128, 256), (1, 32, 128), (2, 64, 320), (2, 128, 128)])
@pytest.mark.parametrize("rows", [1, 40, 64, 65])
def test_few_rows_many_tokens(fmt, qa, cols, rows):
    bq, T = bqmod(), 20001
    canon = synth.blocks(fmt, rows, cols, 3, rows)
    q, d = acts(T, cols, qa, rows)
    y = run(bq.Weights.upload(fmt, canon, rows, cols), q, d, qa, torch().float32)
    within(y, *matmul_ref(fmt, canon, q, d, qa, torch().float32), (fmt, qa, rows))


def test_head_of_a_batch():
    """24 tokens through 151936 rows, as a step's logits: a token's row does not hang on which others are beside it."""
    t, bq = torch(), bqmod()
    rows, cols, T = 151936, 512, 24
    canon = synth.q1_0_blocks(rows, cols, 1)
    w = bq.Weights.upload(1, canon, rows, cols)
    q, d = acts(T, cols, 128, 1)
    y = run(w, q, d, 128, t.float32)
    turned = run(w, np.roll(q, 5, axis=0), np.roll(d, 5, axis=0), 128, t.float32)
    assert t.equal(turned, t.roll(y, 5, 0))
    at = slice(rows - 300, rows)
    within(y[:, at], *matmul_ref(1, canon[at], q, d, 128, t.float32), "last rows")
