"""bq_matmul's activations relative to their values, far below zero too, where
1 + exp(-z) passes what f32's reciprocal gives and the results are still normal
numbers."""
import math

import numpy as np
import pytest

import synth
from gpu_util import bqmod, torch
from layer_util import DT, half_step, within
from model_util import ACTS, EPS

pytestmark = pytest.mark.gpu


def reference(x, act, dt):
    """(act(x), bound).  The bound, in half steps of f32 of the value: exp 2, its argument z (gelu: five roundings and
    the two constants, 7 at most) |z| times as many, x exp(z), sum, reciprocal and product 5; a subnormal exp is off by
    half of 2^-149, its product with x by |x| times that, and a subnormal result by as much again."""
    v = x.astype(np.float64)
    z = v if act == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)
    with np.errstate(over="ignore"):
        want = v / (1.0 + np.exp(-z))
    steps = 7 + (7 * np.abs(z) if act == "gelu" else 0)
    bound = np.where(want == 0, 0.0, steps * EPS * np.abs(want)) + 2.0 ** -149 * (1 + np.minimum(np.abs(v), 200))
    return want, bound + half_step(DT[dt]) * (np.abs(want) + bound) + (2.0 ** -134 if dt == "bf16" else 0.0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [3, 600])
def test_tails(dt, act, T):
    """No weights, the bias alone: y = act(bias)."""
    t, bq = torch(), bqmod()
    rows = 2600  # 600 tokens: a tile kernel
    low = -110.0 if act == "silu" else -11.5
    x = np.linspace(low, 12.0, rows).astype(np.float32)
    x[:5] = [0.0, -0.0, -1e4, -3e38, 3e37]
    canon = synth.q1_0_blocks(rows, 128, 1)
    canon[:, :, :2] = 0
    q, d = t.ones(T, 128, dtype=t.int8, device="cuda"), t.ones(T, 1, device="cuda")
    y = t.empty(T, rows, dtype=DT[dt], device="cuda")
    bq.bq_matmul(bq.Weights.upload(1, canon, rows, 128), bq.Act(q, d, 128, 128, T), y, bias=t.from_numpy(x).cuda(), act=ACTS[act])
    want, bound = reference(x, act, dt)
    assert (np.abs(want[x < -1]) > 1e-37).any()
    for row in y[[0, T - 1]].cpu():
        within(row, t.from_numpy(want), t.from_numpy(bound), (dt, act))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [40, 700])
def test_tails_beside_ordinary_values(dt, act, T):
    """Every third token far below zero: weights of 1, one quant of 1 or -1 a token, so that its row is its scale."""
    t, bq = torch(), bqmod()
    rows = 1600
    x = np.linspace(-6.0, 6.0, T).astype(np.float32)
    x[::3] = np.linspace(-100.0 if act == "silu" else -11.0, -80.0 if act == "silu" else -9.0, len(x[::3]))
    canon = synth.q1_0_blocks(rows, 128, 1)
    canon[:, :, :2], canon[:, :, 2:] = (0, 0x3C), 0xFF
    q = t.zeros(T, 128, dtype=t.int8)
    q[:, 5] = t.from_numpy(np.where(x < 0, -1, 1).astype(np.int8))
    d = t.from_numpy(np.abs(x)).view(T, 1).cuda()
    y = t.empty(T, rows, dtype=DT[dt], device="cuda")
    bq.bq_matmul(bq.Weights.upload(1, canon, rows, 128), bq.Act(q.cuda(), d, 128, 128, T), y, act=ACTS[act])
    want, bound = reference(x, act, dt)
    for column in y[:, [0, rows - 1]].t().cpu():
        within(column, t.from_numpy(want), t.from_numpy(bound), (dt, act))
