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


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [3, 600])
def test_tails(dt, act, T):
    """No weights, the bias alone: y = act(bias).

    The bound, in half steps of f32 of the value: exp 2, its argument z (gelu: five roundings and the two constants,
    7 at most) |z| times as many, x exp(z), sum, reciprocal and product 5; a subnormal exp is off by half of 2^-149,
    its product with x by |x| times that, and a subnormal result by as much again."""
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
    v = x.astype(np.float64)
    z = v if act == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)
    with np.errstate(over="ignore"):
        want = v / (1.0 + np.exp(-z))
    steps = 7 + (7 * np.abs(z) if act == "gelu" else 0)
    bound = np.where(want == 0, 0.0, steps * EPS * np.abs(want)) + 2.0 ** -149 * (1 + np.minimum(np.abs(v), 200))
    bound = bound + half_step(DT[dt]) * (np.abs(want) + bound) + (2.0 ** -134 if dt == "bf16" else 0.0)
    assert (np.abs(want[x < -1]) > 1e-37).any()
    for row in y[[0, T - 1]].cpu():
        within(row, t.from_numpy(want), t.from_numpy(bound), (dt, act))
