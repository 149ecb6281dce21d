"""How near to a border of f32 a value of bq_gated_q8 has to lie to be rounded the
other way: what include/bq.h states, against 64 bits of mantissa."""
import numpy as np
import pytest

from gpu_util import bqmod, torch
from layer_util import gen, normal
from model_util import ACTS

pytestmark = pytest.mark.gpu

LD = np.longdouble
# gates and ups whose product lies 1.3 to 16 times 2^-50 of itself from a border, on the side that binary64 leaves
# (found by trying pairs)
NEAR = [("-0x1.1a5a18p+3", "0x1.a4336cp+0"),
         ("-0x1.3cd080p+3", "0x1.6b0598p+0"),
         ("-0x1.366bfap+3", "0x1.ee4be4p+0"),
         ("-0x1.277c52p+3", "0x1.e4a4d0p+0"),
         ("-0x1.37e518p+3", "0x1.07d2aep+0"),
         ("-0x1.210578p+3", "0x1.3261b8p+0"),
         ("-0x1.11f572p+3", "0x1.fc6858p+0"),
         ("-0x1.2d7716p+3", "0x1.519804p+0"),
         ("-0x1.39ac0ap+3", "0x1.033326p+0"),
         ("-0x1.1e2e5ap+3", "0x1.b24066p+0"),
         ("-0x1.23c41ap+3", "0x1.3c3762p+0"),
         ("-0x1.2f004cp+3", "0x1.b4a4fep+0"),
         ("-0x1.3a79c2p+3", "0x1.342404p+0"),
         ("-0x1.2000bep+3", "0x1.4a6f22p+0"),
         ("-0x1.23f9e2p+3", "0x1.a4c1a0p+0"),
         ("-0x1.f88564p+2", "0x1.3264d0p+0"),
         ("-0x1.2db2fcp+3", "0x1.b4b6f0p+0"),
         ("-0x1.117298p+3", "0x1.01bf8ap+0"),
         ("-0x1.03b788p+3", "0x1.ea6a32p+0"),
         ("-0x1.1e96b2p+3", "0x1.2ba014p+0"),
         ("-0x1.0ec6bap+3", "0x1.670a10p+0"),
         ("-0x1.01505ap+3", "0x1.fba04cp+0"),
         ("-0x1.0c87e8p+3", "0x1.547308p+0"),
         ("-0x1.05dde4p+3", "0x1.f87bb6p+0")]


def exact(gate, up, act):
    """(v, the bound relative to it): 2^-50, with GELU (1 + 2 |z|) 2^-50."""
    x = gate.astype(LD)
    if act == "relu2":
        return np.maximum(x, 0) ** 2 * up.astype(LD), LD(2.0 ** -50)
    z = x / 2
    if act == "gelu":
        z = np.sqrt(LD(2) / (4 * np.arctan(LD(1)))) * (x + LD("0.044715") * x ** 3)
    v = x / (1 + np.exp(-2 * z)) * up.astype(LD)
    return v, LD(2.0 ** -50) * (1 + (2 * np.abs(z) if act == "gelu" else 0))


def check(gate, up, act):
    t, bq = torch(), bqmod()
    T, n = gate.shape
    q, d, y = t.empty(T, n, dtype=t.int8, device="cuda"), t.empty(T, n // 32, device="cuda"), t.empty(T, n, device="cuda")
    bq.bq_gated_q8(t.from_numpy(gate).cuda(), t.from_numpy(up).cuda(), ACTS[act], 32, q, d, y=y)
    y = y.cpu().numpy()
    v, rel = exact(gate, up, act)
    rel = rel * LD(1 + 2.0 ** -10)  # the reference's own roundings, seven and, of the argument, 7 * 2 |z|, of 2^-64
    lo, hi = (v - np.abs(v) * rel).astype(np.float32), (v + np.abs(v) * rel).astype(np.float32)
    assert ((y == lo) | (y == hi)).all(), np.argwhere((y != lo) & (y != hi))[:4]
    return int((y != v.astype(np.float32)).sum())


def test_pairs_next_to_a_border():
    assert np.finfo(LD).eps < 2.0 ** -62
    gate, up = (np.array([float.fromhex(p[i]) for p in NEAR], np.float32) for i in (0, 1))
    both = [np.tile(a, -(-1024 // len(a)))[:1024].reshape(4, 256) for a in (gate, up)]
    check(*both, "gelu")


@pytest.mark.parametrize("act", ["silu", "gelu", "relu2"])
@pytest.mark.parametrize("scale", [1.0, 4.0, 30.0])
def test_many_values(act, scale):
    g = gen(int(scale))
    gate, up = normal(g, 1000, 1024, scale=scale).numpy(), normal(g, 1000, 1024).numpy()
    if act == "gelu":
        gate = np.clip(gate, -13, None)  # 2 |z| < 200: results down to 1e-85 are 0 on both sides
    check(gate, up, act)
