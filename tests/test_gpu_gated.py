"""bq_gated_q8 against its definition step by step: scales, quants and kept
values bit for bit, but where 64-bit arithmetic itself cannot tell on which side
of a border a value lies."""
import numpy as np
import pytest

from gpu_util import bqmod, torch
from layer_util import DT, gen, half_step, normal
from model_util import ACTS, gated_ref, quants_ref

pytestmark = pytest.mark.gpu


def run(gate, up, act, qa, f16_scale=False, keep=True, pad=0, **k):
    t, bq = torch(), bqmod()
    T, n = gate.shape
    q = t.full((T, n + 16 * (pad > 0)), 99, dtype=t.int8, device="cuda")
    d = t.full((T, n // qa + pad), 7.0, device="cuda")
    y = t.full((T, n + 8 * pad), 7.0, dtype=gate.dtype, device="cuda") if keep else None
    bq.bq_gated_q8(gate, up, ACTS[act], qa, q[:, :n], d[:, :n // qa], y=None if y is None else y[:, :n], f16_scale=f16_scale, **k)
    t.cuda.synchronize()
    assert (q[:, n:] == 99).all() and (d[:, n // qa:] == 7.0).all()
    return q[:, :n].cpu().numpy(), d[:, :n // qa].cpu().numpy(), None if y is None else y[:, :n].cpu()


def check(gate, up, act, qa, f16_scale, q, d, y, what):
    """y in f32 tells which of the two neighbours a value is; the quants follow from them."""
    t = torch()
    v, other, want_q, want_d = gated_ref(gate.cpu(), up.cpu(), act, qa, f16_scale)
    if y is not None and y.dtype == t.float32:
        got = y.numpy()
        off = got.view(np.uint32) != v.view(np.uint32)
        assert (got[off] == other[off]).all() and off.mean() < 1e-5, (what, int(off.sum()))
        want_q, want_d = quants_ref(got, qa, f16_scale)
    elif y is not None:
        # a value rounded twice: half a step of the type, and at most one of f32 before it
        tol = half_step(y.dtype) * 1.001 * np.abs(v) + (2.0 ** -25 if y.dtype == t.float16 else 2.0 ** -133)
        assert (np.abs(y.double().numpy() - v) <= tol).all(), what
    same = d.view(np.uint32) == want_d.view(np.uint32)
    assert same.mean() > 0.999 and (np.abs(d - want_d) <= 2.0 ** -10 * want_d).all(), what
    if y is not None and y.dtype == t.float32:
        assert same.all() and (q == want_q).all(), what
    else:
        assert (q != want_q).mean() < 1e-5 and (np.abs(q.astype(int) - want_q) <= 1).all(), what


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu2"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,n,qa,f16_scale", [(1, 32, 32, False), (3, 384, 128, True), (7, 4096, 64, False), (300, 1056, 32, True)])
def test_rows(act, dt, T, n, qa, f16_scale):
    g = gen(T * n)
    gate, up = normal(g, T, n, scale=3.0, dtype=DT[dt]).cuda(), normal(g, T, n, dtype=DT[dt]).cuda()
    check(gate, up, act, qa, f16_scale, *run(gate, up, act, qa, f16_scale, pad=1), (act, dt))
    q, d, _ = run(gate, up, act, qa, f16_scale, keep=False)
    assert np.array_equal(q, run(gate, up, act, qa, f16_scale)[0]) and np.array_equal(d, run(gate, up, act, qa, f16_scale)[1])


@pytest.mark.parametrize("act", ["silu", "gelu", "relu2"])
def test_wide_range(act):
    """Values from subnormal to large, both signs, zeros; whole blocks of zeros."""
    t = torch()
    g = gen(5)
    e = t.randint(-140, 30, (64, 256), generator=g).double()
    gate = (t.randn(64, 256, generator=g).double() * 2.0 ** e).float()
    gate[0, :128] = 0.0
    gate[1] = t.linspace(-120, 120, 256)
    gate[2] = t.linspace(-1e4, 1e4, 256)
    gate[3, 128:] = -0.0
    up = normal(g, 64, 256)
    up[4, :128] = 0.0
    check(gate.cuda(), up.cuda(), act, 128, False, *run(gate.cuda(), up.cuda(), act, 128), act)


def test_halves_of_one_tensor_in_place():
    """Gate and up side by side in one tensor, the values written over the gate."""
    t, bq = torch(), bqmod()
    both = normal(gen(1), 33, 2 * 640).cuda()
    gate, up = both[:, :640], both[:, 640:]
    want = run(gate, up, "silu", 64)
    keep = up.clone()
    q, d = t.empty(33, 640, dtype=t.int8, device="cuda"), t.empty(33, 10, device="cuda")
    bq.bq_gated_q8(gate, up, bq.BQ_SILU, 64, q, d, y=gate)
    assert np.array_equal(q.cpu().numpy(), want[0]) and np.array_equal(d.cpu().numpy(), want[1])
    assert t.equal(gate.cpu(), want[2]) and t.equal(up, keep)


def test_quants_feed_a_product():
    """One token without its first dimension, then the product that reads it."""
    t, bq = torch(), bqmod()
    import synth
    canon = synth.q1_0_blocks(64, 256, 1)
    w = bq.Weights.upload(1, canon, 64, 256)
    gate, up = normal(gen(2), 256).cuda(), normal(gen(3), 256).cuda()
    q, d, y = t.empty(256, dtype=t.int8, device="cuda"), t.empty(2, device="cuda"), t.empty(64, device="cuda")
    bq.bq_gated_q8(gate, up, bq.BQ_GELU, 128, q, d)
    bq.bq_q1_0_matvec(w, bq.Act(q, d, 256, 128), y)
    import oracle
    ref = oracle.matvec(1, canon, 64, 256, q.cpu().numpy(), d.cpu().numpy(), 128)
    assert np.array_equal(y.cpu().numpy().view(np.uint32), np.asarray(ref).reshape(-1).view(np.uint32))


def test_refusals():
    t, bq = torch(), bqmod()
    x, q, d = t.zeros(4, 128, device="cuda"), t.zeros(4, 128, dtype=t.int8, device="cuda"), t.zeros(4, 1, device="cuda")
    for args in ((x, x.half(), 1, 128, q, d), (x, x[:2], 1, 128, q, d), (x, x, 1, 128, q.short(), d), (x, x, 1, 128, q[:, :64], d),
                 (x, x, 1, 128, q, d.half()), (x, x, 9, 128, q, d), (x, x, 1, 100, q, d), (x.double(), x, 1, 128, q, d),
                 (x, x.cpu(), 1, 128, q, d), (x, x.t(), 1, 128, q, d)):
        with pytest.raises(bq.BQError):
            bq.bq_gated_q8(*args)
