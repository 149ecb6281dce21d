"""The f16-valued scales of bq_rmsnorm_q8 are rounded twice, as include/bq.h
has it: max|v| * fl(1/127) to binary32, that to f16.  One rounding of the exact
product differs where the binary32 value falls onto a tie of f16, one block in
about 2^14: maxima picked so that it does in every block, and a million blocks."""
import numpy as np
import pytest

from gpu_util import bqmod, torch
from layer_util import DT, gen, norm_ref, normal

pytestmark = pytest.mark.gpu

INV = np.float32(1) / np.float32(127)


def once_and_twice(m):
    """The scale of maxima m (f32): the exact product rounded to f16 once (48
    bits are exact in 64), and by way of binary32."""
    return (m.astype(np.float64) * np.float64(INV)).astype(np.float16), (m * INV).astype(np.float16)


def run(x, w, qa):
    t, bq = torch(), bqmod()
    q = t.empty(*x.shape, dtype=t.int8, device="cuda")
    d = t.empty(x.shape[0], x.shape[1] // qa, device="cuda")
    bq.bq_rmsnorm_q8(x.cuda(), w.cuda(), 1e-6, qa, q, d, f16_scale=True)
    return q.cpu(), d.cpu()


@pytest.mark.parametrize("qa", [32, 64, 128])
def test_f16_scale_on_ties(qa):
    """Every block's maximum is picked, by its weight, where the two differ."""
    t = torch()
    n, blocks = 32 * qa, 32
    x = normal(gen(qa), 1, n).clamp_(-2, 2)
    at = t.arange(blocks) * qa + 5
    x[0, at] = 3.0 + t.rand(blocks, generator=gen(qa + 1))
    w = t.full((n,), 0.5)
    r = (1.0 / (x.double().square().sum(1) / n + 1e-6).sqrt()).float()
    a = (x[0, at] * r).numpy()
    tries = (np.float32(1) + np.arange(1 << 19, dtype=np.float32) * np.float32(2.0 ** -23)).astype(np.float32)
    once, twice = once_and_twice(a[:, None] * tries[None, :])
    assert (once != twice).any(1).all()
    w[at] = t.from_numpy(tries[(once != twice).argmax(1)])
    _, v, rq, rd = norm_ref(x, None, w, 1e-6, qa, True)
    once, twice = once_and_twice(v.abs().view(blocks, qa).amax(1).numpy())
    assert (once != twice).all() and (twice.astype(np.float32) == rd.numpy()[0]).all()
    q, d = run(x, w, qa)
    assert t.equal(d, rd) and t.equal(q, rq)


@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
def test_f16_scale_of_a_million_blocks(type):
    t = torch()
    x, w = normal(gen(1), 2048, 16384, dtype=DT[type]), normal(gen(2), 16384, dtype=DT[type], scale=0.1, shift=1.0)
    _, v, rq, rd = norm_ref(x, None, w, 1e-6, 32, True)
    once, twice = once_and_twice(v.abs().view(2048, 512, 32).amax(2).numpy())
    assert (once != twice).sum() >= 10
    q, d = run(x, w, 32)
    assert t.equal(d, rd) and t.equal(q, rq)


@pytest.mark.parametrize("f16_scale", [False, True])
@pytest.mark.parametrize("qa", [32, 128])
def test_beside_the_oracles_quantizer(qa, f16_scale):
    """The norm's scale is max * fl(1/127), the quantizer's amax / 127 (the
    oracle's, bq_quantize_act_q8's).  fl(1/127) is within 2^-28 of 1/127, so the
    two f32 scales are at most one unit in the last place apart, and v / d moves
    by at most 127 (2^-23 + 2 * 2^-24) < 2^-15: the quants are the same but next
    to half-integers.  Scales as f16 are the same or neighbours."""
    import oracle
    t, bq = torch(), bqmod()
    x, w = normal(gen(3), 300, 4096), normal(gen(4), 4096, scale=0.1, shift=1.0)
    q, y = t.empty(300, 4096, dtype=t.int8, device="cuda"), t.empty(300, 4096, device="cuda")
    d = t.empty(300, 4096 // qa, device="cuda")
    bq.bq_rmsnorm_q8(x.cuda(), w.cuda(), 1e-6, qa, q, d, y=y, f16_scale=f16_scale)
    v = y.cpu().numpy().reshape(-1, qa)
    oq, od, _ = oracle.quantize_q8(v.ravel(), qa, f16_scale)
    got, oq, d = q.cpu().numpy().reshape(-1, qa).astype(int), oq.reshape(-1, qa).astype(int), d.cpu().numpy().ravel()
    if f16_scale:
        steps = np.abs(d.astype(np.float16).view(np.int16).astype(int) - od.astype(np.float16).view(np.int16))
        assert (d == d.astype(np.float16)).all()
    else:
        steps = np.abs(d.view(np.int32).astype(np.int64) - od.view(np.int32))
    assert steps.max() <= 1
    same = steps == 0
    assert (got[same] == oq[same]).all()
    if f16_scale:
        assert same.mean() > 0.99
    else:
        ratio = np.abs(v.astype(np.float64) / od[:, None])
        border = np.abs(ratio - np.floor(ratio) - 0.5) <= 2.0 ** -15
        assert (np.abs(got - oq) <= border).all()
