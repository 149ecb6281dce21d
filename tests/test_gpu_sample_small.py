"""bq_sample where temperature and differences of the logits are near the
smallest numbers of f32."""
import numpy as np
import pytest

from gpu_util import torch
from model_util import Ranked
from test_gpu_sample import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [7, 3001, 40000])
@pytest.mark.parametrize("temp", [2.0 ** -90, 2.0 ** -101, 2.0 ** -122, 1e-38, 2.0 ** -140])
@pytest.mark.parametrize("shift", [0, 40])
def test_tiny_temperatures(vocab, temp, shift):
    """Logits a few temperatures apart (all numbers of f32), the largest at shift temperatures: each in turn is drawn
    with u in the middle of its share, and the others are too far down."""
    t = torch()
    g = np.random.default_rng(vocab)
    temp = np.float32(temp)
    x = np.full(vocab, -3e38, np.float32)
    near = g.permutation(vocab)[:6]
    x[near] = (np.float64(temp) * (shift - np.arange(6) * 0.75)).astype(np.float32)
    x[g.permutation(np.setdiff1d(np.arange(vocab), near))[:1]] = np.float32(temp * np.float32(shift - 200.0))
    r = Ranked(x, float(temp))
    assert r.w[5] > 0.02 and r.w[6] < 1e-80
    token, logprob = run(t.from_numpy(np.tile(x, (6, 1))).cuda(), [r.inside(i, vocab) for i in range(6)], [temp] * 6)
    assert token.tolist() == r.order[:6].tolist()
    # the two smallest temperatures are subnormal: as given to the kernel and to the reference alike
    assert np.allclose(logprob, [r.logprob(i) for i in range(6)], rtol=1e-6, atol=1e-6)
    # top_k and top_p end between two of them
    top = float(np.float32(1 - 2.0 ** -24))
    share = (r.sums[3] - 0.5 * r.w[3]) / r.sums[-1]
    token, _ = run(t.from_numpy(np.tile(x, (2, 1))).cuda(), [top] * 2, [temp] * 2, top_k=[3, 0], top_p=[1.0, share])
    assert token.tolist() == [r.order[2], r.order[3]]


@pytest.mark.parametrize("vocab", [9, 5000, 40000])
@pytest.mark.parametrize("temp", [2.0 ** -99, 2.0 ** -101, 1e-38, 2.0 ** -149])
def test_tiny_temperatures_and_large_logits(vocab, temp):
    """The largest logit far from zero on either side: nothing but its equals weighs anything."""
    t = torch()
    g = np.random.default_rng(vocab)
    tops = [-3.4e38, -1e30, -2.0 ** 28, -2.0 ** 27, -1.0, 1.0, 2.0 ** 27, 2.0 ** 28, 1e30, 3.4e38]
    x = np.empty((len(tops), vocab), np.float32)
    for b, top in enumerate(tops):
        top = np.float32(top)
        x[b] = np.nextafter(top, np.float32(-np.inf))
        x[b, g.permutation(vocab)[:vocab // 3]] = -np.inf
        x[b, g.permutation(vocab)[:2]] = top
    equal = [np.flatnonzero(row == np.float32(top)) for row, top in zip(x, tops)]
    rows = t.from_numpy(x).cuda()
    for u, which in ((0.25, 0), (0.75, 1)):
        token, logprob = run(rows, [u] * len(tops), [temp] * len(tops))
        assert token.tolist() == [int(e[which]) for e in equal]
        assert np.allclose(logprob, -np.log(2.0), rtol=1e-6)
