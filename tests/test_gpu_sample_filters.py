"""bq_sample: filters that are not numbers filter nothing."""
import numpy as np
import pytest

from gpu_util import torch
from model_util import Ranked
from test_gpu_sample import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["min_p", "top_p"])
@pytest.mark.parametrize("vocab", [5, 2000, 151936])
def test_nan_filters(name, vocab):
    """Each of several places of the order by a u in the middle of its share, as without the filter."""
    x = np.random.default_rng(vocab).standard_normal(vocab).astype(np.float32)
    r = Ranked(x)
    able = np.flatnonzero(r.w / r.sums[-1] > 2.0 ** -21)  # wider than the steps of u
    ranks = [int(able[len(able) * i // 8]) for i in range(8)] + [int(able[-1])]
    u = [r.inside(i, vocab) for i in ranks]
    rows = torch().from_numpy(np.tile(x, (len(u), 1))).cuda()
    nan = [float("nan")] * len(u)
    want = [int(r.order[i]) for i in ranks]
    assert run(rows, u)[0].tolist() == want
    assert run(rows, u, **{name: nan})[0].tolist() == want
    # beside another filter, which still holds
    kept = r.kept(3)
    u = [r.inside(i, kept) for i in range(3)]
    assert run(rows[:3], u, top_k=[3] * 3, **{name: nan[:3]})[0].tolist() == r.order[:3].tolist()
