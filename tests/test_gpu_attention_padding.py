"""staging.StagedAttention on a padded batch: rows behind the last request."""
import pytest

from gpu_util import torch
from test_gpu_attention_block import Model

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [1, 2])
def test_padded_rows_stay_finite(fmt, monkeypatch):
    """The attention leaves the rows of its output behind the last request as
    they were, and the quantizer reads all rows and takes finite values only:
    what the buffers' memory held before must not get there.  The requests'
    rows have the bits of the batch without padding."""
    t = torch()
    lens, new, rows = [37, 5, 20], [37, 5, 20], 62 + 5
    want = Model(fmt, 80)
    s = want.step(lens, new, 1)
    out, h = want.run(s, 37, 37)
    out, h = out.clone(), h.clone()
    real = t.empty

    def dirty(*a, **k):
        v = real(*a, **k)
        return v.fill_(float("nan")) if v.is_floating_point() else v.fill_(-1)

    with monkeypatch.context() as m:
        m.setattr(t, "empty", dirty)
        padded = Model(fmt, 80)
    s = {n: v.clone() for n, v in s.items()}
    s["x"] = t.cat([s["x"], t.ones(5, s["x"].shape[1], device="cuda")])
    s["pos"] = t.cat([s["pos"], s["pos"][:5]])
    s["slot"] = t.cat([s["slot"], t.full_like(s["slot"][:5], -1)])
    got, got_h = padded.run(s, 37, 37)
    assert got.shape[0] == rows and t.equal(got[:62], out) and t.equal(got_h[:62], h)
    for b in padded.blocks:
        for name in ("o", "o_d", "out", "h"):
            assert t.isfinite(getattr(b, name)[:rows]).all(), name
