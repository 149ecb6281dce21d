"""bq_adapters_add at the longest rows of x that it takes."""
import pytest

from gpu_util import bqmod, torch

pytestmark = pytest.mark.gpu


def test_adapters_of_the_longest_rows():
    """n of 2^31 - 8 in one piece (many requests, all but one empty): the piece's
    length passes 31 bits.  A few values at both ends and in between are not 0,
    so that the sums are small whole numbers."""
    t, bq = torch(), bqmod()
    n, rank, rows, requests = (1 << 31) - 8, 8, 5, 200
    at = t.tensor([0, 1, 127, 128, 1 << 20, (1 << 30) + 77, (1 << 31) - 129, (1 << 31) - 128, n - 8, n - 1])
    xs = t.arange(1, len(at) + 1).float()
    a_s = (t.arange(rank)[:, None] + t.arange(len(at))[None, :]) % 5 - 2.0
    b = (t.arange(rows)[:, None] * 3 + t.arange(rank)[None, :]) % 7 - 3.0
    x = t.zeros(1, n, dtype=t.bfloat16, device="cuda")
    a = t.zeros(1, rank, n, dtype=t.bfloat16, device="cuda")
    for j, i in enumerate(at.tolist()):
        x[0, i] = xs[j].item()
        for r in range(rank):
            a[0, r, i] = a_s[r, j].item()
    y = t.arange(rows).float()[None] * 0.5
    cu = t.ones(requests + 1, dtype=t.int32)
    cu[0] = 0
    out = t.full((1, rows), 9.0, device="cuda")
    bq.bq_adapters_add(bq.Adapters(a, b[None].bfloat16().cuda(), t.tensor([2.0]).cuda()), x, cu.cuda(),
                       t.zeros(requests, dtype=t.int32).cuda(), 1, y.cuda(), out=out)
    t.cuda.synchronize()
    del x, a
    t.cuda.empty_cache()
    assert t.equal(out.cpu(), y + 2 * (a_s @ xs) @ b.t())
