"""Requests whose offsets descend, start below 0 or past the rows have none:
their rows stay as they were, the others' come out right."""
import pytest

from gpu_util import bqmod, torch
from layer_util import Paged, adapters_ref, attn_ref, gen, normal, within

pytestmark = pytest.mark.gpu

LEAST = -(1 << 31)


@pytest.mark.parametrize("new,keys,max_keys", [(3, 40, 64), (3, 5000, 5000), (90, 200, 64)])
def test_attention_of_descending_offsets(new, keys, max_keys):
    t, bq = torch(), bqmod()
    H, Hq, D, T = 2, 4, 64, 2 * new + 9
    # rows 0 .. new and T - new .. T are requests', those in between are not
    cu = [0, new, LEAST, T - new, T, LEAST, T + 5, (1 << 31) - 1, -3]
    holds = {0: slice(0, new), 3: slice(T - new, T)}
    p = Paged([keys] * 8, H, D, 16, t.bfloat16, 7)
    q = normal(gen(8), T, Hq, D)
    out = t.full((T, Hq, D), 3.0, device="cuda")
    bq.bq_paged_attn(bq.KVCache(p.k.cuda(), p.v.cuda()), q.cuda(), t.tensor(cu, dtype=t.int64).to(t.int32).cuda(),
                     t.full((8,), keys, dtype=t.int32, device="cuda"), p.table.cuda(), 0.125, new, max_keys, out)
    t.cuda.synchronize()
    for b, rows in holds.items():
        within(out[rows], *attn_ref(q[rows], p.k_of[b], p.v_of[b], keys, 0.125, t.float32), b)
    assert (out[new:T - new] == 3.0).all()


def test_attention_of_one_descending_request():
    t, bq = torch(), bqmod()
    p = Paged([300], 2, 64, 16, t.float16, 9)
    for lo, hi in ((5, LEAST), (6, 2), (-1, 4), (9, 12), (LEAST, (1 << 31) - 1)):
        for max_new in (1, 9):
            for dt in (t.float32, t.float16):
                out = t.full((9, 16, 64), 3.0, dtype=dt, device="cuda")
                bq.bq_paged_attn(bq.KVCache(p.k.cuda(), p.v.cuda()), t.ones_like(out),
                                 t.tensor([lo, hi]).to(t.int32).cuda(), t.tensor([300], dtype=t.int32).cuda(),
                                 p.table.cuda(), 0.125, max_new, 300, out)
                t.cuda.synchronize()
                assert (out == 3.0).all(), (lo, hi, max_new)


@pytest.mark.parametrize("new", [3, 70])
def test_adapters_of_descending_offsets(new):
    t, bq = torch(), bqmod()
    n, rows, rank, T = 264, 70, 16, 2 * new + 9
    cu = [0, new, LEAST, T - new, T, LEAST, T + 5, (1 << 31) - 1, -3]
    g = gen(new)
    x, y = normal(g, T, n), normal(g, T, rows)
    a, b = normal(g, 2, rank, n, dtype=t.bfloat16), normal(g, 2, rows, rank, dtype=t.bfloat16)
    gain = normal(g, 2, scale=0.3, shift=1.0)
    ids = [0, 1, 1, 1, 0, 0, -1, 1]
    out = t.full((T, rows), 3.0, device="cuda")
    bq.bq_adapters_add(bq.Adapters(a.cuda(), b.cuda(), gain.cuda()), x.cuda(), t.tensor(cu).to(t.int32).cuda(),
                       t.tensor(ids, dtype=t.int32).cuda(), new, y.cuda(), out=out)
    t.cuda.synchronize()
    for r, s in ((0, slice(0, new)), (3, slice(T - new, T))):
        within(out[s], *adapters_ref(x[s], a[ids[r]], b[ids[r]], gain[ids[r]], y[s]), r)
    assert (out[new:T - new] == 3.0).all()
