"""Infinities and NaN in one row of an operator between the products stay in
that row: the header gives no value for it, and its own for all others."""
import pytest

from gpu_util import bqmod, torch
from layer_util import DT, Paged, adapters_ref, attn_ref, gen, norm_ref, normal, within

pytestmark = pytest.mark.gpu

BAD = [float("inf"), -float("inf"), float("nan")]


@pytest.mark.parametrize("type,cache", [("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("new,keys", [(1, 200), (9, 3000), (100, 300)])
def test_attention_keeps_them_in_their_row(type, cache, new, keys):
    t, bq = torch(), bqmod()
    D, H, Hq, requests = 64, 2, 4, 3
    p = Paged([keys] * requests, H, D, 16, DT[cache], 3)
    q = normal(gen(4), requests * new, Hq, D, dtype=DT[type])
    clean = q.clone()
    bad = [(0, 1), (requests * new - 1, 0), (requests * new // 2, 3)]
    for (row, head), v in zip(bad, BAD):
        q[row, head, 7] = v
    cu = t.arange(requests + 1, dtype=t.int32) * new
    out = t.empty(q.shape, dtype=q.dtype, device="cuda")
    bq.bq_paged_attn(bq.KVCache(p.k.cuda(), p.v.cuda()), q.cuda(), cu.cuda(),
                     t.full((requests,), keys, dtype=t.int32, device="cuda"), p.table.cuda(), 0.125, new, keys, out)
    out = out.cpu()
    for b in range(requests):
        rows = slice(b * new, (b + 1) * new)
        want, bound = attn_ref(clean[rows], p.k_of[b], p.v_of[b], keys, 0.125, DT[type])
        got = out[rows].clone()
        for row, head in bad:
            if row // new == b:
                got[row - b * new, head] = want[row - b * new, head].to(got.dtype)
        within(got, want, bound, b)


@pytest.mark.parametrize("x_type,type", [("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("new", [[1, 1, 1], [40, 3, 20]])
def test_adapters_keep_them_in_their_row(x_type, type, new):
    t, bq = torch(), bqmod()
    n, rows, rank, T = 264, 100, 24, sum(new)
    g = gen(T)
    x, y = normal(g, T, n, dtype=DT[x_type]), normal(g, T, rows)
    a, b = normal(g, 2, rank, n, dtype=DT[type], scale=n ** -0.5), normal(g, 2, rows, rank, dtype=DT[type])
    gain, ids = t.tensor([0.5, 2.0]), [1, 0, 1]
    clean, bad = x.clone(), (0, T - 1, new[0])
    for row, v in zip(bad, BAD):
        x[row, 11] = v
    cu = t.tensor([0] + new).cumsum(0).to(t.int32)
    out = t.empty(T, rows, device="cuda")
    bq.bq_adapters_add(bq.Adapters(a.cuda(), b.cuda(), gain.cuda()), x.cuda(), cu.cuda(),
                       t.tensor(ids, dtype=t.int32).cuda(), max(new), y.cuda(), out=out)
    out = out.cpu()
    for row in bad:
        assert not t.isfinite(out[row]).any(), row
    keep = t.tensor([r not in bad for r in range(T)])
    for r, i in enumerate(ids):
        rows_ = slice(int(cu[r]), int(cu[r + 1]))
        want, bound = adapters_ref(clean[rows_], a[i], b[i], gain[i], y[rows_])
        k = keep[rows_]
        within(out[rows_][k], want[k], bound[k], r)


@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
def test_norm_keeps_them_in_their_row(type):
    t, bq = torch(), bqmod()
    x, w = normal(gen(1), 5, 512, dtype=DT[type]), normal(gen(2), 512, dtype=DT[type], scale=0.1, shift=1.0)
    _, _, rq, rd = norm_ref(x, None, w, 1e-6, 64, False)
    for row, v in zip((0, 2, 4), BAD):
        x[row, 100] = v
    q, d = t.empty(5, 512, dtype=t.int8, device="cuda"), t.empty(5, 8, device="cuda")
    bq.bq_rmsnorm_q8(x.cuda(), w.cuda(), 1e-6, 64, q, d)
    for row in (1, 3):
        assert t.equal(q[row].cpu(), rq[row]) and t.equal(d[row].cpu(), rd[row])
