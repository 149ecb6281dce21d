"""The operators between the products where one launch's grid is not enough, or
its first dimension is full: results of the last rows, as those of small calls."""
import pytest

from gpu_util import bqmod, torch
from layer_util import Paged, adapters_ref, attn_ref, gen, normal, within

pytestmark = pytest.mark.gpu


def test_norm_of_more_rows_than_a_launch():
    t, bq = torch(), bqmod()
    T, n, part = (1 << 21) + 700, 64, (1 << 20) + 64
    base = normal(gen(1), 4099, n, dtype=t.bfloat16).cuda()
    x = base[t.arange(T, device="cuda") % 4099]
    w = normal(gen(2), n, dtype=t.bfloat16, scale=0.2, shift=1.0).cuda()

    def run(*cuts):
        q = t.empty(T, n, dtype=t.int8, device="cuda")
        d, y = t.empty(T, n // 32, device="cuda"), t.empty_like(x)
        for a, b in zip((0,) + cuts, cuts + (T,)):
            bq.bq_rmsnorm_q8(x[a:b], w, 1e-6, 32, q[a:b], d[a:b], y=y[a:b])
        return q, d, y

    for whole, parts in zip(run(), run(part, 2 * part - 100)):
        assert t.equal(whole, parts)


def test_append_of_more_tokens_than_a_launch():
    t, bq = torch(), bqmod()
    T, D, page = (1 << 17) + 77, 64, 16
    g = gen(3)
    rows = normal(g, T, 3 * D).cuda()
    q, k, v = (r.unflatten(1, (1, D)) for r in rows.split(D, 1))
    pages = -(-T // page) + 1
    slot = t.randperm(pages * page, generator=g)[:T].cuda()
    pos = t.arange(T, dtype=t.int32).cuda()
    freq = (1e4 ** (-t.arange(0, D, 2).double() / D)).float().cuda()

    def run(*cuts):
        kv = bq.KVCache(t.zeros(pages, 1, page, D, dtype=t.bfloat16, device="cuda"),
                        t.zeros(pages, 1, D, page, dtype=t.bfloat16, device="cuda"))
        qo = t.empty(T, 1, D, dtype=t.bfloat16, device="cuda")
        for a, b in zip((0,) + cuts, cuts + (T,)):
            bq.bq_kv_append(kv, k[a:b], v[a:b], pos[a:b], slot[a:b], freq, q=q[a:b], q_out=qo[a:b])
        return kv.k, kv.v, qo

    for whole, parts in zip(run(), run(60000, 100003)):
        assert t.equal(whole, parts)


def test_attention_join_of_more_rows_than_a_grid_row():
    t, bq = torch(), bqmod()
    H, G, D, keys, last = 64, 16, 64, 1024, 100
    T = (1 << 15) + last
    p = Paged([keys], H, D, 16, t.bfloat16, 5)
    tail = normal(gen(6), last, H * G, D, dtype=t.bfloat16)
    q = t.zeros(T, H * G, D, dtype=t.bfloat16, device="cuda")
    q[-last:] = tail.cuda()
    out = t.full_like(q, 3.0)
    cu, lens = t.tensor([0, T], dtype=t.int32).cuda(), t.tensor([keys], dtype=t.int32).cuda()
    bq.bq_paged_attn(bq.KVCache(p.k.cuda(), p.v.cuda()), q, cu, lens, p.table.cuda(), D ** -0.5, 5, keys, out)
    assert not out[:T - keys].any(), "rows that see no key"
    for kh in (0, 1, H - 1):
        mine = slice(kh * G, (kh + 1) * G)
        want, bound = attn_ref(tail[:, mine], p.k_of[0][:, kh:kh + 1], p.v_of[0][:, kh:kh + 1], keys, D ** -0.5,
                               t.bfloat16)
        within(out[-last:, mine], want, bound, kh)


def test_adapters_walk_past_a_grid():
    """More items of 16 tokens than workgroups are launched."""
    t, bq = torch(), bqmod()
    T, n, rows, rank = (1 << 26) + 1000, 8, 1, 8
    g = gen(7)
    x = normal(g, 4099, n, dtype=t.bfloat16).cuda().repeat(T // 4099 + 1, 1)[:T]
    a, b = normal(g, 1, rank, n, dtype=t.bfloat16), normal(g, 1, rows, rank, dtype=t.bfloat16)
    gain, y = t.tensor([0.75]), normal(g, 4099, rows).cuda().repeat(T // 4099 + 1, 1)[:T]
    out = t.full_like(y, 9.0)
    bq.bq_adapters_add(bq.Adapters(a.cuda(), b.cuda(), gain.cuda()), x, t.tensor([0, T], dtype=t.int32).cuda(),
                       t.tensor([0], dtype=t.int32).cuda(), T, y, out=out)
    for s in (slice(0, 4099), slice(1 << 26, T), slice((1 << 26) - 50, (1 << 26) + 50), slice(T // 2, T // 2 + 4099)):
        within(out[s], *adapters_ref(x[s].cpu(), a[0], b[0], gain[0], y[s].cpu()), s)
    repeats = T // 4099 * 4099
    assert t.equal(x[:repeats].view(-1, 4099, n), x[:4099].view(1, 4099, n).expand(repeats // 4099, 4099, n))
    assert t.equal(out[:repeats].view(-1, 4099), out[:4099].view(1, 4099).expand(repeats // 4099, 4099))
