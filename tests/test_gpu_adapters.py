"""bq_adapters_add against the formula in 64 bits: requests of one row to many,
with and without an adapter, ids out of range, in place and not, rows with
gaps, every rank from 8 to 128, all types."""
import pytest

from gpu_util import bqmod, torch
from layer_util import DT, adapters_ref, gen, normal, within

pytestmark = pytest.mark.gpu

# new, ids, n, rows, rank, count, x type, type
CASES = [
    ([1], [0], 4096, 4096, 8, 1, "f32", "bf16"),
    ([1] * 16, [0, 1, 2, 3, 1, 1, -1, 0, 3, 2, 2, 9, 0, 1, 2, 3], 4096, 1024, 16, 4, "f32", "bf16"),
    ([1] * 5, [2, 0, 1, 1, -1], 1024, 777, 24, 3, "f16", "f16"),
    ([1, 1, 1], [0, 0, 0], 128, 1, 8, 2, "f32", "f16"),
    ([7, 0, 1, 33], [1, 0, -1, 0], 640, 300, 32, 2, "bf16", "bf16"),
    ([100, 20], [1, 1], 1032, 513, 64, 2, "f32", "f16"),
    ([17, 64, 3], [0, -3, 2], 256, 4097, 128, 3, "f32", "bf16"),
    ([300], [0], 4096, 4096, 40, 1, "bf16", "bf16"),
    ([129, 2, 2, 2], [3, 1, 0, 7], 8, 8, 8, 4, "f16", "f16"),
    ([65, 31], [0, 1], 12288, 130, 104, 2, "f32", "bf16"),
    ([50], [0], 520, 64, 72, 1, "f32", "f16"),
]


def run(new, ids, n, rows, rank, count, x_type, type, pad=0, in_place=False, max_new=None, work=None, size=1.0):
    t, bq = torch(), bqmod()
    g = gen(n + rows + rank)
    T = sum(new) + 2
    x = normal(g, T, n, dtype=DT[x_type], scale=size)
    a = normal(g, count, rank, n, dtype=DT[type], scale=n ** -0.5)
    b = normal(g, count, rows, rank, dtype=DT[type], scale=rank ** -0.5)
    gain = normal(g, count, scale=0.3, shift=1.0)
    y = normal(g, T, rows, scale=size)
    cu = t.tensor([0] + new).cumsum(0).to(t.int32)
    xd = t.full((T, n + pad), 9.0, dtype=DT[x_type], device="cuda")
    xd[:, :n] = x
    yd = t.full((T, rows + pad), 9.0, device="cuda")
    yd[:, :rows] = y
    od = yd if in_place else t.full((T, rows + 2 * pad), 9.0, device="cuda")
    bq.bq_adapters_add(bq.Adapters(a.cuda(), b.cuda(), gain.cuda()), xd[:, :n], cu.cuda(),
                       t.tensor(ids, dtype=t.int32).cuda(), max_new or max(new), yd[:, :rows],
                       out=None if in_place else od[:, :rows], work=work)
    t.cuda.synchronize()
    end = sum(new)
    assert t.equal(od[end:, :rows].cpu(), y[end:] if in_place else t.full((2, rows), 9.0)), "rows behind the last request"
    assert (od[:, rows:] == 9.0).all(), "between the rows"
    for r, i in enumerate(ids):
        s = slice(int(cu[r]), int(cu[r + 1]))
        got = od[s, :rows].cpu()
        if 0 <= i < count:
            within(got, *adapters_ref(x[s], a[i], b[i], gain[i], y[s]), (r, i))
        else:
            assert t.equal(got, y[s]), (r, i)
    return od


@pytest.mark.parametrize("new,ids,n,rows,rank,count,x_type,type", CASES)
def test_adapters(new, ids, n, rows, rank, count, x_type, type):
    run(new, ids, n, rows, rank, count, x_type, type)


@pytest.mark.parametrize("in_place", [False, True])
def test_adapters_strided(in_place):
    for new in ([1, 1, 1], [40, 1, 9]):
        run(new, [1, -1, 0], 264, 100, 16, 2, "f32", "bf16", pad=8, in_place=in_place)


def test_adapters_bound_only_splits_the_work():
    t = torch()
    outs = [run([5, 70, 1], [0, 1, 0], 512, 200, 16, 2, "f32", "bf16", max_new=m) for m in (1, 70, 10000)]
    assert all(o is not None for o in outs)


def test_adapters_many_requests():
    """More requests than a wavefront has lanes: one row each, and up to forty."""
    import random
    r = random.Random(1)
    ids = [r.randint(-1, 3) for _ in range(150)]
    run([r.randint(0, 2) for _ in ids], ids, 264, 70, 16, 4, "f32", "bf16")
    run([r.choice((0, 1, 2, 40)) for _ in ids], ids, 264, 70, 16, 4, "f32", "f16")


@pytest.mark.parametrize("size", [1e-20, 1e6, 1e15])
def test_adapters_f32_rows_of_any_size(size):
    """x far outside f16's range through f16 adapters."""
    run([1, 30], [1, 0], 512, 96, 16, 2, "f32", "f16", size=size)
    run([1, 30], [1, 0], 512, 96, 16, 2, "f32", "bf16", size=size)


def test_adapters_scratch():
    t, bq = torch(), bqmod()
    args = ([1, 30], [1, 0], 512, 96, 16, 2, "f32", "bf16")
    p = bq.Adapters(t.zeros(2, 16, 512, dtype=t.bfloat16, device="cuda"),
                    t.zeros(2, 96, 16, dtype=t.bfloat16, device="cuda"), t.zeros(2, device="cuda"))
    need = bq.bq_adapters_work_bytes(p, 33, 2, 30)
    work = t.full((need // 4,), float("nan"), device="cuda")
    assert t.equal(run(*args, work=work), run(*args))
    with pytest.raises(bq.BQError) as e:
        run(*args, work=work[4:])
    assert "work" in str(e.value)


def test_adapters_refusals():
    t, bq = torch(), bqmod()
    a, b = t.zeros(2, 8, 64, dtype=t.half, device="cuda"), t.zeros(2, 32, 8, dtype=t.half, device="cuda")
    gain = t.ones(2, device="cuda")
    p = bq.Adapters(a, b, gain)
    x, y = t.zeros(3, 64, device="cuda"), t.zeros(3, 32, device="cuda")
    cu, ids = t.tensor([0, 3], dtype=t.int32).cuda(), t.tensor([0], dtype=t.int32).cuda()

    def refused(text, *args, **kw):
        with pytest.raises(bq.BQError) as e:
            bq.bq_adapters_add(*args, **kw)
        assert e.value.code in (bq.BQ_EARG, bq.BQ_EALIGN) and text in str(e.value), str(e.value)

    refused("x", p, x[:, :32], cu, ids, 3, y)
    refused("x_type", p, x.bfloat16(), cu, ids, 3, y)
    refused("y", p, x, cu, ids, 3, y.half())
    refused("y", p, x, cu, ids, 3, y[:2])
    refused("cu", p, x, cu.long(), ids, 3, y)
    refused("ids", p, x, cu, ids.long(), 3, y)
    refused("max_new", p, x, cu, ids, 0, y)
    for what, aa, bb in (("rank", t.zeros(2, 12, 64, dtype=t.half, device="cuda"), t.zeros(2, 32, 12, dtype=t.half, device="cuda")),
                         ("rank", t.zeros(2, 136, 64, dtype=t.half, device="cuda"), t.zeros(2, 32, 136, dtype=t.half, device="cuda"))):
        refused(what, bq.Adapters(aa, bb, gain), x, cu, ids, 3, y)
    with pytest.raises(bq.BQError):
        bq.Adapters(a, b.float(), gain)
    with pytest.raises(bq.BQError):
        bq.Adapters(a, b[:1], gain)
    bq.bq_adapters_add(p, x[:0], cu[:1], ids[:0], 1, y[:0])
