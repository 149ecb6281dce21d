"""bq_paged_attn against the formula in 64 bits, every output within a bound
made of its roundings: one token to long chunks, whole prompts, ragged batches,
requests without rows or keys, rows that see no key, every page size, head
grouping and type; pages and places that hold no token are NaN."""
import pytest

from gpu_util import bqmod, torch
from layer_util import DT, Paged, attn_ref, gen, normal, within

pytestmark = pytest.mark.gpu


def attend(new, keys, Hq, H, D, type, cache, page, seed, max_new=None, max_keys=None, pad=0, cols=None, work=None,
           scale=None, spread=1.5):
    """(out, reference, bound) with two rows behind the last request."""
    t, bq = torch(), bqmod()
    dt, ct = DT[type], DT[cache]
    p = Paged(keys, H, D, page, ct, seed, cols, spread)
    g = gen(seed + 1)
    T = sum(new) + 2
    q = normal(g, T, Hq, D, dtype=dt)
    cu = t.tensor([0] + list(new)).cumsum(0).to(t.int32)
    scale = D ** -0.5 if scale is None else scale
    rows = t.full((T, Hq * D + pad), 3.0, dtype=dt, device="cuda")
    qd = t.empty(T, Hq * D + pad, dtype=dt, device="cuda")
    qd[:, :Hq * D] = q.flatten(1)
    wide = t.cat([p.table, t.full((len(keys), 3), -9, dtype=t.int32)], 1).cuda()
    bq.bq_paged_attn(bq.KVCache(p.k.cuda(), p.v.cuda()), qd[:, :Hq * D].unflatten(1, (Hq, D)), cu.cuda(),
                     t.tensor(keys, dtype=t.int32).cuda(), wide[:, :p.table.shape[1]], scale, max_new or max(max(new), 1),
                     max_keys if max_keys is not None else max(keys), rows[:, :Hq * D].unflatten(1, (Hq, D)), work=work)
    t.cuda.synchronize()
    assert (rows[sum(new):] == 3.0).all(), "rows behind the last request"
    assert (rows[:, Hq * D:] == 3.0).all(), "between the rows"
    out = rows[:sum(new), :Hq * D].unflatten(1, (Hq, D)).cpu()
    refs = [attn_ref(q[cu[b]:cu[b + 1]], p.k_of[b], p.v_of[b], keys[b], scale, dt) for b in range(len(keys))]
    return out, t.cat([r[0] for r in refs]), t.cat([r[1] for r in refs])


def check(*a, **k):
    within(*attend(*a, **k), (a, k))


TYPES = [("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")]


@pytest.mark.parametrize("type,cache", TYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_one_token(type, cache, D):
    """Decode over caches of 0, 1 and lengths around the tile and page sizes."""
    keys = [1, 0, 15, 16, 17, 31, 32, 33, 127, 128, 129, 1000, 2, 511]
    check([1] * len(keys), keys, 8, 2, D, type, cache, 16, 1)


@pytest.mark.parametrize("type,cache", TYPES)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages(type, cache, page):
    """Chunks, some requests without new rows, keys that end inside a page."""
    check([3, 0, 70, 1, 20], [300, 50, 333, 1, 20], 4, 2, 64, type, cache, page, page)


@pytest.mark.parametrize("type,cache", TYPES)
@pytest.mark.parametrize("Hq,H", [(1, 1), (3, 1), (7, 1), (16, 1), (10, 2), (8, 8), (32, 2), (12, 4)])
def test_head_groups(type, cache, Hq, H):
    check([1, 5, 2], [260, 131, 77], Hq, H, 128, type, cache, 32, Hq)
    check([40, 9], [40, 300], Hq, H, 128, type, cache, 16, Hq + 1)


@pytest.mark.parametrize("type,cache", TYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_prompts(type, cache, D):
    """Whole prompts packed together, odd lengths, one of a single token."""
    check([200, 1, 333, 64], [200, 1, 333, 64], 4, 1, D, type, cache, 64, 11)
    check([129], [900], 8, 2, D, type, cache, 16, 12)
    check([257, 0, 31], [800, 0, 1500], 4, 2, D, type, cache, 128, 13)


@pytest.mark.parametrize("type,cache", TYPES)
def test_rows_that_see_nothing(type, cache):
    """More new rows than keys: the first ones are 0."""
    new, keys = [5, 40, 3, 100], [2, 1, 0, 70]
    out, want, bound = attend(new, keys, 4, 2, 64, type, cache, 16, 21)
    within(out, want, bound, "rows")
    assert (out[:3] == 0).all() and (out[5:44] == 0).all() and (out[45:48] == 0).all() and (out[48:78] == 0).all()


@pytest.mark.parametrize("type,cache", TYPES)
@pytest.mark.parametrize("new,keys", [([1], [9000]), ([1, 1], [9000, 3]), ([6], [5000]), ([16], [4097]), ([64], [6000])])
def test_long_keys_split(type, cache, new, keys):
    """Few rows over many keys: the work is split over the keys and joined."""
    check(new, keys, 8, 2, 128, type, cache, 16, 31)


@pytest.mark.parametrize("type,cache", TYPES)
def test_bounds_only_split_the_work(type, cache):
    """max_new and max_keys below and far above the true counts."""
    for new, keys in (([3, 70], [500, 900]), ([1, 1], [700, 64])):
        for mn, mk in ((1, 1), (1, 0), (1000, 100000), (max(new), max(keys))):
            check(new, keys, 4, 1, 64, type, cache, 32, 41, max_new=mn, max_keys=mk)


@pytest.mark.parametrize("type,cache", TYPES)
def test_more_rows_than_max_new_says(type, cache):
    """Enough for the kernel of many rows, but a fraction of the true counts:
    its workgroups walk several tiles each, of several requests."""
    check([600, 3, 40, 700], [600, 300, 900, 1100], 8, 2, 64, type, cache, 16, 45, max_new=20, max_keys=64)
    # split over the keys as well: the tiles that the scratch has no place for are not
    check([600, 3, 40, 700], [600, 300, 900, 5100], 8, 2, 64, type, cache, 16, 48, max_new=20, max_keys=4000)
    check([900], [6000], 8, 2, 64, type, cache, 16, 49, max_new=20, max_keys=4000)


@pytest.mark.parametrize("type,cache", [("f32", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("requests", [65, 130, 300])
def test_many_requests(type, cache, requests):
    """More requests than a wavefront has lanes, decode tokens and chunks among
    each other, some empty."""
    import random
    r = random.Random(requests)
    keys = [r.choice((0, 1, 17, 64, 300, r.randint(1, 2000))) for _ in range(requests)]
    check([r.choice((0, 1, 1, 1)) for _ in keys], keys, 4, 2, 64, type, cache, 16, 46)
    new = [r.choice((0, 1, 1, 5, 40)) for _ in keys]
    check(new, [max(k, n) for k, n in zip(keys, new)], 4, 2, 64, type, cache, 32, 47)


@pytest.mark.parametrize("type,cache", TYPES)
def test_strides_and_wide_tables(type, cache):
    check([2, 33], [100, 250], 6, 2, 64, type, cache, 16, 51, pad=64, cols=40)


@pytest.mark.parametrize("type,cache", TYPES)
def test_peaked_and_large_scores(type, cache):
    """One weight takes all; scores of hundreds; a negative and a zero scale."""
    check([1, 50], [600, 300], 4, 2, 64, type, cache, 16, 61, spread=20.0, scale=1.0)
    check([1, 50], [600, 300], 4, 2, 64, type, cache, 16, 62, scale=-0.5)
    check([1, 50], [600, 300], 4, 2, 64, type, cache, 16, 63, scale=0.0)


def test_f32_rows_of_any_size():
    """f32 queries far outside f16's range over an f16 cache."""
    t, bq = torch(), bqmod()
    p = Paged([100], 1, 64, 16, t.float16, 71)
    for size in (1e-30, 1e-6, 1e5, 1e12):
        q = normal(gen(72), 3, 2, 64, scale=size)
        q[1, :, 3] = 0
        q[2, 1] = 0
        out = t.empty(3, 2, 64, device="cuda")
        scale = 0.125 / size
        bq.bq_paged_attn(bq.KVCache(p.k.cuda(), p.v.cuda()), q.cuda(), t.tensor([0, 3], dtype=t.int32).cuda(),
                         t.tensor([100], dtype=t.int32).cuda(), p.table.cuda(), scale, 3, 100, out)
        import numpy as np
        want, bound = attn_ref(q, p.k_of[0], p.v_of[0], 100, float(np.float32(scale)), t.float32)
        within(out, want, bound, size)


def test_pages_outside_the_cache_count_as_unseen():
    """A bad table entry inside the keys is not read: its keys are left out."""
    t, bq = torch(), bqmod()
    for bad in (-1, 1 << 20, -(1 << 31)):
        for n in (1, 50):
            p = Paged([200], 2, 64, 16, t.bfloat16, 81)
            q = normal(gen(82), n, 4, 64)
            p.table[0, 3] = bad
            out = t.empty(n, 4, 64, device="cuda")
            bq.bq_paged_attn(bq.KVCache(p.k.cuda(), p.v.cuda()), q.cuda(), t.tensor([0, n], dtype=t.int32).cuda(),
                             t.tensor([200], dtype=t.int32).cuda(), p.table.cuda(), 0.125, n, 200, out)
            keep = t.cat([t.arange(48), t.arange(64, 200)])
            want, bound = attn_ref(q, p.k_of[0][keep], p.v_of[0][keep], 184, 0.125, t.float32)
            # the kept keys are 0..47 and 64..199: the last n rows see the same ones as over 184 keys
            within(out, want, bound, (bad, n))


def test_lengths_beyond_the_table_and_rows():
    """lens above the table's keys and offsets above the rows are bounded."""
    t, bq = torch(), bqmod()
    p = Paged([64, 64], 1, 64, 16, t.float16, 91)
    q = normal(gen(92), 4, 1, 64, dtype=t.float16)
    out = t.full((4, 1, 64), 5.0, dtype=t.float16, device="cuda")
    bq.bq_paged_attn(bq.KVCache(p.k.cuda(), p.v.cuda()), q.cuda(), t.tensor([0, 1, 400], dtype=t.int32).cuda(),
                     t.tensor([1 << 30, -5], dtype=t.int32).cuda(), p.table.cuda(), 0.125, 3, 64, out)
    want, bound = attn_ref(q[:1], p.k_of[0], p.v_of[0], 64, 0.125, t.float16)
    within(out[:1], want, bound, "the table's 64 keys")
    assert (out[1:] == 0).all()


def test_scratch_is_not_read_before_written():
    """A dirty scratch of the exact size gives the same bits, call after call."""
    t, bq = torch(), bqmod()
    kv = bq.KVCache.empty(1, 2, 128, 16, t.bfloat16)
    need = bq.bq_paged_attn_work_bytes(kv, 5, 8, 2, 3, 4000)
    assert need > 0 and need % 4 == 0
    work = t.full((need // 4,), float("nan"), device="cuda")
    first = attend([3, 0], [4000, 10], 8, 2, 128, "f32", "bf16", 16, 95, work=work)[0]
    again = attend([3, 0], [4000, 10], 8, 2, 128, "f32", "bf16", 16, 95)[0]
    assert t.equal(first, again)
    with pytest.raises(bq.BQError) as e:
        attend([3, 0], [4000, 10], 8, 2, 128, "f32", "bf16", 16, 95, work=work[1:])
    assert "work" in str(e.value)


def test_far_pages():
    """Pages whose byte offset passes 32 bits."""
    t, bq = torch(), bqmod()
    H, D, page, pages = 8, 128, 16, (1 << 31) // (8 * 128 * 16) + 40
    k = t.zeros(pages, H, page, D, dtype=t.bfloat16, device="cuda")
    v = t.zeros(pages, H, D, page, dtype=t.bfloat16, device="cuda")
    p = Paged([100], H, D, page, t.bfloat16, 96)
    n = p.k.shape[0]
    k[-n:] = p.k.cuda()
    v[-n:] = p.v.cuda()
    for new in (1, 70):
        q = normal(gen(97), new, 16, D, dtype=t.bfloat16)
        out = t.empty(new, 16, D, dtype=t.bfloat16, device="cuda")
        bq.bq_paged_attn(bq.KVCache(k, v), q.cuda(), t.tensor([0, new], dtype=t.int32).cuda(),
                         t.tensor([100], dtype=t.int32).cuda(), (p.table + (pages - n)).cuda(), 0.1, new, 100, out)
        want, bound = attn_ref(q, p.k_of[0], p.v_of[0], 100, float(t.tensor(0.1)), t.bfloat16)
        within(out, want, bound, new)


def test_attn_refusals():
    t, bq = torch(), bqmod()
    kv = bq.KVCache.empty(4, 2, 64, 16, t.bfloat16)
    q = t.zeros(3, 4, 64, device="cuda")
    cu, lens = t.tensor([0, 3], dtype=t.int32).cuda(), t.tensor([3], dtype=t.int32).cuda()
    table = t.zeros(1, 4, dtype=t.int32, device="cuda")
    out = t.empty_like(q)

    def refused(text, *a, **kw):
        with pytest.raises(bq.BQError) as e:
            bq.bq_paged_attn(*a, **kw)
        assert e.value.code in (bq.BQ_EARG, bq.BQ_EALIGN) and text in str(e.value), str(e.value)

    refused("q_heads", kv, q[:, :3].contiguous(), cu, lens, table, 1.0, 3, 3, out[:, :3].contiguous())
    refused("type", kv, q.half(), cu, lens, table, 1.0, 3, 3, out.half())
    refused("out", kv, q, cu, lens, table, 1.0, 3, 3, out.bfloat16())
    refused("out must not be q", kv, q, cu, lens, table, 1.0, 3, 3, q)
    refused("cu", kv, q, cu[:1], lens, table, 1.0, 3, 3, out)
    refused("lens", kv, q, cu, lens.long(), table, 1.0, 3, 3, out)
    refused("table", kv, q, cu, lens, table.long(), 1.0, 3, 3, out)
    refused("max_new", kv, q, cu, lens, table, 1.0, 0, 3, out)
    refused("max_keys", kv, q, cu, lens, table, 1.0, 3, -1, out)
    refused("scale", kv, q, cu, lens, table, float("inf"), 3, 3, out)
    refused("q_heads", kv, t.zeros(3, 34, 64, device="cuda"), cu, lens, table, 1.0, 3, 3, t.empty(3, 34, 64, device="cuda"))
    bq.bq_paged_attn(kv, q[:0], cu[:1], lens[:0], table[:0], 1.0, 1, 1, out[:0])
