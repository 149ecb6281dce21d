"""bq_kv_append against the formulas in 64 bits: keys and queries normed and
rotated, values transposed into their pages, every place that no token names
left as it was; all types, page and head sizes, partial rotation, far
positions, places in runs and out of order, padded rows, rows with gaps."""
import pytest

from gpu_util import bqmod, torch
from layer_util import DT, gen, half_step, normal, rotate_ref, within

pytestmark = pytest.mark.gpu

# tokens, q_heads, heads, dim, rot, type, cache, page, norms, q_out type, first position, places
CASES = [
    (1, 32, 8, 128, 128, "f32", "bf16", 16, True, "f32", 40000, "run"),
    (1, 1, 1, 64, 64, "bf16", "bf16", 16, False, "bf16", 0, "run"),
    (16, 32, 8, 128, 128, "f32", "bf16", 16, True, "bf16", 131000, "mixed"),
    (17, 5, 1, 64, 32, "f32", "f16", 32, False, "f16", 1 << 20, "run"),
    (40, 6, 2, 128, 16, "f16", "f16", 64, True, "f16", 77, "padded"),
    (131, 8, 8, 64, 64, "bf16", "bf16", 128, True, "bf16", 5, "run"),
    (64, 0, 3, 128, 128, "f32", "f16", 256, True, None, 9, "aligned"),
    (600, 7, 1, 128, 96, "bf16", "bf16", 16, False, "bf16", 1000, "two"),
    (1030, 16, 4, 64, 48, "f32", "bf16", 32, True, "f32", 2_000_000_000, "padded"),
    (33, 4, 2, 64, 0, "f16", "f16", 16, False, "f16", 3, "mixed"),
]


def places(kind, T, pages, page, g):
    t = torch()
    order = t.randperm(pages, generator=g)

    def of(at):
        return order[at // page] * page + at % page

    at = t.arange(T)
    if kind == "aligned":
        return of(at)
    if kind == "run":
        return of(at + 5)
    if kind == "mixed":
        return t.randperm(pages * page, generator=g)[:T]
    if kind == "two":  # two requests, a run each
        return of(t.where(at < T // 3, at + 3, at + 24))
    slots = of(at + 8)  # padded: rows without a place, one outside the cache
    slots[::3] = -1
    slots[-1] = pages * page
    return slots


@pytest.mark.parametrize("T,Hq,H,D,rot,type,cache,page,norms,q_type,start,kind", CASES)
def test_append(T, Hq, H, D, rot, type, cache, page, norms, q_type, start, kind):
    t, bq = torch(), bqmod()
    g = gen(T + rot)
    dt, ct = DT[type], DT[cache]
    pages = -(-(T + 32) // page) + 2
    k0, v0 = normal(g, pages, H, page, D, dtype=ct), normal(g, pages, H, D, page, dtype=ct)
    # q, k and v as views of one fused projection's rows
    rows = normal(g, T, (Hq + 2 * H) * D, dtype=dt)
    q, k, v = (r.unflatten(1, (-1, D)) if r.shape[1] else None
               for r in rows.split((Hq * D, H * D, H * D), 1))
    slot = places(kind, T, pages, page, g)
    pos = (start + t.arange(T)).to(t.int32)
    freq = (1e4 ** (-t.arange(0, rot, 2).double() / max(rot, 1))).float()
    qn, kn = (normal(g, D, scale=0.1, shift=1.0) if norms else None for _ in range(2))
    dev = rows.cuda()
    qd, kd, vd = (r.unflatten(1, (-1, D)) if r.shape[1] else None for r in dev.split((Hq * D, H * D, H * D), 1))
    kv = bq.KVCache(k0.cuda(), v0.cuda())
    qo = t.full((T, Hq * D + 32), 7.0, dtype=DT[q_type], device="cuda") if Hq else None
    up = lambda x: None if x is None else x.cuda()  # noqa: E731
    bq.bq_kv_append(kv, kd, vd, pos.cuda(), slot.cuda(), freq.cuda(), q=qd,
                    q_out=qo[:, :Hq * D].unflatten(1, (Hq, D)) if Hq else None, q_norm=up(qn), k_norm=up(kn), eps=1e-5)
    t.cuda.synchronize()
    keep = (slot >= 0) & (slot < pages * page)
    at, off = slot[keep] // page, slot[keep] % page
    kr, kb = rotate_ref(k, pos, freq, kn, 1e-5)
    want_k, bound_k = k0.double(), t.zeros(pages, H, page, D, dtype=t.float64)
    want_k[at, :, off] = kr[keep]
    bound_k[at, :, off] = (kb + kr.abs() * half_step(ct) + 2.0 ** -25)[keep]
    within(kv.k, want_k, bound_k, "keys")
    want_v = v0.clone()
    want_v[at, :, :, off] = v[keep].to(ct)
    assert t.equal(kv.v.cpu(), want_v), "values"
    if Hq:
        qr, qb = rotate_ref(q, pos, freq, qn, 1e-5)
        within(qo[:, :Hq * D].unflatten(1, (Hq, D)), qr, qb + qr.abs() * half_step(DT[q_type]) + 2.0 ** -25, "queries")
        assert (qo[:, Hq * D:] == 7.0).all()


def test_append_in_place_and_far_offsets():
    """q_out in place of q; a place whose byte offset passes 32 bits."""
    t, bq = torch(), bqmod()
    g = gen(1)
    H, D, page, pages = 8, 128, 16, (1 << 31) // (8 * 128 * 16) + 40  # more than 2^31 values a plane
    kv = bq.KVCache.empty(pages, H, D, page, t.bfloat16)
    q, k, v = normal(g, 8, 8, D), normal(g, 8, H, D), normal(g, 8, H, D)
    slot = t.cat([(pages - 2) * page + t.arange(4), (pages - 1) * page + 8 + t.arange(4)])
    pos = t.arange(8, dtype=t.int32)
    freq = t.ones(64)
    qd = q.cuda()
    bq.bq_kv_append(kv, k.cuda(), v.cuda(), pos.cuda(), slot.cuda(), freq.cuda(), q=qd, q_out=qd)
    kr, kb = rotate_ref(k, pos, freq, None, 1e-6)
    at, off = (slot // page).cuda(), (slot % page).cuda()
    within(kv.k[at, :, off], kr, kb + kr.abs() * half_step(t.bfloat16) + 1e-30, "keys")
    assert t.equal(kv.v[at, :, :, off].cpu(), v.bfloat16())
    qr, qb = rotate_ref(q, pos, freq, None, 1e-6)
    within(qd, qr, qb + 1e-30, "queries in place")


def test_append_refusals():
    t, bq = torch(), bqmod()
    kv = bq.KVCache.empty(4, 2, 64, 16, t.bfloat16)
    k = t.ones(3, 2, 64, device="cuda")
    pos = t.zeros(3, dtype=t.int32, device="cuda")
    slot = t.arange(3, device="cuda")
    freq = t.ones(32, device="cuda")

    def refused(text, *a, **kw):
        with pytest.raises(bq.BQError) as e:
            bq.bq_kv_append(*a, **kw)
        assert e.value.code in (bq.BQ_EARG, bq.BQ_EALIGN) and text in str(e.value), str(e.value)

    refused("shape", kv, k[:, :1], k, pos, slot, freq)
    refused("type", kv, k.half(), k.half(), pos, slot, freq)
    refused("v must be", kv, k, k.bfloat16(), pos, slot, freq)
    refused("pos", kv, k, k, pos.long(), slot, freq)
    refused("slot", kv, k, k, pos, slot[:2], freq)
    refused("rot", kv, k, k, pos, slot, t.ones(40, device="cuda"))
    refused("rot", kv, k, k, pos, slot, t.ones(4, device="cuda"))
    refused("eps", kv, k, k, pos, slot, freq, k_norm=t.ones(64, device="cuda"), eps=0.0)
    refused("together", kv, k, k, pos, slot, freq, q=k)
    refused("q_out", kv, k, k, pos, slot, freq, q=k, q_out=k.half())
    refused("k_norm", kv, k, k, pos, slot, freq, k_norm=t.ones(128, device="cuda"))
    bq.bq_kv_append(kv, k[:0], k[:0], pos[:0], slot[:0], freq)  # no tokens: nothing to do
    with pytest.raises(bq.BQError):
        bq.KVCache.empty(4, 2, 64, 16, t.bfloat16).__class__(t.empty(4, 2, 16, 64, device="cuda", dtype=t.half),
                                                             t.empty(4, 2, 16, 64, device="cuda", dtype=t.half))
    with pytest.raises(bq.BQError) as e:
        bq.bq_kv_append(bq.KVCache.empty(4, 2, 64, 24, t.bfloat16), k, k, pos, slot, freq)
    assert "page" in str(e.value)
    with pytest.raises(bq.BQError) as e:
        bq.bq_kv_append(bq.KVCache.empty(4, 2, 96, 16, t.bfloat16), t.ones(3, 2, 96, device="cuda"),
                        t.ones(3, 2, 96, device="cuda"), pos, slot, freq)
    assert "dim" in str(e.value)
