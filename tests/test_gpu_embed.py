"""bq_embed against the table's values: every product is rounded once to f32 and
once to the output's type, so the rows are compared bit for bit."""
import numpy as np
import pytest

import synth
from gpu_util import bqmod, torch
from layer_util import DT, gen, normal
from model_util import codes

pytestmark = pytest.mark.gpu


def run(table, ids, n, dt, scale, pad=0, **k):
    t, bq = torch(), bqmod()
    out = t.full((len(ids), n + pad), 7.0, dtype=dt, device="cuda")
    bq.bq_embed(table, t.tensor(ids, dtype=t.int64, device="cuda"), out[:, :n], scale=scale, **k)
    t.cuda.synchronize()
    assert (out[:, n:] == 7.0).all()
    return out[:, :n].cpu()


def wanted(rows, ids, dt, scale):
    """rows f32 [count, n] (numpy), ids out of range give zeros."""
    t = torch()
    out = np.zeros((len(ids), rows.shape[1]), np.float32)
    for i, r in enumerate(ids):
        if 0 <= r < len(rows):
            with np.errstate(over="ignore"):
                out[i] = rows[r] * np.float32(scale)
    return t.from_numpy(out).to(dt)


def same(got, want):
    t = torch()
    bits = t.int32 if got.dtype == t.float32 else t.int16
    assert t.equal(got.view(bits), want.view(bits))


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("count,blocks,dt,scale", [
    (1, 1, "f32", 1.0), (63, 3, "bf16", -0.3), (64, 8, "f16", 2.0 ** -20), (1000, 9, "f32", 1e30), (700, 33, "bf16", 11.313708)])
def test_packed_rows(fmt, count, blocks, dt, scale):
    t, bq = torch(), bqmod()
    n = blocks * bq.BLOCK_LEN[fmt]
    canon = (synth.q2_0_blocks_all_codes if fmt == 2 else synth.q1_0_blocks)(count, n, 3, blocks)
    w, d = codes(fmt, canon)
    rows = (w * d[..., None]).reshape(count, n).astype(np.float32)
    ids = [0, count - 1, -1, count, 1 << 40, -(1 << 40), count // 2, 0] + list(range(min(count, 70)))
    table = bq.Weights.upload(fmt, canon, count, n)
    same(run(table, ids, n, DT[dt], scale), wanted(rows, ids, DT[dt], scale))
    same(run(table, ids[:1], n, DT[dt], scale), wanted(rows, ids[:1], DT[dt], scale))


@pytest.mark.parametrize("table_type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("count,n,tokens", [(1, 8, 1), (50, 520, 300), (3, 4096, 5)])
def test_dense_rows(table_type, dt, count, n, tokens):
    t = torch()
    g = gen(count + n)
    wide = normal(g, count, n + 16, dtype=DT[table_type])
    table = wide[:, :n]  # rows further apart than they are long
    ids = t.randint(-1, count + 1, (tokens,), generator=g).tolist()
    got = run(table.cuda() if count == 1 else wide.cuda()[:, :n], ids, n, DT[dt], 1.7, pad=8)
    same(got, wanted(table.float().numpy(), ids, DT[dt], 1.7))


def test_large_offsets():
    """A table and an output whose elements pass 2^31 bytes, and 2^32."""
    t, bq = torch(), bqmod()
    n, count = 4096, 600000
    table = t.zeros(count, n, dtype=t.bfloat16, device="cuda")  # 4.9 GB
    ids = t.tensor([count - 1, 1, count - 2], dtype=t.int64, device="cuda")
    table[ids] = t.tensor([3.0, 5.0, 7.0], device="cuda").bfloat16()[:, None]
    out = t.empty(3, n, device="cuda")
    bq.bq_embed(table, ids, out, scale=2.0)
    assert t.equal(out[:, 0].cpu(), t.tensor([6.0, 10.0, 14.0])) and (out == out[:, :1]).all()
    del table
    many = t.full((300000,), -1, dtype=t.int64, device="cuda")  # 4.9 GB of rows
    many[-1] = 0
    out = t.empty(300000, n, device="cuda")
    bq.bq_embed(t.ones(1, n, device="cuda"), many, out)
    assert (out[-1] == 1).all() and (out[:-1] == 0).all()


def test_refusals():
    t, bq = torch(), bqmod()
    x, ids = t.zeros(4, 64, device="cuda"), t.zeros(4, dtype=t.int64, device="cuda")
    ok = t.zeros(4, 64, device="cuda")
    for args in ((x, ids.int(), ok), (x, ids, ok[:, :32]), (x, ids, ok.double()), (x, ids[None], ok), (x[0], ids, ok),
                 (x.cpu(), ids, ok), (x, ids, ok.t()), (x, ids.cpu(), ok), (x[:, ::2], ids, ok[:, :32].contiguous())):
        with pytest.raises(bq.BQError):
            bq.bq_embed(*args)
    with pytest.raises(bq.BQError):
        bq.bq_embed(x, ids, ok, scale=float("nan"))
