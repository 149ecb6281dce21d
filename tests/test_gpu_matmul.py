"""bq_matmul against 64-bit sums, element by element within a bound counted from
its roundings (model_util.matmul_ref)."""
import numpy as np
import pytest

import synth
from gpu_util import bqmod, torch
from layer_util import DT, gen, normal, within
from model_util import ACTS, matmul_ref

pytestmark = pytest.mark.gpu


def acts(T, cols, qa, seed, pad=0):
    """Quantized activations as the quantizer leaves them (largest quant of a block 127): q, d on the host."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((T, cols // qa, qa)).astype(np.float32) * np.exp2(g.integers(-6, 6, (T, cols // qa, 1))).astype(np.float32)
    d = np.abs(x).max(2) / np.float32(127)
    return np.rint(x / d[..., None]).astype(np.int8).reshape(T, cols), d


def run(w, q, d, qa, dt, bias=None, act="none", mul=None, res=None, pad=0, y=None, **k):
    t, bq = torch(), bqmod()
    T, cols = q.shape
    if pad:  # rows of the activations further apart than they are long
        qq, dd = t.full((T, cols + 16 * pad), 77, dtype=t.int8, device="cuda"), t.full((T, cols // qa + pad), 1e30, device="cuda")
        qq[:, :cols], dd[:, :cols // qa] = t.from_numpy(q).cuda(), t.from_numpy(d).cuda()
    else:
        qq, dd = t.from_numpy(q).cuda(), t.from_numpy(d).cuda()
    whole = t.full((T, w.rows + pad), 7.0, dtype=dt, device="cuda")
    bq.bq_matmul(w, bq.Act(qq, dd, cols, qa, T), whole[:, :w.rows], bias=None if bias is None else bias.cuda(), act=ACTS[act],
                 mul=None if mul is None else mul.cuda(), res=None if res is None else res.cuda(), **k)
    t.cuda.synchronize()
    assert (whole[:, w.rows:] == 7.0).all()
    return whole[:, :w.rows].cpu()


SHAPES = [(1, 1, 128), (16, 64, 256), (17, 65, 128), (33, 130, 1152), (64, 96, 640), (127, 200, 384), (129, 31, 896),
          (300, 513, 512), (257, 1024, 128), (520, 260, 2304)]


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("qa", [32, 64, 128])
@pytest.mark.parametrize("T,rows,cols", SHAPES)
def test_products(fmt, qa, T, rows, cols):
    bq = bqmod()
    canon = synth.blocks(fmt, rows, cols, 7, T)
    q, d = acts(T, cols, qa, T + rows)
    y = run(bq.Weights.upload(fmt, canon, rows, cols), q, d, qa, DT["f32"], pad=(T % 2) * 3)
    within(y, *matmul_ref(fmt, canon, q, d, qa, DT["f32"]), (fmt, qa, T, rows, cols))


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("qa", [32, 64, 128])
@pytest.mark.parametrize("T,rows,cols", [(600, 2000, 128), (601, 2001, 384), (1025, 1030, 640), (2100, 2600, 256), (4100, 1500, 896)])
def test_many_tokens(fmt, qa, T, rows, cols):
    """Enough tiles for the kernels of 32 and of 64 tokens a workgroup, ends inside a tile on both sides."""
    bq = bqmod()
    canon = synth.blocks(fmt, rows, cols, 7, T)
    q, d = acts(T, cols, qa, T + rows)
    y = run(bq.Weights.upload(fmt, canon, rows, cols), q, d, qa, DT["f32"], pad=(T % 2) * 3)
    within(y, *matmul_ref(fmt, canon, q, d, qa, DT["f32"]), (fmt, qa, T, rows, cols))


@pytest.mark.parametrize("qa", [32, 64])
@pytest.mark.parametrize("T", [600, 2200])
def test_many_tokens_odd_number_of_blocks(qa, T):
    bq = bqmod()
    for cols in (64, 320):
        canon = synth.q2_0_blocks_all_codes(2500, cols, 3, T)
        q, d = acts(T, cols, qa, T)
        y = run(bq.Weights.upload(2, canon, 2500, cols), q, d, qa, DT["f32"])
        within(y, *matmul_ref(2, canon, q, d, qa, DT["f32"]), (qa, T, cols))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu2"])
@pytest.mark.parametrize("T", [601, 2150])
def test_many_tokens_epilogues(dt, act, T):
    bq = bqmod()
    rows, cols, qa, g = 2049, 256, 64, gen(T)
    canon = synth.blocks(1, rows, cols, 8, T)
    w = bq.Weights.upload(1, canon, rows, cols)
    q, d = acts(T, cols, qa, 3)
    d = d * np.float32(0.3)
    bias, mul, res = normal(g, rows), normal(g, T, rows, dtype=DT[dt]), normal(g, T, rows, dtype=DT[dt])
    y = run(w, q, d, qa, DT[dt], bias, act, mul, res, pad=3)
    within(y, *matmul_ref(1, canon, q, d, qa, DT[dt], bias, act, mul, res), (act, dt))


@pytest.mark.parametrize("qa", [32, 64])
@pytest.mark.parametrize("T", [5, 40, 130, 400])
@pytest.mark.parametrize("cols", [64, 192, 576, 1088])
def test_odd_number_of_blocks(qa, T, cols):
    """Q2_0 rows that end in the middle of a step of 128."""
    bq = bqmod()
    canon = synth.q2_0_blocks_all_codes(150, cols, 3, T)
    q, d = acts(T, cols, qa, T)
    y = run(bq.Weights.upload(2, canon, 150, cols), q, d, qa, DT["f32"])
    within(y, *matmul_ref(2, canon, q, d, qa, DT["f32"]), (qa, T, cols))


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu2"])
@pytest.mark.parametrize("T,rows", [(9, 100), (200, 333)])
def test_epilogues(fmt, dt, act, T, rows):
    bq = bqmod()
    cols, qa, g = 512, 128, gen(T)
    canon = synth.blocks(fmt, rows, cols, 8, T)
    w = bq.Weights.upload(fmt, canon, rows, cols)
    q, d = acts(T, cols, qa, 3)
    d = d * np.float32(0.3)
    bias, mul, res = normal(g, rows), normal(g, T, rows, dtype=DT[dt]), normal(g, T, rows, dtype=DT[dt])
    for b in (None, bias):
        for m in (None, mul):
            for r in (None, res):
                y = run(w, q, d, qa, DT[dt], b, act, m, r)
                within(y, *matmul_ref(fmt, canon, q, d, qa, DT[dt], b, act, m, r), (act, dt, b is None, m is None, r is None))


@pytest.mark.parametrize("T", [4, 150])
def test_in_place(T):
    """y over the residual, and over the gate."""
    t, bq = torch(), bqmod()
    canon = synth.q1_0_blocks(100, 256, 1)
    w = bq.Weights.upload(1, canon, 100, 256)
    q, d = acts(T, 256, 128, 1)
    a = bq.Act(t.from_numpy(q).cuda(), t.from_numpy(d).cuda(), 256, 128, T)
    other = normal(gen(1), T, 100)
    for name in ("res", "mul"):
        want = run(w, q, d, 128, t.float32, act="silu", **{name: other})
        y = other.cuda()
        bq.bq_matmul(w, a, y, act=bq.BQ_SILU, **{name: y})
        assert t.equal(y.cpu(), want)


@pytest.mark.parametrize("T", [3, 200])
def test_int8_ends_and_scales(T):
    """Quants of -128 (times -1: +128), largest sums of a block, zero activation scales, zero and subnormal weight scales."""
    t, bq = torch(), bqmod()
    for fmt in (1, 2):
        canon = synth.blocks(fmt, 70, 512, 2)
        canon[0, :, 2:], canon[1, :, 2:] = (0xFF, 0) if fmt == 1 else (0xAA, 0)  # all +1, all -1
        canon[2, :, :2] = 0
        canon[3, :, 0], canon[3, :, 1] = 1, 0  # the smallest subnormal f16
        q, d = acts(T, 512, 128, 4)
        q[0], q[1], q[2] = -128, 127, 0
        d[2] = 0
        y = run(bq.Weights.upload(fmt, canon, 70, 512), q, d, 128, t.float32)
        want, bound = matmul_ref(fmt, canon, q, d, 128, t.float32)
        within(y, want, bound, fmt)
        assert (y[2] == 0).all() and (y[:, 2] == 0).all() and y[0, 1] > 0


@pytest.mark.parametrize("fmt", [1, 2])
def test_near_the_single_products(fmt):
    """The same numbers as bq_q1_0_matvec / bq_q2_0_matvec to f32 sums, whatever the number of tokens beside a token."""
    t, bq = torch(), bqmod()
    rows, cols, qa = 320, 1024, 128
    canon = synth.blocks(fmt, rows, cols, 9)
    w = bq.Weights.upload(fmt, canon, rows, cols)
    q, d = acts(200, cols, qa, 5)
    _, bound = matmul_ref(fmt, canon, q[:16], d[:16], qa, t.float32)
    y = t.empty(16, rows, device="cuda")
    (bq.bq_q1_0_matvec if fmt == 1 else bq.bq_q2_0_matvec)(w, bq.Act(t.from_numpy(q[:16]).cuda(), t.from_numpy(d[:16]).cuda(), cols, qa, 16), y)
    q, d = np.tile(q, (20, 1)), np.tile(d, (20, 1))
    for T in (16, 40, 200, 4000):
        within(run(w, q[:T], d[:T], qa, t.float32)[:16], y.cpu(), 2 * bound, T)


@pytest.mark.parametrize("T,rows", [(20, 300), (300, 300), (610, 2000), (2200, 2500)])
def test_streams_scratch_and_graphs(T, rows):
    """On another stream, with the caller's scratch, two calls at once, and captured and replayed: the same bits."""
    t, bq = torch(), bqmod()
    canon = synth.q2_0_blocks(rows, 1024, 1)
    w = bq.Weights.upload(2, canon, rows, 1024)
    q, d = acts(T, 1024, 64, 6)
    a = bq.Act(t.from_numpy(q).cuda(), t.from_numpy(d).cuda(), 1024, 64, T)
    want = run(w, q, d, 64, t.float32)
    need = bq.bq_matmul_work_bytes(w, T, 64)
    works = [t.empty(need, dtype=t.uint8, device="cuda") for _ in range(2)]
    ys = [t.zeros(T, rows, device="cuda") for _ in range(2)]
    streams = [t.cuda.Stream() for _ in range(2)]
    t.cuda.synchronize()
    for _ in range(3):
        for s, y, work in zip(streams, ys, works):
            bq.bq_matmul(w, a, y, work=work, stream=s)
    t.cuda.synchronize()
    assert t.equal(ys[0].cpu(), want) and t.equal(ys[1].cpu(), want)
    y = t.zeros(T, rows, device="cuda")
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        bq.bq_matmul(w, a, y, work=works[0])
    for i in range(4):
        y.fill_(i)
        a.q.copy_(t.from_numpy(np.roll(q, i, axis=0)))
        a.d.copy_(t.from_numpy(np.roll(d, i, axis=0)))
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(y.cpu(), t.from_numpy(np.roll(want.numpy(), i, axis=0))), i


def test_large_offsets():
    """Outputs whose byte offsets pass 2^31 and 2^32: 40000 rows of 30001 tokens."""
    t, bq = torch(), bqmod()
    rows, T = 40000, 30001  # 4.8 GB of f32
    canon = synth.q1_0_blocks(rows, 128, 1)
    w = bq.Weights.upload(1, canon, rows, 128)
    q, d = acts(T, 128, 128, 1)
    y = t.empty(T, rows, device="cuda")
    bq.bq_matmul(w, bq.Act(t.from_numpy(q).cuda(), t.from_numpy(d).cuda(), 128, 128, T), y)
    for at in (slice(0, 3), slice(T - 40, T)):
        within(y[at].cpu(), *matmul_ref(1, canon, q[at], d[at], 128, t.float32), at)


def test_refusals():
    t, bq = torch(), bqmod()
    w = bq.Weights.upload(1, synth.q1_0_blocks(64, 256, 1), 64, 256)
    q, d, y = t.zeros(4, 256, dtype=t.int8, device="cuda"), t.zeros(4, 2, device="cuda"), t.zeros(4, 64, device="cuda")
    a = bq.Act(q, d, 256, 128, 4)
    for args, k in (((w, a, y[:, :32]), {}), ((w, a, y.double()), {}), ((w, a, y.cpu()), {}), ((w, a, y.t()), {}), ((w, a, None), {}),
                    ((w, a, y), {"bias": y[0].half()}), ((w, a, y), {"bias": y[0, :32]}), ((w, a, y), {"mul": y.half()}),
                    ((w, a, y), {"res": y[:2]}), ((w, a, y), {"act": 7}), ((w, bq.Act(q[:, :128].contiguous(), d, 128, 128, 4), y), {})):
        with pytest.raises(bq.BQError):
            bq.bq_matmul(*args, **k)
