"""bq_rmsnorm_q8 against its definition: quants, scales and the stored sum bit
for bit (max|v| * fl(1/127) and v / d step by step; f16-valued scales by the
oracle's narrowing), the normed rows within the roundings of their f32 steps;
every type, block length, scale flavour, with and without residual, in place,
strided, one row to many, 32 to 65536 values."""
import pytest

from gpu_util import bqmod, torch
from layer_util import DT, gen, half_step, norm_ref, normal, within

pytestmark = pytest.mark.gpu

# tokens, n, type, qa, residual, y, f16_scale
CASES = [
    (1, 4096, "f32", 128, True, False, False),
    (1, 32, "f32", 32, True, True, False),
    (1, 65536, "bf16", 64, True, True, False),
    (2, 65536, "f32", 128, True, True, True),
    (3, 128, "f16", 128, False, True, False),
    (5, 96, "bf16", 32, True, False, True),
    (7, 12288, "bf16", 128, True, True, False),
    (16, 4096, "f16", 64, True, True, True),
    (33, 8224, "f32", 32, False, False, True),
    (513, 4160, "f32", 64, True, True, False),
    (600, 16384, "bf16", 32, True, False, False),
    (700, 32, "f16", 32, True, True, False),
    (2, 33024, "f16", 128, True, True, False),
]


def run(x, res, w, qa, y, f16_scale, pad=0, stream=None):
    """Outputs on the host; rows `pad` elements longer than n."""
    t, bq = torch(), bqmod()
    T, n = x.shape

    def strided(v, dtype, cols):
        full = t.full((T, cols + pad), -77, dtype=dtype, device="cuda")
        view = full[:, :cols]
        if v is not None:
            view.copy_(v)
        return full, view

    xs, rs = strided(x, x.dtype, n), strided(res, x.dtype, n)
    hs, ys = strided(None, x.dtype, n), strided(None, x.dtype, n)
    qs, ds = strided(None, t.int8, n), strided(None, t.float32, n // qa)
    bq.bq_rmsnorm_q8(xs[1], w.cuda(), 1e-6, qa, qs[1], ds[1], res=rs[1] if res is not None else None, h=hs[1],
                     y=ys[1] if y else None, f16_scale=f16_scale)
    t.cuda.synchronize()
    for full, cols in ((hs[0], n), (ys[0], n), (qs[0], n), (ds[0], n // qa)):
        assert (full[:, cols:] == -77).all(), "written between the rows"
    return [v[1].cpu() for v in (hs, ys, qs, ds)]


def check(x, res, w, qa, y, f16_scale, pad=0):
    t = torch()
    h, yy, q, d = run(x, res, w, qa, y, f16_scale, pad)
    rh, rv, rq, rd = norm_ref(x, res, w, 1e-6, qa, f16_scale)
    assert t.equal(h, rh)
    assert t.equal(d, rd)
    assert t.equal(q, rq)
    if y:
        assert t.equal(yy, rv.to(x.dtype))
        # and the formula in 64 bits: r, two products, and the rounding to the type
        hd = rh.double()
        full = hd / (hd.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
        within(yy, full, full.abs() * (4 * 2.0 ** -24 + half_step(x.dtype)) + (2.0 ** -25 if x.dtype == t.float16 else 1e-38), "y")


@pytest.mark.parametrize("tokens,n,type,qa,residual,y,f16_scale", CASES)
def test_norm(tokens, n, type, qa, residual, y, f16_scale):
    g = gen(tokens + n)
    dt = DT[type]
    check(normal(g, tokens, n, dtype=dt), normal(g, tokens, n, dtype=dt, scale=2.0) if residual else None,
          normal(g, n, dtype=dt, scale=0.2, shift=1.0), qa, y, f16_scale)


@pytest.mark.parametrize("type", ["f32", "bf16"])
def test_norm_strided_rows(type):
    g = gen(5)
    dt = DT[type]
    check(normal(g, 9, 256, dtype=dt), normal(g, 9, 256, dtype=dt), normal(g, 256, dtype=dt), 64, True, False, pad=16)


@pytest.mark.parametrize("f16_scale", [False, True])
def test_norm_extremes(f16_scale):
    """Zero rows and blocks, values whose sum of squares overflows or
    underflows f32, scales in f16's subnormal range, zero weights."""
    t = torch()
    g = gen(9)
    x = normal(g, 8, 512)
    x[0] = 0
    x[1, 128:256] = 0
    x[2] *= 1e25   # squares above f32's range
    x[3] *= 1e-25  # squares below it: eps decides
    x[4] *= 1e-3
    x[4, 0] = 1e4  # the other blocks of the row get small values
    x[5] *= 1e-2
    w = normal(g, 512, scale=0.2, shift=1.0)
    w[256:384] = 0
    w[384:] *= 1e-3
    check(x, None, w, 32, True, f16_scale)
    check(x, t.zeros_like(x), w, 128, True, f16_scale)


def test_norm_least_eps():
    """Zero rows and rows of subnormal values at the smallest eps."""
    t, bq = torch(), bqmod()
    x = t.zeros(3, 128)
    x[1] = 1e-42
    x[2, 5] = -3e-39
    w = t.ones(128)
    q = t.empty(3, 128, dtype=t.int8, device="cuda")
    d = t.empty(3, 1, device="cuda")
    bq.bq_rmsnorm_q8(x.cuda(), w.cuda(), 1e-30, 128, q, d)
    _, _, rq, rd = norm_ref(x, None, w, 1e-30, 128, False)
    assert t.equal(q.cpu(), rq) and t.equal(d.cpu(), rd) and (rq[0] == 0).all()


def test_norm_in_place():
    """h in place of the residual and y in place of x."""
    t, bq = torch(), bqmod()
    g = gen(3)
    x, res = normal(g, 6, 384, dtype=t.bfloat16), normal(g, 6, 384, dtype=t.bfloat16)
    w = normal(g, 384, dtype=t.bfloat16, scale=0.1, shift=1.0)
    rh, rv, rq, rd = norm_ref(x, res, w, 1e-6, 128, False)
    xd, rd_ = x.cuda(), res.cuda()
    q = t.empty(6, 384, dtype=t.int8, device="cuda")
    d = t.empty(6, 3, device="cuda")
    bq.bq_rmsnorm_q8(xd, w.cuda(), 1e-6, 128, q, d, res=rd_, h=rd_, y=xd)
    assert t.equal(rd_.cpu(), rh) and t.equal(xd.cpu(), rv.to(x.dtype))
    assert t.equal(q.cpu(), rq) and t.equal(d.cpu(), rd)


def test_norm_feeds_the_products():
    """The rows are what a product takes: bq_q1_0_matvec on them equals the
    oracle on the oracle's quants."""
    import oracle
    import synth
    from pins import same_bits
    t, bq = torch(), bqmod()
    g = gen(4)
    x, w = normal(g, 3, 512), normal(g, 512, scale=0.1, shift=1.0)
    q = t.empty(3, 512, dtype=t.int8, device="cuda")
    d = t.empty(3, 4, device="cuda")
    bq.bq_rmsnorm_q8(x.cuda(), w.cuda(), 1e-6, 128, q, d)
    canon = synth.blocks(1, 100, 512, 1, 2)
    y = t.empty(300, device="cuda")
    bq.bq_q1_0_matvec(bq.Weights.upload(1, canon, 100, 512), bq.Act(q, d, 512, 128, 3), y)
    _, _, rq, rd = norm_ref(x, None, w, 1e-6, 128, False)
    ref = oracle.matvec(1, canon, 100, 512, rq.numpy(), rd.numpy(), 128, ncols=3, threads=4)
    assert same_bits(y.cpu().numpy().reshape(3, 100), ref)


def test_norm_refusals():
    t, bq = torch(), bqmod()
    x, w = t.ones(2, 256, device="cuda"), t.ones(256, device="cuda")
    q, d = t.empty(2, 256, dtype=t.int8, device="cuda"), t.empty(2, 2, device="cuda")

    def refused(text, *a, **k):
        with pytest.raises(bq.BQError) as e:
            bq.bq_rmsnorm_q8(*a, **k)
        assert e.value.code in (bq.BQ_EARG, bq.BQ_EALIGN) and text in str(e.value), str(e.value)

    refused("qa", x, w, 1e-6, 48, q, t.empty(2, 5, device="cuda"))
    refused("eps", x, w, 0.0, 128, q, d)
    refused("eps", x, w, float("nan"), 128, q, d)
    refused("w", x, w.half(), 1e-6, 128, q, d)
    refused("w", x, w[:128], 1e-6, 128, q, d)
    refused("res", x, w, 1e-6, 128, q, d, res=x.bfloat16())
    refused("q", x, w, 1e-6, 128, q[:1], d)
    refused("d", x, w, 1e-6, 128, q, d[:, :1])
    refused("x", x.cpu(), w, 1e-6, 128, q, d)
    refused("rows of x", x.t().contiguous().t(), w, 1e-6, 128, q, d)
    refused("float32, float16", x.double(), w, 1e-6, 128, q, d)
    refused("leading dimension", x, w, 1e-6, 128, q, d, h=t.empty(2, 512, device="cuda")[:, :256],
            res=t.empty(1, 256, device="cuda").expand(2, 256))
    odd = t.empty(2 * 256 + 1, device="cuda")[1:].view(2, 256)
    refused("16-byte", odd, w, 1e-6, 128, q, d)
    bq.bq_rmsnorm_q8(x[:0], w, 1e-6, 128, q[:0], d[:0])  # no rows: nothing to do
