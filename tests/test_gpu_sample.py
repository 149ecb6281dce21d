"""bq_sample against the definition in 64 bits.  The random numbers are placed in
the middle of a token's share, and the filters' limits between two places of the
order, so that the token follows from the definition alone and has to be it."""
import numpy as np
import pytest

from gpu_util import bqmod, torch
from layer_util import DT
from model_util import Ranked

pytestmark = pytest.mark.gpu


def run(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, **k):
    t, bq = torch(), bqmod()
    B = logits.shape[0]
    f = lambda x, dt=t.float32: None if x is None else t.as_tensor(np.asarray(x), device="cuda").to(dt)  # noqa: E731
    token, logprob = t.full((B,), -7, dtype=t.int64, device="cuda"), t.full((B,), 7.0, device="cuda")
    bq.bq_sample(logits, f(u), token, logprob=logprob, temperature=f(temperature), top_k=f(top_k, t.int32), top_p=f(top_p),
                 min_p=f(min_p), **k)
    t.cuda.synchronize()
    return token.cpu().numpy(), logprob.cpu().numpy()


def row_of(kind, vocab, g):
    if kind == "flat":
        return np.zeros(vocab)
    if kind == "two":
        return np.where(g.random(vocab) < 0.5, 1.0, 1.25)
    if kind == "wide":
        return g.standard_normal(vocab) * 30
    if kind == "peaked":
        x = g.standard_normal(vocab) * 2
        x[g.integers(0, vocab, 20)] += 9
        return x
    x = g.standard_normal(vocab) * 1.5
    if kind == "masked":
        x[g.random(vocab) < 0.7] = -np.inf
        x[g.integers(0, vocab)] = 0.5
    return x


def limits(r, g):
    """(k, p, min_p, kept) with the limits between two places of the order."""
    n = int((r.w > 2.0 ** -30).sum())
    k = int(g.integers(1, n + 3)) if g.random() < 0.6 else 0
    p, least = 1.0, 0.0
    if g.random() < 0.6:
        m = r.kept(k)
        j = int(g.integers(0, min(m, n)))
        p = float(np.float32((r.sums[j] - 0.5 * r.w[j]) / r.sums[m - 1]))
    if g.random() < 0.4:
        j = int(g.integers(0, n))
        least = float(np.float32(r.w[j] * 0.999))
        if np.any(np.abs(r.w / least - 1) < 1e-4):
            least = 0.0
    if p < 1:  # not where 32 bits of p could fall on the other side
        m = r.kept(k)
        if np.min(np.abs(r.sums[:m] - p * r.sums[m - 1])) < 1e-6 * r.sums[m - 1]:
            p = 1.0
    return k, p, least, r.kept(k, p, least)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["normal", "peaked", "flat", "two", "wide", "masked"])
@pytest.mark.parametrize("vocab", [1, 2, 63, 1000, 4097, 33001, 151936])
def test_draws(dt, kind, vocab):
    t = torch()
    g = np.random.default_rng(vocab + len(kind))
    B = 3 if vocab > 100000 else 12
    rows = t.from_numpy(np.stack([row_of(kind, vocab, g) for _ in range(B)])).to(DT[dt])
    temp = np.where(np.arange(B) % 4 == 3, 0.3, np.where(np.arange(B) % 4 == 2, 2.5, 1.0)).astype(np.float32)
    ranked = [Ranked(rows[b].double().numpy(), float(temp[b])) for b in range(B)]
    for trial in range(3):
        sets = [limits(r, g) if trial else (0, 1.0, 0.0, r.kept()) for r in ranked]
        u, want = [], []
        for r, (_, _, _, kept) in zip(ranked, sets):
            share = r.w[:kept] / r.sums[kept - 1]
            able = np.flatnonzero(share > 2.0 ** -21)  # wider than the steps of u
            rank = int(able[[0, len(able) // 2, -1][trial]]) if trial < 2 else int(able[-1])
            u.append(r.inside(rank, kept))
            want.append(rank)
        k, p, least = ([s[i] for s in sets] for i in range(3))
        token, logprob = run(rows.cuda(), u, temp, k if trial else None, p if trial else None, least if trial else None)
        for b, (r, rank) in enumerate(zip(ranked, want)):
            assert token[b] == r.order[rank], (b, sets[b], rank, token[b], r.order[rank])
            # the weight of the row's whole sum is rounded at most by vocab times 2^-40, the logarithm once
            assert abs(logprob[b] - r.logprob(rank)) <= 2.0 ** -23 * (1 + abs(r.logprob(rank))), (b, logprob[b], r.logprob(rank))


@pytest.mark.parametrize("vocab", [5, 2000, 151936])
def test_ends_of_u_and_of_the_filters(vocab):
    t = torch()
    g = np.random.default_rng(vocab)
    x = g.standard_normal(vocab).astype(np.float32)
    rows = t.from_numpy(np.tile(x, (9, 1))).cuda()
    r = Ranked(x)
    best = r.order[0]
    top = float(np.float32(1 - 2.0 ** -24))
    token, logprob = run(rows, [0, -1, float("nan"), top, 1.0, 2.0, top, top, top], top_k=[0, 0, 0, 1, 1, 1, 3, -5, vocab + 9],
                         top_p=[1, 1, 1, 1, 2, float("nan"), 1, 0, 0.0], min_p=[0] * 7 + [0, -1])
    assert (token[:6] == best).all() and token[6] == r.order[2] and token[7] == best and token[8] == best
    # min_p of 1 and more: the largest alone; nothing else left
    token, _ = run(rows[:3], [top] * 3, min_p=[1.0, 3.0, float("nan")])
    assert (token[:2] == best).all()
    assert token[2] in r.order[-2000:]
    # no filter: the last of the order with a weight
    token, _ = run(rows[:2], [1.0, float("inf")])
    assert (token == r.order[-1]).all()


def test_greedy_and_temperatures():
    t = torch()
    x = t.zeros(6, 5000)
    x[:, 4000] = x[:, 1234] = x[:, 3000] = 2.0
    x[3, 17], x[3, 18] = float("inf"), float("inf")
    token, logprob = run(x.cuda(), [0.99] * 6, temperature=[0.0, -1.0, float("nan"), 0.0, 1e-30, 1e-38], top_k=[5] * 6, top_p=[0.5] * 6)
    assert token.tolist()[:4] == [1234, 1234, 1234, 17] and (logprob[:4] == 0).all()
    small, lp = token, logprob
    # rows long enough to be read several loads at a time, the largest anywhere
    g = np.random.default_rng(1)
    long = t.from_numpy(g.standard_normal((40, 70001)).astype(np.float32))
    token, _ = run(long.cuda(), [0.7] * 40, temperature=[[0.0, -2.0, float("nan"), -0.0][i % 4] for i in range(40)])
    assert token.tolist() == long.argmax(1).tolist()
    # a tiny temperature leaves the largest, each a third
    assert all(v in (1234, 3000) for v in small[4:]) and np.allclose(lp[4:], np.log(1 / 3), rtol=1e-6)
    # an infinite one all alike
    token, logprob = run(x[:1].cuda(), [0.5], temperature=[float("inf")])
    order = Ranked(x[0].numpy()).order
    assert token[0] == order[2500] and np.allclose(logprob, -np.log(5000), rtol=1e-6)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_without_weight_and_non_finite(dt):
    t = torch()
    nan, inf = float("nan"), float("inf")
    x = t.full((6, 777), -inf, dtype=DT[dt])
    x[1] = nan
    x[2, 5], x[2, 6] = nan, 1.0
    x[3, 9], x[3, 700] = inf, inf
    x[3, 3] = 4.0
    x[4] = -1e4
    x[4, 100:200] = nan
    x[5, 776] = -1e38
    token, logprob = run(x.cuda(), [0.4, 0.4, 0.999, 0.75, 0.999, 0.0])
    assert token.tolist()[:4] == [-1, -1, 6, 700] and token[4] == 776 and token[5] == 776
    assert logprob[0] == -inf and logprob[1] == -inf and logprob[2] == 0 and np.isclose(logprob[3], np.log(0.5))
    assert np.isclose(logprob[4], -np.log(677), rtol=1e-6) and logprob[5] == 0


def test_differences_past_the_range_of_f32():
    """Logits at both ends of f32 under a temperature that brings them near each other."""
    t = torch()
    x = t.full((4, 900), -3e38)
    x[:, 5], x[:, 700] = 3e38, 0.0
    temp = np.float32(1e38)
    w = np.exp(np.array([0.0, -3.0, -6.0]))  # of 5, 700 and the others
    total = w[0] + w[1] + 898 * w[2]
    at = [w[0] / 2, w[0] + w[1] / 2, w[0] + w[1] + 0.5 * w[2], w[0] + w[1] + 897.5 * w[2]]
    token, logprob = run(x.cuda(), np.array(at) / total, temperature=[temp] * 4, top_p=[1.0, 1.0, 0.999, 1.0])
    assert token.tolist()[:2] == [5, 700] and token[2] == 0 and token[3] == 899
    want = np.log(np.array([w[0], w[1], w[2], w[2]]) / total)
    assert np.allclose(logprob, want, rtol=0, atol=6 * 2.0 ** -22)  # T and the logits are f32: 6 nats off by two roundings


def test_signed_zeros_are_one_value():
    t = torch()
    x = t.zeros(1, 4000)
    x[0, ::2] = -0.0
    token, _ = run(x.cuda(), [(1000 + 0.5) / 4000])
    assert token[0] == 1000


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("vocab,pad", [(1001, 0), (999, 2), (32000, 7)])
def test_strides_and_offsets(dt, vocab, pad):
    """Rows at any element; what lies between them is not read."""
    t = torch()
    g = np.random.default_rng(vocab)
    store = t.full((7 * (vocab + pad) + 3,), float("inf"), dtype=DT[dt])
    rows = store[1:1 + 7 * (vocab + pad)].view(7, vocab + pad)[:, :vocab]
    rows.copy_(t.from_numpy(g.standard_normal((7, vocab))))
    ranked = [Ranked(rows[b].double().numpy()) for b in range(7)]
    whole = store.cuda()
    view = whole[1:1 + 7 * (vocab + pad)].view(7, vocab + pad)[:, :vocab]
    token, _ = run(view, [r.inside(j, vocab) for j, r in enumerate(ranked)])
    assert token.tolist() == [int(r.order[j]) for j, r in enumerate(ranked)]


@pytest.mark.parametrize("B", [1, 2, 40, 300])
def test_many_rows_agree_with_one_at_a_time(B):
    """However many rows a call has, a row's token is the same; a graph replayed on other values too."""
    t, bq = torch(), bqmod()
    g = t.Generator().manual_seed(B)
    x = (t.randn(B, 20011, generator=g) * 2).cuda()
    u, temp = t.rand(B, generator=g).cuda(), (0.5 + t.rand(B, generator=g)).cuda()
    k, p = t.randint(0, 200, (B,), generator=g).int().cuda(), (0.5 + 0.6 * t.rand(B, generator=g)).cuda()
    least = (0.05 * t.rand(B, generator=g)).cuda()
    token, logprob = t.empty(B, dtype=t.int64, device="cuda"), t.empty(B, device="cuda")
    one, lone = t.empty(1, dtype=t.int64, device="cuda"), t.empty(1, device="cuda")
    work = t.empty(bq.bq_sample_work_bytes(B, 20011), dtype=t.uint8, device="cuda")
    t.cuda.synchronize()

    def call(stream=None):
        bq.bq_sample(x, u, token, logprob=logprob, temperature=temp, top_k=k, top_p=p, min_p=least, work=work, stream=stream)

    def check():
        for b in {0, B // 2, B - 1}:
            s = slice(b, b + 1)
            bq.bq_sample(x[s], u[s], one, logprob=lone, temperature=temp[s], top_k=k[s], top_p=p[s], min_p=least[s])
            assert one[0] == token[b] and lone[0] == logprob[b]

    stream = t.cuda.Stream()
    call(stream)
    stream.synchronize()
    check()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        call()
    for i in range(4):
        x.copy_(t.roll(x, 1, 0) * 1.01)
        u.copy_(t.rand(B, device="cuda"))
        token.fill_(-3)
        graph.replay()
        t.cuda.synchronize()
        check()


def test_shares_over_many_draws():
    """Each token comes up as often as its share says: u on an even grid of 4096 over one row."""
    t = torch()
    x = np.array([1.0, 3.0, 2.0, -1.0, 3.0, 0.0], np.float32)
    B = 4096
    token, _ = run(t.from_numpy(np.tile(x, (B, 1))).cuda(), (np.arange(B) + 0.5) / B)
    share = np.exp(x.astype(np.float64)) / np.exp(x.astype(np.float64)).sum()
    assert (np.abs(np.bincount(token, minlength=6) - B * share) <= 1.0).all()
    assert (np.diff(x[token]) <= 0).all()  # in the order of the logits


def test_refusals():
    t, bq = torch(), bqmod()
    x, u, tok = t.zeros(4, 100, device="cuda"), t.zeros(4, device="cuda"), t.zeros(4, dtype=t.int64, device="cuda")
    for args, k in (((x.double(), u, tok), {}), ((x, u[:3], tok), {}), ((x, u, tok.int()), {}), ((x, u.half(), tok), {}),
                    ((x, None, tok), {}), ((x, u, None), {}), ((x.cpu(), u, tok), {}), ((x.t(), u, tok), {}),
                    ((x, u, tok), {"temperature": u.double()}), ((x, u, tok), {"top_k": u}), ((x, u, tok), {"top_p": u.cpu()}),
                    ((x, u, tok), {"min_p": u[:2]}), ((x, u, tok), {"logprob": u.half()})):
        with pytest.raises(bq.BQError):
            bq.bq_sample(*args, **k)
