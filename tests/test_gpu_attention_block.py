"""The operators between the products as they run together
(staging.StagedAttention): prompts of several requests, then decode steps over
the same cache, two blocks deep; every stage against its reference on the
stage's own inputs, products and quantizers bit for bit.  The same steps
captured into a graph and replayed, on another stream, and on two streams at
once give the same bits."""
import numpy as np
import pytest

import oracle
import synth
from gpu_util import bqmod, torch
from layer_util import adapters_ref, attn_ref, gen, half_step, norm_ref, normal, rotate_ref, within
from pins import same_bits

pytestmark = pytest.mark.gpu

HIDDEN, HQ, H, D, PAGE = 512, 8, 2, 64, 16
PAGES, COLS = 40, 12
ROWS = {"q": HQ * D, "k": H * D, "v": H * D, "o": HIDDEN}


class Model:
    """Two attention blocks, each with its cache, and the tables of three requests."""

    def __init__(self, fmt, max_tokens, with_adapters=True):
        t, bq = torch(), bqmod()
        from ternary_quantized_gemv_amd.staging import StagedAttention
        self.fmt, self.host, self.blocks, self.caches = fmt, [], [], []
        freq = (1e4 ** (-t.arange(0, D, 2).double() / D)).float()
        for i in range(2):
            g = gen(10 + i)
            cols = {"q": HIDDEN, "k": HIDDEN, "v": HIDDEN, "o": HQ * D}
            canon = {n: synth.blocks(fmt, ROWS[n], cols[n], 5, i, j) for j, n in enumerate("qkvo")}
            host = {"canon": canon, "cols": cols, "freq": freq, "norm": normal(g, HIDDEN, scale=0.1, shift=1.0),
                    "q_norm": normal(g, D, scale=0.1, shift=1.0), "k_norm": normal(g, D, scale=0.1, shift=1.0)}
            host["adapters"] = {n: (normal(g, 2, 16, cols[n], dtype=t.bfloat16, scale=cols[n] ** -0.5),
                                    normal(g, 2, ROWS[n], 16, dtype=t.bfloat16, scale=0.25),
                                    normal(g, 2, scale=0.1, shift=1.0)) for n in ("q", "v", "o")} if with_adapters else {}
            cache = bq.KVCache(t.full((PAGES, H, PAGE, D), float("nan"), dtype=t.bfloat16, device="cuda"),
                               t.full((PAGES, H, D, PAGE), float("nan"), dtype=t.bfloat16, device="cuda"))
            self.caches.append(cache)
            self.host.append(host)
            self.blocks.append(StagedAttention(
                fmt, canon, HIDDEN, HQ, cache, host["norm"].cuda(), freq.cuda(), max_tokens, q_norm=host["q_norm"].cuda(),
                k_norm=host["k_norm"].cuda(),
                adapters={n: bq.Adapters(*(p.cuda() for p in a)) for n, a in host["adapters"].items()}))
        order = t.randperm(PAGES, generator=gen(3))[:3 * COLS].view(3, COLS)
        self.table = order.to(t.int32)
        self.ids = t.tensor([1, -1, 0], dtype=t.int32)

    def step(self, lens, new, seed):
        """Inputs of a step that brings each request from lens - new to lens keys."""
        t = torch()
        pos = t.cat([t.arange(n - k, n) for n, k in zip(lens, new)])
        slot = t.cat([self.table[b].long()[p // PAGE] * PAGE + p % PAGE
                      for b, p in enumerate(t.arange(n - k, n) for n, k in zip(lens, new))])
        return {"x": normal(gen(seed), sum(new), HIDDEN).cuda(), "pos": pos.to(t.int32).cuda(), "slot": slot.cuda(),
                "cu": t.tensor([0] + list(new)).cumsum(0).to(t.int32).cuda(), "lens": t.tensor(lens, dtype=t.int32).cuda(),
                "table": self.table.cuda(), "ids": self.ids.cuda()}

    def run(self, s, max_new, max_keys, stream=None, work=None, adapter_work=None):
        x, res = s["x"], None
        for b in self.blocks:
            x, res = b.run(x, res, s["pos"], s["slot"], s["cu"], s["lens"], s["table"], max_new, max_keys, ids=s["ids"],
                           work=work, adapter_work=adapter_work, stream=stream)
        return x, res


def check_block(m, i, s, x, res, lens, new):
    """Block i's buffers after a step, stage by stage."""
    t = torch()
    b, host = m.blocks[i], m.host[i]
    T = x.shape[0]
    cu = [0] + list(np.cumsum(new))
    got = {n: getattr(b, n)[:T].cpu() for n in ("h", "act", "act_d", "q", "k", "v", "o", "o_act", "o_d", "out")}
    h, v, q8, d = norm_ref(x, res, host["norm"], 1e-6, 128, False)
    assert t.equal(got["h"], h) and t.equal(got["act"], q8) and t.equal(got["act_d"], d)

    def product(name, q8, d, x):
        """(y, bound) behind the adapters."""
        canon = host["canon"][name]
        y = t.from_numpy(oracle.matvec(m.fmt, canon, ROWS[name], host["cols"][name], q8.numpy(), d.numpy(), 128, ncols=T, threads=8))
        out, bound = y.double(), t.zeros(T, ROWS[name], dtype=t.float64)
        if name in host["adapters"]:
            a, bb, gain = host["adapters"][name]
            for r, ad in enumerate(m.ids.tolist()):
                if ad >= 0:
                    rows = slice(cu[r], cu[r + 1])
                    out[rows], bound[rows] = adapters_ref(x[rows], a[ad], bb[ad], gain[ad], y[rows])
        return out, bound

    pos = s["pos"].cpu()
    # q after norm and rotation; k and v in the cache.  What went into the norm is known within its bound, which
    # the norm scales up to the size of a row: a few times the bound over the row's rms, added per row.
    for name, heads in (("q", HQ), ("k", H), ("v", H)):
        y, bound = product(name, q8, d, v)
        y, bound = y.unflatten(1, (heads, D)), bound.unflatten(1, (heads, D))
        if name == "v":
            want, tol = y, bound
        else:
            want, tol = rotate_ref(y, pos, host["freq"], host[name + "_norm"], 1e-6)
            rms = y.square().mean(-1, keepdim=True).sqrt()
            tol = tol + 8 * bound.amax(-1, keepdim=True) / rms
        if name == "q":
            within(got["q"].unflatten(1, (heads, D)), want, tol + 1e-30, f"block {i} q")
        else:
            plane = m.caches[i].k if name == "k" else m.caches[i].v
            slot = s["slot"]
            held = plane[slot // PAGE, :, slot % PAGE] if name == "k" else plane[slot // PAGE, :, :, slot % PAGE]
            within(held, want, tol + want.abs() * half_step(t.bfloat16) + 1e-30, f"block {i} {name}")
    # attention over what the cache holds
    for r, (n, k) in enumerate(zip(lens, new)):
        p = t.arange(n)
        at, off = m.table[r].long()[p // PAGE].cuda(), (p % PAGE).cuda()
        kk, vv = m.caches[i].k[at, :, off].cpu(), m.caches[i].v[at, :, :, off].cpu()
        rows = slice(cu[r], cu[r + 1])
        want, tol = attn_ref(got["q"][rows].unflatten(1, (HQ, D)), kk, vv, n, D ** -0.5, t.float32)
        within(got["o"][rows].unflatten(1, (HQ, D)), want, tol, f"block {i} request {r}")
    rq, rd, _ = oracle.quantize_q8(got["o"].numpy().ravel(), 128)
    assert np.array_equal(got["o_act"].numpy().ravel(), rq) and same_bits(got["o_d"].numpy().ravel(), rd)
    out, bound = product("o", got["o_act"], got["o_d"], got["o"])
    within(got["out"], out, bound + 1e-30, f"block {i} out")
    return got["out"], got["h"]


STEPS = [([37, 5, 20], [37, 5, 20]), ([38, 6, 21], [1, 1, 1]), ([70, 7, 22], [32, 1, 1]), ([71, 7, 40], [1, 0, 18])]


@pytest.mark.parametrize("fmt", [1, 2])
def test_prompts_then_tokens(fmt):
    m = Model(fmt, 64)
    for i, (lens, new) in enumerate(STEPS):
        s = m.step(lens, new, 100 + i)
        m.run(s, max(new), max(lens))
        torch().cuda.synchronize()
        x, res = s["x"].cpu(), None
        for b in range(2):
            x, res = check_block(m, b, s, x, res, lens, new)


def test_one_graph_for_many_tokens():
    """A decode step captured once and replayed as the requests grow, with
    eager work between the replays, gives the eager run's bits."""
    t = torch()
    eager, graphed = Model(1, 64), Model(1, 64)
    first = eager.step([37, 5, 20], [37, 5, 20], 200)
    for m in (eager, graphed):
        m.run(first, 37, 37)
    s = graphed.step([38, 6, 21], [1, 1, 1], 201)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        graphed.run(s, 1, COLS * PAGE)
    t.cuda.current_stream().wait_stream(side)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        out, h = graphed.run(s, 1, COLS * PAGE)
    noise = t.ones(1 << 20, device="cuda")
    for k in range(6):
        lens = [38 + k, 6 + k, 21 + k]
        now = eager.step(lens, [1, 1, 1], 300 + k)
        want, want_h = eager.run(now, 1, COLS * PAGE)
        want, want_h = want.clone(), want_h.clone()
        for n, v in now.items():
            s[n].copy_(v)
        noise.mul_(1.0001)
        graph.replay()
        noise.sum().item()  # eager work and a synchronization between replays
        assert t.equal(out, want) and t.equal(h, want_h), k
    for a, b in zip(eager.caches, graphed.caches):
        assert t.equal(a.k.view(t.int16), b.k.view(t.int16)) and t.equal(a.v.view(t.int16), b.v.view(t.int16))


def test_streams():
    """The same step on the default stream, on another one by argument, as a
    raw handle, and two models at once on two streams."""
    t = torch()
    lens, new = [37, 5, 20], [37, 5, 20]
    models = [Model(2, 64) for _ in range(4)]
    s = models[0].step(lens, new, 400)
    want = models[0].run(s, 37, 37)[0].clone()
    t.cuda.synchronize()
    one, two = t.cuda.Stream(), t.cuda.Stream()
    outs = [models[1].run(s, 37, 37, stream=one)[0], models[2].run(s, 37, 37, stream=two.cuda_stream)[0]]
    with t.cuda.stream(one):
        outs.append(models[3].run(s, 37, 37)[0])
    t.cuda.synchronize()
    for o in outs:
        assert t.equal(o, want)


def test_nothing_is_allocated_with_scratch_given():
    t, bq = torch(), bqmod()
    m = Model(1, 64)
    s = m.step([37, 5, 20], [37, 5, 20], 500)
    need = bq.bq_paged_attn_work_bytes(m.caches[0], 62, HQ, 3, 37, 37)
    need_a = max(bq.bq_adapters_work_bytes(a, 62, 3, 37) for b in m.blocks for a in b.adapters.values())
    work = t.empty(max(need, 16), dtype=t.uint8, device="cuda")
    adapter_work = t.empty(need_a, dtype=t.uint8, device="cuda")
    m.run(s, 37, 37, work=work, adapter_work=adapter_work)
    t.cuda.synchronize()
    before = t.cuda.memory_stats()["allocation.all.allocated"]
    m.run(s, 37, 37, work=work, adapter_work=adapter_work)
    assert t.cuda.memory_stats()["allocation.all.allocated"] == before
    t.cuda.synchronize()
