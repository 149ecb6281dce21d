"""The operators around the layers as they run together (staging.StagedDecoder,
StagedMLP): prompts of several requests, then steps of one token each that feed
on the tokens drawn before; every stage against its reference on the stage's own
inputs.  Captured into a graph and replayed, and on another stream: the same
tokens."""
import numpy as np
import pytest

import oracle
import synth
from gpu_util import bqmod, torch
from layer_util import gen, norm_ref, normal, within
from model_util import Ranked, codes, gated_ref, matmul_ref, quants_ref

pytestmark = pytest.mark.gpu

HIDDEN, HQ, H, D, PAGE, INNER, VOCAB, QA = 512, 8, 2, 64, 16, 768, 1500, 128
PAGES, COLS, LAYERS = 40, 12, 2


class Model:
    def __init__(self, fmt, max_tokens, matmul_from=17, act=1):
        t, bq = torch(), bqmod()
        from ternary_quantized_gemv_amd.staging import StagedAttention, StagedDecoder, StagedMLP
        self.fmt, self.act = fmt, act
        freq = (1e4 ** (-t.arange(0, D, 2).double() / D)).float().cuda()
        self.canon_head = synth.blocks(fmt, VOCAB, HIDDEN, 77)
        self.norms, self.canon_mlp, layers = [], [], []
        for i in range(LAYERS):
            g = gen(20 + i)
            canon = {n: synth.blocks(fmt, r, c, 5, i, j) for j, (n, r, c) in enumerate(
                (("q", HQ * D, HIDDEN), ("k", H * D, HIDDEN), ("v", H * D, HIDDEN), ("o", HIDDEN, HQ * D)))}
            mlp = {n: synth.blocks(fmt, r, c, 6, i, j) for j, (n, r, c) in enumerate(
                (("gate", INNER, HIDDEN), ("up", INNER, HIDDEN), ("down", HIDDEN, INNER)))}
            norms = [normal(g, HIDDEN, scale=0.1, shift=1.0) for _ in range(2)]
            self.norms.append(norms)
            self.canon_mlp.append(mlp)
            cache = bq.KVCache.empty(PAGES, H, D, PAGE)
            layers.append((StagedAttention(fmt, canon, HIDDEN, HQ, cache, norms[0].cuda(), freq, max_tokens, matmul_from=matmul_from),
                           StagedMLP(fmt, mlp, HIDDEN, INNER, norms[1].cuda(), max_tokens, act=act, matmul_from=matmul_from)))
        self.norm = normal(gen(9), HIDDEN, scale=0.1, shift=1.0)
        self.head = bq.Weights.upload(fmt, self.canon_head, VOCAB, HIDDEN)
        self.d = StagedDecoder(self.head, layers, self.norm.cuda(), self.head, max_tokens, 3, scale=HIDDEN ** 0.5, matmul_from=matmul_from)
        self.table = t.randperm(PAGES, generator=gen(3))[:3 * COLS].view(3, COLS).to(t.int32)

    def step(self, lens, new, ids, seed):
        t = torch()
        place = lambda b, p: self.table[b].long()[p // PAGE] * PAGE + p % PAGE  # noqa: E731
        pos = [t.arange(n - k, n) for n, k in zip(lens, new)]
        cu = t.tensor([0] + list(new)).cumsum(0)
        g = gen(seed)
        return dict(ids=ids.cuda(), last=(cu[1:] - 1).cuda(), u=t.rand(3, generator=g).cuda(), pos=t.cat(pos).to(t.int32).cuda(),
                    slot=t.cat([place(b, p) for b, p in enumerate(pos)]).cuda(), cu=cu.to(t.int32).cuda(),
                    lens=t.tensor(lens, dtype=t.int32).cuda(), table=self.table.cuda(),
                    temperature=t.tensor([0.8, 0.0, 1.3]).cuda(), top_k=t.tensor([40, 0, 0], dtype=t.int32).cuda(),
                    top_p=t.tensor([0.9, 1.0, 0.95]).cuda())

    def product(self, canon, q, d, wide, res=None):
        """(y, bound): exact bits, or matmul's bound where the product is one bq_matmul."""
        t = torch()
        rows, cols = canon.shape[0], canon.shape[1] * bqmod().BLOCK_LEN[self.fmt]
        if wide:
            return matmul_ref(self.fmt, canon, q.numpy(), d.numpy(), QA, t.float32, res=res)
        y = t.from_numpy(np.asarray(oracle.matvec(self.fmt, canon, rows, cols, q.numpy(), d.numpy(), QA, ncols=q.shape[0], threads=8)))
        return y.double().view(q.shape[0], rows), 0.0

    def check(self, s, token, logprob):
        """All buffers of the decoder's own stages after a step."""
        t = torch()
        T, B = len(s["ids"]), 3
        w, d0 = codes(self.fmt, self.canon_head)
        rows = (w * d0[..., None]).reshape(VOCAB, HIDDEN).astype(np.float32)
        ids = s["ids"].cpu().numpy()
        assert np.array_equal(self.d.x[:T].cpu().numpy(), rows[ids] * np.float32(HIDDEN ** 0.5))
        for i, (attention, mlp) in enumerate(self.d.layers):
            get = lambda name, n=T: getattr(mlp, name)[:n].cpu()  # noqa: E731
            wide = mlp.products.wide(T)
            x, res = attention.out[:T].cpu(), attention.h[:T].cpu()
            h, _, q, d = norm_ref(x, res, self.norms[i][1], 1e-6, QA, False)
            assert t.equal(get("h"), h) and t.equal(get("act"), q) and t.equal(get("act_d"), d)
            for name in ("gate", "up"):
                within(get(name), *self.product(self.canon_mlp[i][name], q, d, wide), (i, name))
            v, other, wq, wd = gated_ref(get("gate"), get("up"), ("none", "silu", "gelu", "relu2")[self.act], QA, False)
            assert (get("inner_act").numpy() != wq).mean() < 1e-4 and np.allclose(get("inner_d").numpy(), wd, rtol=2e-7)
            within(get("out"), *self.product(self.canon_mlp[i]["down"], get("inner_act"), get("inner_d"), wide, h if wide else None), (i, "down"))
        last = s["last"].cpu()
        x = get("out")[last]
        res = None if wide else get("h")[last]
        _, _, q, d = norm_ref(x, res, self.norm, 1e-6, QA, False)
        assert t.equal(self.d.act[:B].cpu(), q) and t.equal(self.d.act_d[:B].cpu(), d)
        logits = self.d.logits[:B].cpu()
        within(logits, *self.product(self.canon_head, q, d, self.d.products.wide(B)), "logits")
        for b in range(B):
            r = Ranked(logits[b].double().numpy(), float(s["temperature"][b]))
            kept = r.kept(int(s["top_k"][b]), float(s["top_p"][b]))
            passed = r.sums[:kept] > float(s["u"][b]) * r.sums[kept - 1]
            rank = 0 if r.greedy else int(np.argmax(passed))
            near = np.min(np.abs(r.sums[:kept] - float(s["u"][b]) * r.sums[kept - 1])) < 1e-9 * r.sums[-1]
            assert near or int(token[b]) == r.order[rank], (b, int(token[b]), r.order[rank])
            assert near or abs(float(logprob[b]) - r.logprob(rank)) <= 2.0 ** -23 * (1 + abs(r.logprob(rank)))


@pytest.mark.parametrize("fmt,act", [(1, 1), (2, 3)])
@pytest.mark.parametrize("matmul_from", [17, None])
def test_prompts_then_steps(fmt, act, matmul_from):
    t = torch()
    m = Model(fmt, 90, matmul_from, act)
    lens = [37, 5, 20]
    ids = t.randint(0, VOCAB, (sum(lens),), generator=gen(1))
    s = m.step(lens, lens, ids, 1)
    token, logprob = m.d.run(**s, max_new=37, max_keys=37)
    m.check(s, token.cpu(), logprob.cpu())
    for i in range(3):
        lens = [n + 1 for n in lens]
        s = m.step(lens, [1, 1, 1], token.cpu(), 10 + i)
        token, logprob = m.d.run(**s, max_new=1, max_keys=64)
        m.check(s, token.cpu(), logprob.cpu())


@pytest.mark.parametrize("fmt", [1, 2])
def test_captured_steps(fmt):
    """One step captured with fixed tensors; each replay continues from the tokens of the one before, as eager runs do."""
    t, bq = torch(), bqmod()
    runs = []
    for captured in (False, True):
        m = Model(fmt, 90)
        lens = [37, 5, 20]
        ids = t.randint(0, VOCAB, (sum(lens),), generator=gen(1))
        stream = t.cuda.Stream()
        t.cuda.synchronize()
        first = m.step(lens, lens, ids, 1)
        t.cuda.synchronize()
        token, _ = m.d.run(**first, max_new=37, max_keys=37, stream=None if captured else stream)
        t.cuda.synchronize()
        work = t.empty(bq.bq_paged_attn_work_bytes(m.d.layers[0][0].cache, 3, HQ, 3, 1, 64), dtype=t.uint8, device="cuda")
        fixed, graph, seen = None, t.cuda.CUDAGraph(), [token.tolist()]
        for i in range(4):
            lens = [n + 1 for n in lens]
            s = m.step(lens, [1, 1, 1], token.clone(), 10 + i)  # (the buffer itself is written again below)
            if not captured:
                token, logprob = m.d.run(**s, max_new=1, max_keys=64, work=work)
            else:
                if fixed is None:
                    fixed = {k: v.clone() for k, v in s.items()}
                    m.d.run(**fixed, max_new=1, max_keys=64, work=work)  # loads the kernels
                    t.cuda.synchronize()
                    with t.cuda.graph(graph):
                        token, logprob = m.d.run(**fixed, max_new=1, max_keys=64, work=work)
                for k, v in s.items():
                    fixed[k].copy_(v)
                graph.replay()
            t.cuda.synchronize()
            seen.append(token.tolist() + [round(float(x), 5) for x in logprob])
        runs.append(seen)
    assert runs[0] == runs[1]


@pytest.mark.parametrize("fmt", [1, 2])
def test_wide_products_near_the_narrow_ones(fmt):
    """A prompt with its products in one call each, and 16 tokens at a time: the first layer's hidden rows agree to f32
    sums through its quantizers (a quant next to a border may move by one step)."""
    t = torch()
    lens = [37, 5, 20]
    ids = t.randint(0, VOCAB, (sum(lens),), generator=gen(1))
    outs = []
    for matmul_from in (17, None):
        m = Model(fmt, 90, matmul_from)
        s = m.step(lens, lens, ids, 1)
        m.d.run(**s, max_new=37, max_keys=37)
        outs.append(m.d.layers[0][0].out[:62].double().cpu())
    a, b = outs
    assert ((a - b).norm() / b.norm()) < 0.02
