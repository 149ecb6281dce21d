"""The attention block with each of its products as one bq_matmul, stage by stage
against its reference on the stage's own inputs; and a decoder whose steps take
the drawn tokens where they lie, eagerly and captured."""
import numpy as np
import pytest

import oracle
from gpu_util import bqmod, torch
from layer_util import attn_ref, gen, half_step, norm_ref, rotate_ref, within
from model_util import matmul_ref
from pins import same_bits
from test_gpu_attention_block import D, H, HIDDEN, HQ, PAGE, ROWS, STEPS
from test_gpu_attention_block import Model as Blocks
from test_gpu_decoder import VOCAB
from test_gpu_decoder import Model as Decoder

pytestmark = pytest.mark.gpu


def check(m, i, s, x, res, lens, new):
    """Block i's buffers after a step."""
    t = torch()
    b, host = m.blocks[i], m.host[i]
    T = x.shape[0]
    cu = [0] + list(np.cumsum(new))
    got = {n: getattr(b, n)[:T].cpu() for n in ("h", "act", "act_d", "q", "k", "v", "o", "o_act", "o_d", "out")}
    h, _, q8, d = norm_ref(x, res, host["norm"], 1e-6, 128, False)
    assert t.equal(got["h"], h) and t.equal(got["act"], q8) and t.equal(got["act_d"], d)
    pos, slot = s["pos"].cpu(), s["slot"]
    for name, heads in (("q", HQ), ("k", H), ("v", H)):
        y = t.full((T, ROWS[name]), float("nan"), device="cuda")  # q's own buffer holds the rotated rows by now
        b._product(name, b.act, b.act_d, y, T, None)
        y = y.cpu()
        within(y, *matmul_ref(m.fmt, host["canon"][name], q8.numpy(), d.numpy(), 128, t.float32), f"block {i} {name}")
        if name != "q":
            assert t.equal(got[name], y), name
        y = y.unflatten(1, (heads, D))
        if name == "v":
            want, tol = y.double(), t.zeros(1, dtype=t.float64)
        else:
            want, tol = rotate_ref(y, pos, host["freq"], host[name + "_norm"], 1e-6)
        if name == "q":
            within(got["q"].unflatten(1, (heads, D)), want, tol + 1e-30, f"block {i} rotated q")
        else:
            plane = m.caches[i].k if name == "k" else m.caches[i].v
            held = plane[slot // PAGE, :, slot % PAGE] if name == "k" else plane[slot // PAGE, :, :, slot % PAGE]
            within(held, want, tol + (want.abs() + tol) * half_step(t.bfloat16) + 1e-30, f"block {i} {name} in the cache")
    for r, n in enumerate(lens):
        p = t.arange(n)
        at, off = m.table[r].long()[p // PAGE].cuda(), (p % PAGE).cuda()
        kk, vv = m.caches[i].k[at, :, off].cpu(), m.caches[i].v[at, :, :, off].cpu()
        rows = slice(cu[r], cu[r + 1])
        want, tol = attn_ref(got["q"][rows].unflatten(1, (HQ, D)), kk, vv, n, D ** -0.5, t.float32)
        within(got["o"][rows].unflatten(1, (HQ, D)), want, tol, f"block {i} request {r}")
    rq, rd, _ = oracle.quantize_q8(got["o"].numpy().ravel(), 128)
    assert np.array_equal(got["o_act"].numpy().ravel(), rq) and same_bits(got["o_d"].numpy().ravel(), rd)
    within(got["out"], *matmul_ref(m.fmt, host["canon"]["o"], got["o_act"].numpy(), got["o_d"].numpy(), 128, t.float32), f"block {i} out")
    return got["out"], got["h"]


@pytest.mark.parametrize("fmt", [1, 2])
def test_attention_blocks_with_wide_products(fmt):
    from ternary_quantized_gemv_amd import staging
    m = Blocks(fmt, 64, with_adapters=False)
    for b in m.blocks:
        b.products = staging._Products(fmt, b.weights.values(), 128, 64, 1, b.device)
    for i, (lens, new) in enumerate(STEPS):
        s = m.step(lens, new, 100 + i)
        m.run(s, max(new), max(lens))
        torch().cuda.synchronize()
        x, res = s["x"].cpu(), None
        for b in range(2):
            x, res = check(m, b, s, x, res, lens, new)


@pytest.mark.parametrize("fmt", [1, 2])
def test_steps_on_the_drawn_tokens_where_they_lie(fmt):
    """The returned tokens themselves as the next step's ids: the tokens of a run that copies them first."""
    t = torch()
    prompt = t.randint(0, VOCAB, (62,), generator=gen(1))
    runs = []
    for how in ("copied", "eager", "captured"):
        m, lens = Decoder(fmt, 90), [37, 5, 20]
        token, _ = m.d.run(**m.step(lens, lens, prompt, 1), max_new=37, max_keys=37)
        assert token.data_ptr() == m.d.token.data_ptr()
        seen, graph, fixed = [token.tolist()], t.cuda.CUDAGraph(), None
        for i in range(5):
            lens = [n + 1 for n in lens]
            s = m.step(lens, [1, 1, 1], token.clone(), 10 + i)
            if how != "copied":
                s["ids"] = token
            if how == "captured":
                if fixed is None:
                    fixed = {k: v if k == "ids" else v.clone() for k, v in s.items()}
                    before = token.clone()
                    m.d.run(**fixed, max_new=1, max_keys=64)  # loads the kernels
                    token.copy_(before)
                    t.cuda.synchronize()
                    with t.cuda.graph(graph):
                        token, logprob = m.d.run(**fixed, max_new=1, max_keys=64)
                for k, v in s.items():
                    if k != "ids":
                        fixed[k].copy_(v)
                graph.replay()
            else:
                token, logprob = m.d.run(**s, max_new=1, max_keys=64)
            t.cuda.synchronize()
            seen.append(token.tolist() + logprob.tolist())
        runs.append(seen)
    assert runs[0] == runs[1] and runs[0] == runs[2]
