"""staging.StagedAttention without a GPU: where its buffers lie and which device
its calls are made under, with stand-ins for the calls."""
from types import SimpleNamespace

import pytest
import torch

import ternary_quantized_gemv_amd.staging as staging

HIDDEN, HQ, H, D, T = 256, 4, 2, 64, 3


@pytest.mark.parametrize("index", [0, 1])
def test_attention_block_on_the_caches_device(index, monkeypatch):
    """Buffers and weights go to the cache's device, whichever is current, and
    run() makes all its calls with that device current: the products and the
    quantizer take the current device's stream."""
    dev = torch.device("cuda", index)
    asked, calls, stack = [], [], [7]
    norm, freq, ids = torch.ones(HIDDEN), torch.ones(D // 2), torch.zeros(1)

    class Device:
        def __init__(self, d):
            self.d = d if isinstance(d, int) else torch.device(d).index

        def __enter__(self):
            stack.append(self.d)

        def __exit__(self, *a):
            stack.pop()

    def allocate(real):
        def make(*a, device=None, **k):
            asked.append(torch.device(device))
            return real(*a, **k)
        return make

    def upload(fmt, canon, rows, cols, device="cuda"):
        asked.append(torch.device(device))
        return SimpleNamespace(rows=rows, cols=cols)

    monkeypatch.setattr(staging, "Weights", SimpleNamespace(upload=upload))
    monkeypatch.setattr(staging, "Act", lambda *a: None)
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, allocate(getattr(torch, name)))
    for name in ("bq_rmsnorm_q8", "bq_kv_append", "bq_paged_attn", "bq_adapters_add", "bq_quantize_act_q8",
                 "bq_q1_0_matvec", "bq_q2_0_matvec"):
        monkeypatch.setattr(staging, name, lambda *a, name=name, **k: calls.append((name, stack[-1])))
    monkeypatch.setattr(torch.cuda, "device", Device)
    cache = SimpleNamespace(heads=H, dim=D, dev=index, k=SimpleNamespace(device=dev))
    block = staging.StagedAttention(1, {n: None for n in "qkvo"}, HIDDEN, HQ, cache, norm, freq, 16, adapters={"q": None, "o": None})
    assert len(asked) == 15 and all(d == dev for d in asked), asked
    x, cu = torch.ones(T, HIDDEN), torch.tensor([0, T])
    out, h = block.run(x, None, None, None, cu, None, None, T, T, ids=ids)
    assert out.shape == h.shape == (T, HIDDEN)
    assert {c[0] for c in calls} >= {"bq_rmsnorm_q8", "bq_kv_append", "bq_paged_attn", "bq_adapters_add",
                                     "bq_quantize_act_q8", "bq_q1_0_matvec"}
    assert all(c[1] == index for c in calls), calls
    assert stack == [7]
