"""staging.StagedMLP without a GPU: which device its buffers lie on and its calls
are made under, with stand-ins for the calls."""
from types import SimpleNamespace

import pytest
import torch

import ternary_quantized_gemv_amd.staging as staging

HIDDEN, INNER = 256, 512


@pytest.mark.parametrize("device", ["cuda", "cuda:1", torch.device("cuda"), torch.device("cuda", 1)])
@pytest.mark.parametrize("tokens", [3, 40])
def test_mlp_stays_on_its_device(device, tokens, monkeypatch):
    """Built while device 1 is current, run while device 0 is: a device without an index means the one that was
    current, and all calls are made under it (the products take the current device's stream)."""
    asked, calls, stack = [], [], [1]

    class Device:
        def __init__(self, d):
            self.d = torch.device(d).index

        def __enter__(self):
            stack.append(stack[-1] if self.d is None else self.d)

        def __exit__(self, *a):
            stack.pop()

    def empty(*a, device=None, real=torch.empty, **k):
        asked.append(torch.device(device))
        return real(*a, **k)

    def upload(fmt, canon, rows, cols, device="cuda"):
        asked.append(torch.device(device))
        return SimpleNamespace(rows=rows, cols=cols)

    monkeypatch.setattr(staging, "Weights", SimpleNamespace(upload=upload))
    monkeypatch.setattr(staging, "Act", lambda *a: None)
    monkeypatch.setattr(staging, "bq_matmul_work_bytes", lambda *a: 64)
    monkeypatch.setattr(torch, "empty", empty)
    for name in ("bq_rmsnorm_q8", "bq_gated_q8", "bq_matmul", "bq_q1_0_matvec"):
        monkeypatch.setattr(staging, name, lambda *a, name=name, **k: calls.append((name, stack[-1])))
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: stack[-1])
    mlp = staging.StagedMLP(1, {n: None for n in ("gate", "up", "down")}, HIDDEN, INNER, torch.ones(HIDDEN), 64, device=device)
    assert len(asked) == 12 and all(d == torch.device("cuda", 1) for d in asked), asked
    stack[:] = [0]
    mlp.run(torch.ones(tokens, HIDDEN), None)
    assert {c[0] for c in calls} == {"bq_rmsnorm_q8", "bq_gated_q8", "bq_matmul" if tokens > 16 else "bq_q1_0_matvec"}
    assert all(c[1] == 1 for c in calls), calls
    assert stack == [0]
