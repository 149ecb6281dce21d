"""References in 64 bits for the operators around the layers, written from
their formulas (include/bq.h) with numpy and CPU torch, and the error bounds
that the tests hold the kernels to."""
from __future__ import annotations

import math

import numpy as np
import torch

from layer_util import half_step

ACTS = {"none": 0, "silu": 1, "gelu": 2, "relu2": 3}
EPS = 2.0 ** -24  # the largest relative error of one rounding to f32


def codes(fmt: int, canon: np.ndarray):
    """Canonical blocks -> (weights without their scale [rows, blocks, n], f16 scales widened [rows, blocks])."""
    d = np.ascontiguousarray(canon[:, :, :2]).view("<f2")[:, :, 0].astype(np.float64)
    payload = canon[:, :, 2:]
    if fmt == 1:
        w = np.unpackbits(payload, axis=2, bitorder="little").astype(np.int64) * 2 - 1
    else:
        w = ((payload[..., None] >> np.array([0, 2, 4, 6], np.uint8)) & 3).reshape(*payload.shape[:2], 64).astype(np.int64) - 1
    return w, d


def activate(x, name):
    """An activation in 64 bits (numpy)."""
    with np.errstate(over="ignore"):
        if name == "silu":
            return x / (1.0 + np.exp(-x))
        if name == "gelu":
            return x / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))
    return np.maximum(x, 0.0) ** 2 if name == "relu2" else x


def matmul_ref(fmt, canon, q, d, qa, dt, bias=None, act="none", mul=None, res=None):
    """(y, bound) in 64 bits.  q int8 [T, cols], d f32 [T, cols / qa] (numpy); bias f32 [rows]; mul, res [T, rows]
    (torch, of type dt).

    The bound: each of the G groups of a row (what one weight and one activation scale cover; G at most cols / 32)
    is rounded once when it is scaled by d0 and once at each addition behind it, G of them and at most 16 more
    where parts of k are added up: (G + 18) half steps of the sum of magnitudes, counted from the error-free sum,
    one more for the bias.  Then the activation: its slope is at most 1.13 (relu2: 2 |x|), exp's argument z is off
    by 4 half steps and exp by 2, which moves x s(z) by at most |x| z s (1 - s) <= 0.28 |x| times as much, and
    division, sum and product cost 4 half steps of the result; 2 for the product and the sum with mul and res."""
    w, d0 = codes(fmt, canon)
    G = min(qa, w.shape[2])
    T, cols = q.shape
    rows = w.shape[0]
    wd = (w * d0[..., None]).reshape(rows, cols)
    xs = q.astype(np.float64) * np.repeat(d.astype(np.float64), qa, axis=1)
    y = xs @ wd.T
    size = np.zeros((T, rows))  # the groups' magnitudes
    qi, wi = q.reshape(T, cols // G, G).astype(np.float64), w.reshape(rows, cols // G, G).astype(np.float64)
    dw = np.repeat(d0, w.shape[2] // G, axis=1)
    dx = np.repeat(d.astype(np.float64), qa // G, axis=1)
    for g in range(cols // G):
        size += np.abs(qi[:, g] @ wi[:, g].T) * (np.abs(dx[:, g])[:, None] * np.abs(dw[:, g])[None])
    err = (cols // G + 18) * EPS * size
    if bias is not None:
        y = y + bias.double().numpy()
        err = err + EPS * np.abs(y)
    x = y
    y = activate(x, act)
    if act == "relu2":
        err = 2 * (np.abs(x) + err) * err + 2 * EPS * y
    elif act != "none":
        err = 1.13 * err + EPS * (0.28 * 6 * np.abs(x) + 4 * np.abs(y))
    if mul is not None:
        y, err = y * mul.double().numpy(), err * np.abs(mul.double().numpy())
        err = err + EPS * np.abs(y)
    if res is not None:
        y = y + res.double().numpy()
        err = err + EPS * np.abs(y)
    tiny = 2.0 ** -25 if dt == torch.float16 else 2.0 ** -133  # half the distance of subnormal results
    err = 1.001 * err
    err = err + half_step(dt) * (np.abs(y) + err) + tiny
    return torch.from_numpy(y), torch.from_numpy(err)


def gated_ref(gate, up, act, qa, f16_scale):
    """(v f32, q int8, d f32, next) step by step; next: v where it is rounded the other way, for the values that
    64-bit arithmetic cannot tell apart (v elsewhere)."""
    exact = activate(gate.double().numpy(), act) * up.double().numpy()
    v = exact.astype(np.float32)
    lo, hi = (exact * (1 - 2.0 ** -46)).astype(np.float32), (exact * (1 + 2.0 ** -46)).astype(np.float32)
    return v, np.where(lo == v, hi, lo), *quants_ref(v, qa, f16_scale)


def quants_ref(v, qa, f16_scale):
    """The norm's quantizer of f32 values [T, n]: (q int8, d f32)."""
    import oracle
    blocks = v.reshape(v.shape[0], -1, qa)
    d = np.abs(blocks).max(2) * (np.float32(1) / np.float32(127))
    if f16_scale:
        d = oracle.f32_to_f16(d.ravel()).view(np.float16).astype(np.float32).reshape(d.shape)
    with np.errstate(divide="ignore", invalid="ignore"):
        ratio = (blocks / d[..., None]).astype(np.float64)
    q = np.copysign(np.floor(np.abs(ratio) + 0.5), ratio).clip(-127, 127)
    return np.where(d[..., None] == 0, 0, q).astype(np.int8).reshape(v.shape), d


class Ranked:
    """A row of logits in the order that bq_sample draws from, in 64 bits."""

    def __init__(self, logits, temperature=1.0):
        x = np.asarray(logits, np.float64)
        x = np.where(np.isnan(x), -np.inf, x)
        self.order = np.argsort(-x, kind="stable")
        x = x[self.order]
        self.top = x[0]
        self.greedy = not temperature > 0
        with np.errstate(invalid="ignore", over="ignore"):
            y = np.where(x == x[0], 0.0, (x - x[0]) / (temperature if temperature > 0 else 1.0))
            self.w = np.where(x == x[0], 1.0, 0.0) if self.greedy else np.exp(np.where(np.isnan(y), -np.inf, y))
        if self.top == -np.inf:
            self.w[:] = 0
        self.sums = np.cumsum(self.w)

    def kept(self, k=0, p=1.0, least=0.0):
        """How many of the order the filters keep."""
        n = len(self.w)
        if self.greedy:
            return 1
        if k > 0:
            n = min(n, k)
        if p < 1:
            n = min(n, int((self.sums[:n] < float(np.float32(p)) * self.sums[n - 1]).sum()) + 1)
        if least > 0:
            n = min(n, int((self.w >= float(np.float32(least))).sum()))
        return max(n, 1)

    def inside(self, rank, kept):
        """A u in the middle of the share of the token at this rank."""
        before = self.sums[rank - 1] if rank else 0.0
        return np.float32((before + 0.5 * self.w[rank]) / self.sums[kept - 1])

    def logprob(self, rank):
        return 0.0 if self.greedy else float(np.log(self.w[rank] / self.sums[-1]))
