"""References in 64 bits for the operators between the products, written from
their formulas (include/bq.h) with CPU torch and numpy, and the error bounds
that the tests hold the kernels to."""
from __future__ import annotations

import numpy as np
import torch

import oracle

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dt) -> float:
    """The largest relative error of one rounding to dt."""
    return torch.finfo(dt).eps / 2


def gen(seed: int):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype)


def within(got, want, bound, what):
    """Every element within its bound; NaN never is."""
    got, want = got.double().cpu(), want.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = bad.flatten().nonzero()[0].item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {np.unravel_index(i, got.shape)}: "
                             f"{got.flatten()[i].item()} for {want.flatten()[i].item()}, bound "
                             f"{(bound + torch.zeros_like(off)).flatten()[i].item()}")


# ------------------------------------------------------------------- norm
def norm_ref(x, res, w, eps, qa, f16_scale):
    """The definition step by step: (h, v in f32, q int8, d f32)."""
    dt = x.dtype
    h = x if res is None else (x.float() + res.float()).to(dt)
    hf = h.float()
    r = (1.0 / torch.sqrt(hf.double().square().sum(1) / x.shape[1] + eps)).float()
    v = hf * r[:, None] * w.float()
    blocks = v.unflatten(1, (-1, qa)).numpy()
    d = np.abs(blocks).max(2) * (np.float32(1) / np.float32(127))
    if f16_scale:
        d = oracle.f32_to_f16(d.ravel()).view(np.float16).astype(np.float32).reshape(d.shape)
    with np.errstate(divide="ignore", invalid="ignore"):
        ratio = (blocks / d[..., None]).astype(np.float64)
    q = np.copysign(np.floor(np.abs(ratio) + 0.5), ratio).clip(-127, 127)
    q = np.where(d[..., None] == 0, 0, q).astype(np.int8).reshape(v.shape)
    return h, v, torch.from_numpy(q), torch.from_numpy(d)


# ----------------------------------------------------------------- append
def rotate_ref(x, pos, freq, weight, eps):
    """(rows, bound on the error of f32 arithmetic) of heads x [T, H, D] in 64
    bits.  The bound: the sum of squares, its root, its inverse and two
    products are within 11 half steps, cosine and sine within 4, their two
    products and the sum within 2: 17 * 2^-24 < 2^-19 of |v1| + |v2|."""
    v = x.double()
    if weight is not None:
        v = v / torch.sqrt(v.square().mean(-1, keepdim=True) + float(np.float32(eps))) * weight.double()
    half = freq.numel()
    ang = pos.double()[:, None] * freq.double()[None, :]
    c, s = ang.cos()[:, None, :], ang.sin()[:, None, :]
    a, b = v[..., :half], v[..., half:2 * half]
    out = torch.cat([a * c - b * s, b * c + a * s, v[..., 2 * half:]], -1)
    size = torch.cat([a.abs() + b.abs(), a.abs() + b.abs(), v[..., 2 * half:].abs()], -1)
    return out, size * 2.0 ** -19


# -------------------------------------------------------------- attention
def attn_ref(q, k_of, v_of, keys, scale, dt):
    """Rows q [n, Hq, D] of one request over its keys k_of, v_of [L, H, D]
    (cast by the caller): (out, bound) in 64 bits.

    The bound per row and value, with P|v| = sum p |v| / sum p: a score is off
    by at most (4 D + 8) 2^-24 sum |q k| scale (D products in up to three parts
    and their sum, the scaling and the subtraction of the maximum), which moves
    a weight by that much relative to itself, as numerator and denominator;
    exp2 and the sums over the keys add (L / 16 + 64) 2^-23; 16-bit rows round
    every weight and the result once."""
    n, Hq, D = q.shape
    H = k_of.shape[1]
    out = torch.zeros(n, Hq, D, dtype=torch.float64)
    bound = torch.zeros(n, Hq, D, dtype=torch.float64)
    if keys == 0:
        return out, bound
    hidden = torch.arange(keys)[None, :] > (keys - n + torch.arange(n))[:, None]
    for h in range(Hq):
        k, v = k_of[:, h // (Hq // H)].double(), v_of[:, h // (Hq // H)].double()
        s = (q[:, h].double() @ k.t()) * scale
        size = (q[:, h].double().abs() @ k.abs().t()) * abs(scale)
        s = s.masked_fill(hidden, -torch.inf)
        top = s.max(1, keepdim=True).values
        p = torch.exp(s - torch.where(top.isinf(), torch.zeros_like(top), top))
        l = p.sum(1, keepdim=True)
        l = torch.where(l > 0, l, torch.ones_like(l))
        o, pv = p @ v / l, p @ v.abs() / l
        rel = 2 * (4 * D + 8) * 2.0 ** -24 * size.masked_fill(hidden, 0).max(1, keepdim=True).values
        rel = rel + (keys / 16 + 64) * 2.0 ** -23
        if dt != torch.float32:
            rel = rel + half_step(dt)
        out[:, h] = o
        bound[:, h] = rel * pv + half_step(dt) * o.abs()
    return out, bound + 1e-30


class Paged:
    """A cache of `keys[b]` random tokens per request in pages of random order;
    every place that holds no token, and two spare pages, are NaN.  Table
    entries that no key needs are out of range."""

    def __init__(self, keys, heads, dim, page, dtype, seed, cols=None, spread=1.5):
        g = gen(seed)
        self.k_of = [normal(g, n, heads, dim, dtype=dtype, scale=spread) for n in keys]
        self.v_of = [normal(g, n, heads, dim, dtype=dtype) for n in keys]
        each = [-(-n // page) for n in keys]
        pages = sum(each) + 2
        k = torch.full((pages, heads, page, dim), float("nan"), dtype=dtype)
        v = torch.full((pages, heads, dim, page), float("nan"), dtype=dtype)
        order = torch.randperm(pages, generator=g)
        table = torch.full((len(keys), cols or max(max(each), 1)), 1 << 30, dtype=torch.int32)
        table[:, 1::2] = -7
        at = 0
        for b, n in enumerate(keys):
            for c in range(each[b]):
                p, lo, hi = int(order[at]), c * page, min(n, (c + 1) * page)
                k[p, :, :hi - lo] = self.k_of[b][lo:hi].transpose(0, 1)
                v[p, :, :, :hi - lo] = self.v_of[b][lo:hi].permute(1, 2, 0)
                table[b, c] = p
                at += 1
        self.k, self.v, self.table = k, v, table


# --------------------------------------------------------------- adapters
def adapters_ref(x, a, b, gain, y):
    """One request's rows through one adapter: (out, bound).  u = A x and B u
    are sums of n and rank products in f32: (n / 32 + 64) and (rank + 64)
    roundings of 2^-23 at most, the gain and the addition one each."""
    xd, ad, bd, g = x.double(), a.double(), b.double(), abs(float(gain))
    out = y.double() + float(gain) * (xd @ ad.t()) @ bd.t()
    size = (xd.abs() @ ad.abs().t()) @ bd.abs().t() * g
    steps = x.shape[1] / 32 + 64 + a.shape[0] + 64 + 2
    return out, steps * 2.0 ** -23 * size + 2.0 ** -23 * (y.double().abs() + out.abs())
