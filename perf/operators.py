"""Cases of the operators that stand between the products of a decode or
prompt step, for timing them and for comparing them with their plain forms:

  norm      residual addition, root-mean-square norm and 8-bit activation in
            one pass (bq_rmsnorm_q8): what every group of products reads
  append    per-head norm, rotation by position, and the write of new keys and
            values into the paged cache (bq_kv_append)
  attn      attention of each request's new tokens, one or many, over its
            pages of the cache, causal, grouped heads (bq_paged_attn)
  adapters  the low-rank updates of many requests added to the outputs of a
            shared projection (bq_adapters_add)

With ``own`` false, ``run`` computes the operator from elementary torch
operations in 32 bits (64 where a rounding border or a far angle asks for it);
with ``own`` true it makes the calls of this package.  ``exact`` evaluates the
definition in 64 bits.  Head counts, head size and matrix sizes are those of
the decode token this repository benches (32 query heads and 8 key heads of
128, 4096 and 12288 columns) or generic.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
DEV = "cuda"
EPS = 1e-6


def listed():
    return [
        # one decode token: the norm in front of q, k, v or gate, up
        norm("norm_token", 1, 4096, "f32", 128),
        # a prompt of an odd number of tokens in bf16, the q8_0 block length,
        # the normed row itself kept for the adapters
        norm("norm_prompt", 4099, 4096, "bf16", 32, y=True),
        # the sixteen columns a product takes, f32 outputs of the products, far positions
        append("append_batch", 16, 32, 8, 128, 128, "f32", "bf16", 16, True, 131072),
        # a prompt: f16 throughout, larger pages, rotation of the head's first half only
        append("append_prompt", 2049, 32, 8, 128, 64, "f16", "f16", 64, False, 4096),
        # one request, one token, f32 queries: latency and the split over keys
        attn("attn_token", 1, 1, 8191, 32, 8, 128, "f32", "bf16", 16, 1),
        # a serving batch of decode tokens over caches of very different lengths
        attn("attn_batch", 32, 1, 8192, 32, 8, 128, "bf16", "bf16", 16, 2),
        # sixteen new tokens of one request (the products' column limit) over a long cache
        attn("attn_columns", 1, 16, 16384, 32, 8, 128, "f32", "f16", 32, 3),
        # a chunk of a prompt over what earlier chunks left in the cache
        attn("attn_chunk", 1, 512, 30011, 32, 8, 128, "bf16", "bf16", 64, 4),
        # whole prompts of different lengths packed together, nothing before them
        attn("attn_prompt", 3, 4999, 4999, 32, 8, 128, "bf16", "bf16", 64, 5, fresh=True),
        # one token of one request with a small adapter
        adapters("adapters_token", 1, 1, 4096, 4096, 8, 4, "f32", "bf16", 6),
        # sixteen requests, one token each, their adapters among 32
        adapters("adapters_batch", 16, 1, 4096, 12288, 16, 32, "f32", "bf16", 7),
        # prompts of five requests, one of them without an adapter
        adapters("adapters_prompt", 5, 601, 4096, 4096, 64, 8, "bf16", "bf16", 8),
    ]


def norm(name, tokens, n, type, qa, residual=True, y=False, f16_scale=False):
    return {"name": name, "op": "norm", "tokens": tokens, "n": n, "type": type, "qa": qa, "residual": residual,
            "y": y, "f16_scale": f16_scale}


def append(name, tokens, q_heads, kv_heads, dim, rot, type, cache, page, norms, far):
    return {"name": name, "op": "append", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "type": type, "cache": cache, "page": page, "norms": norms, "far": far}


def attn(name, requests, max_new, max_keys, q_heads, kv_heads, dim, type, cache, page, mix, fresh=False):
    return {"name": name, "op": "attn", "requests": requests, "max_new": max_new, "max_keys": max_keys,
            "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "type": type, "cache": cache, "page": page,
            "mix": mix, "fresh": fresh}


def adapters(name, requests, max_new, n, rows, rank, count, type, weights, mix):
    return {"name": name, "op": "adapters", "requests": requests, "max_new": max_new, "n": n, "rows": rows,
            "rank": rank, "count": count, "type": type, "weights": weights, "mix": mix}


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "append", "attn", "attn", "adapters"))
    if op == "norm":
        qa = rng.choice((32, 64, 128))
        c = norm("", _log(rng, 1, 6000), qa * _log(rng, 1, 16384 // qa), rng.choice(("f32", "f16", "bf16")), qa,
                 rng.random() < 0.8, rng.random() < 0.5, rng.random() < 0.3)
        while c["tokens"] * c["n"] > 4099 * 4096:
            c["tokens"] = (c["tokens"] + 1) // 2
    elif op == "append":
        dim = rng.choice((64, 128))
        type = rng.choice(("f32", "f16", "bf16"))
        heads = rng.choice((1, 2, 4, 8))
        c = append("", _log(rng, 1, 4000), heads * rng.choice((1, 2, 3, 4, 5, 8)), heads, dim,
                   rng.choice((dim, dim, dim // 2)), type, type if type != "f32" else rng.choice(("f16", "bf16")),
                   rng.choice((16, 32, 64, 128)), rng.random() < 0.5, _log(rng, 1000, 1 << 20))
    elif op == "attn":
        kind = rng.choice(("token", "token", "few", "chunk", "fresh"))
        cache = rng.choice(("f16", "bf16"))
        heads = rng.choice((1, 2, 4, 8))
        new = {"token": 1, "few": rng.randint(2, 16), "chunk": _log(rng, 17, 1024), "fresh": _log(rng, 2, 5000)}[kind]
        keys = new if kind == "fresh" else _log(rng, max(new, 16), 30011)
        c = attn("", _log(rng, 1, 48), new, keys, heads * rng.choice((1, 2, 3, 4, 5, 7, 8)), heads,
                 rng.choice((64, 128)), rng.choice((cache, cache, "f32")), cache, rng.choice((16, 32, 64, 128)),
                 rng.randrange(1 << 20), kind == "fresh")
        while _attn_cost(c) > 1 and c["requests"] > 1:
            c["requests"] = (c["requests"] + 1) // 2
        while _attn_cost(c) > 1:
            c["max_new"] = max(1, c["max_new"] // 2)
            c["max_keys"] = c["max_new"] if c["fresh"] else max(c["max_new"], c["max_keys"] * 3 // 4)
    else:
        one = rng.random() < 0.5
        c = adapters("", _log(rng, 1, 64) if one else _log(rng, 1, 8), 1 if one else _log(rng, 2, 800),
                     128 * _log(rng, 1, 96), _log(rng, 16, 12288), 8 * _log(rng, 1, 16), _log(rng, 1, 32),
                     rng.choice(("f32", "f16", "bf16")), "bf16", rng.randrange(1 << 20))
        c["weights"] = c["type"] if c["type"] != "f32" else rng.choice(("f16", "bf16"))
    del c["name"]
    return c


def _attn_cost(c):
    """At most 1: no more work than attn_prompt, no more scores in the plain form, no more cache than attn_batch."""
    big = attn("", 3, 4999, 4999, 32, 8, 128, "f32", "bf16", 64, 5, True)

    def scores(a):
        return a["requests"] * a["q_heads"] * a["max_new"] * a["max_keys"]

    return max(work(c)["flops"] / work(big)["flops"] * (3 if c["type"] == "f32" else 1), scores(c) / scores(big),
               work(c)["bytes"] / 0.5e9)


# ------------------------------------------------------------------ lengths
# The lengths and adapters of a case's requests follow from the case alone.
def lengths(case):
    """(new tokens, keys) of each request: the first has the most of both; without earlier keys, keys = new."""
    r = random.Random(case["mix"])
    new = [case["max_new"]] + [_log(r, 1, case["max_new"]) for _ in range(case["requests"] - 1)]
    if case["fresh"]:
        return new, new
    return new, [case["max_keys"]] + [_log(r, n, case["max_keys"]) for n in new[1:]]


def adapter_lengths(case):
    """(tokens, adapter) of each request; one request in five has none (-1) where there are several."""
    r = random.Random(case["mix"])
    new = [case["max_new"]] + [_log(r, 1, case["max_new"]) for _ in range(case["requests"] - 1)]
    return new, [-1 if i % 5 == 4 else r.randrange(case["count"]) for i in range(case["requests"])]


def offsets(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return cu


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)

    def normal(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        x = torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, scale, generator=g)
        return x.add_(shift) if shift else x

    if case["op"] == "norm":
        T, n, dt = case["tokens"], case["n"], DT[case["type"]]
        s["x"] = normal(T, n, dtype=dt)
        s["res"] = normal(T, n, dtype=dt, scale=2.0) if case["residual"] else None
        s["w"] = normal(n, dtype=dt, scale=0.1, shift=1.0)
        s["h"] = torch.empty(T, n, dtype=dt, device=DEV)
        s["y_out"] = torch.empty(T, n, dtype=dt, device=DEV) if case["y"] else None
        s["q"] = torch.empty(T, n, dtype=torch.int8, device=DEV)
        s["d"] = torch.empty(T, n // case["qa"], dtype=torch.float32, device=DEV)
    elif case["op"] == "append":
        T, Hq, H, D, page = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
        dt, ct = DT[case["type"]], DT[case["cache"]]
        pages = -(-T // page) + 3
        s["new_q"], s["new_k"], s["new_v"] = (normal(T, h, D, dtype=dt) for h in (Hq, H, H))
        s["k"], s["v"] = normal(pages, H, page, D, dtype=ct), normal(pages, H, D, page, dtype=ct)
        # consecutive tokens in consecutive places of pages in any order, as a prompt's or,
        # for the sixteen columns, as different requests' tokens
        order = torch.randperm(pages, generator=g, device=DEV)
        at = torch.arange(T, device=DEV) + 5 if T > 16 else torch.randperm(pages * page, generator=g, device=DEV)[:T]
        s["slot"] = order[at // page] * page + at % page
        start = torch.randint(0, max(1, case["far"] - T), (1,), generator=g, device=DEV)
        s["pos"] = (torch.arange(T, device=DEV) + start).to(torch.int32)
        s["freq"] = (1e6 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEV) / case["rot"])).float()
        s["q_norm"], s["k_norm"] = (normal(D, scale=0.1, shift=1.0) for _ in range(2)) if case["norms"] else (None, None)
        s["q_out"] = torch.empty(T, Hq, D, dtype=dt, device=DEV)
    elif case["op"] == "attn":
        new, keys = lengths(case)
        H, D, page, ct = case["kv_heads"], case["dim"], case["page"], DT[case["cache"]]
        each = [-(-k // page) for k in keys]
        pages = sum(each) + 2
        s["k"], s["v"] = normal(pages, H, page, D, dtype=ct, scale=1.5), normal(pages, H, D, page, dtype=ct)
        s["new_q"] = normal(sum(new), case["q_heads"], D, dtype=DT[case["type"]])
        # page tables: the used entries take pages in random order, the others hold -1
        column = torch.arange(max(each), device=DEV)
        counts = torch.tensor(each, device=DEV)
        first = torch.tensor(offsets(each)[:-1], device=DEV)
        order = torch.randperm(pages, generator=g, device=DEV)
        table = order[(first[:, None] + column[None, :]).clamp_(max=pages - 1)]
        s["table"] = torch.where(column[None, :] < counts[:, None], table, -1).to(torch.int32)
        s["cu"] = torch.tensor(offsets(new), dtype=torch.int32, device=DEV)
        s["lens"] = torch.tensor(keys, dtype=torch.int32, device=DEV)
        s["scale"] = 1.0 / math.sqrt(D)
        s["out"] = torch.empty_like(s["new_q"])
    else:
        new, ids = adapter_lengths(case)
        n, rows, rank, count = case["n"], case["rows"], case["rank"], case["count"]
        wt = DT[case["weights"]]
        s["x"] = normal(sum(new), n, dtype=DT[case["type"]])
        s["a"] = normal(count, rank, n, dtype=wt, scale=1.0 / math.sqrt(n))
        s["b"] = normal(count, rows, rank, dtype=wt, scale=1.0 / math.sqrt(rank))
        s["gain"] = torch.empty(count, device=DEV).uniform_(0.5, 2.0, generator=g)
        s["y"] = normal(sum(new), rows)
        s["out"] = torch.empty_like(s["y"])
        s["cu"] = torch.tensor(offsets(new), dtype=torch.int32, device=DEV)
        s["ids"] = torch.tensor(ids, dtype=torch.int32, device=DEV)
        s["most"] = max(new)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"norm": run_norm, "append": run_append, "attn": run_attn, "adapters": run_adapters}[s["op"]](s)


def run_norm(s):
    T, n, qa = s["tokens"], s["n"], s["qa"]
    if own:
        import ternary_quantized_gemv_amd as bq
        bq.bq_rmsnorm_q8(s["x"], s["w"], EPS, qa, s["q"], s["d"], res=s["res"], h=s["h"], y=s["y_out"],
                         f16_scale=s["f16_scale"])
        h, q, d, y = s["h"], s["q"], s["d"], s["y_out"]
    else:
        dt = s["x"].dtype
        h = (s["x"].float() + s["res"].float()).to(dt) if s["residual"] else s["x"].clone()
        hf = h.float()
        r = (1.0 / torch.sqrt(hf.double().square().sum(1) / n + EPS)).float()  # next to a border: 64 bits
        normed = hf * r[:, None] * s["w"].float()
        blocks = normed.view(T, n // qa, qa)
        d = blocks.abs().amax(2) / 127.0
        if s["f16_scale"]:
            d = d.half().float()
        ratio = blocks / torch.where(d == 0, torch.ones_like(d), d)[..., None]
        q = torch.where(ratio < 0, -1.0, 1.0) * torch.floor(ratio.abs().double() + 0.5).float()  # ties away from zero
        q = torch.where(d[..., None] == 0, torch.zeros_like(q), q.clamp_(-127, 127)).view(T, n)
        y = normed.to(dt) if s["y"] else None
    # the quants as the values that they stand for
    out = {"h": h, "d": d, "values": (q.view(T, n // qa, qa) * d.view(T, n // qa, 1)).view(T, n)}
    if s["y"]:
        out["y"] = y
    return out


def run_append(s):
    if own:
        import ternary_quantized_gemv_amd as bq
        bq.bq_kv_append(bq.KVCache(s["k"], s["v"]), s["new_k"], s["new_v"], s["pos"], s["slot"], s["freq"],
                        q=s["new_q"], q_out=s["q_out"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        return {"k": s["k"], "v": s["v"], "q": s["q_out"]}
    half, page = s["rot"] // 2, s["page"]
    angle = s["pos"].double()[:, None] * s["freq"].double()[None, :]
    c, sn = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * (1.0 / torch.sqrt(x.square().mean(2, keepdim=True) + EPS)) * weight
        x1, x2 = x[..., :half], x[..., half:2 * half]
        return torch.cat((x1 * c - x2 * sn, x2 * c + x1 * sn, x[..., 2 * half:]), 2)

    at, off = (s["slot"] // page)[:, None], (s["slot"] % page)[:, None]
    head = torch.arange(s["kv_heads"], device=DEV)[None, :]
    s["k"][at, head, off] = turned(s["new_k"], s["k_norm"]).to(s["k"].dtype)
    s["v"][at, head, :, off] = s["new_v"].float().to(s["v"].dtype)
    return {"k": s["k"], "v": s["v"], "q": turned(s["new_q"], s["q_norm"]).to(s["new_q"].dtype)}


def run_attn(s):
    if own:
        import ternary_quantized_gemv_amd as bq
        bq.bq_paged_attn(bq.KVCache(s["k"], s["v"]), s["new_q"], s["cu"], s["lens"], s["table"], s["scale"],
                         s["max_new"], s["max_keys"], s["out"])
        return s["out"]
    B, N, S, H, D, page = s["requests"], s["max_new"], s["max_keys"], s["kv_heads"], s["dim"], s["page"]
    G = s["q_heads"] // H
    cu, lens = s["cu"].long(), s["lens"].long()
    table = s["table"].long().clamp(min=0)
    new = cu[1:] - cu[:-1]
    i, j = torch.arange(N, device=DEV), torch.arange(S, device=DEV)
    # every request padded to the most new tokens and the most keys
    q = s["new_q"].float()[(cu[:-1, None] + i[None, :]).clamp(max=s["new_q"].shape[0] - 1)]  # B N Hq D
    q = q.view(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    k = s["k"][table].float().permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)[:, :, :S]
    v = s["v"][table].float().permute(0, 2, 1, 4, 3).reshape(B, H, -1, D)[:, :, :S]
    v = torch.where((j[None, :] < lens[:, None])[:, None, :, None], v, torch.zeros_like(v))
    sees = j[None, None, :] <= (lens - new)[:, None, None] + i[None, :, None]  # B N S
    scores = (torch.matmul(q, k.transpose(2, 3)) * s["scale"]).view(B, H, G, N, S)
    scores = scores.masked_fill_(~sees[:, None, None], float("-inf"))
    most = scores.amax(4, keepdim=True)
    p = torch.exp(scores.sub_(torch.where(most == float("-inf"), torch.zeros_like(most), most)))
    total = p.sum(4, keepdim=True)
    o = torch.matmul(p.view(B, H, G * N, S), v).view(B, H, G, N, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(B, N, H * G, D)
    t = torch.arange(s["new_q"].shape[0], device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return o[b, t - cu[b]].to(s["new_q"].dtype)


def run_adapters(s):
    if own:
        import ternary_quantized_gemv_amd as bq
        bq.bq_adapters_add(bq.Adapters(s["a"], s["b"], s["gain"]), s["x"], s["cu"], s["ids"], s["most"], s["y"],
                           out=s["out"])
        return s["out"]
    T, count, rank = s["x"].shape[0], s["count"], s["rank"]
    # all adapters of all tokens, those that a token does not have times zero
    t = torch.arange(T, device=DEV)
    of = s["ids"].long()[torch.searchsorted(s["cu"].long()[1:].contiguous(), t, right=True)]
    share = (of[:, None] == torch.arange(count, device=DEV)[None, :]).float() * s["gain"][None, :]
    low = torch.matmul(s["x"].float(), s["a"].float().view(count * rank, -1).t()).view(T, count, rank)
    low = (low * share[..., None]).view(T, count * rank)
    return s["y"] + torch.matmul(low, s["b"].float().permute(0, 2, 1).reshape(count * rank, -1))


# ------------------------------------------------------------------ work
def work(case):
    if case["op"] == "norm":
        T, n, b = case["tokens"], case["n"], SIZE[case["type"]]
        # x, residual, new residual, y; quants and scales; the weight
        moved = T * n * b * (2 + case["residual"] + case["y"]) + T * n + 4 * T * (n // case["qa"]) + n * b
        return {"bytes": moved, "flops": 8 * T * n}
    if case["op"] == "append":
        T, D, Hq, H = case["tokens"], case["dim"], case["q_heads"], case["kv_heads"]
        b, cb = SIZE[case["type"]], SIZE[case["cache"]]
        # q in and out, k and v in, their places of the cache out; positions, slots, frequencies, norm weights
        moved = T * D * (2 * Hq * b + 2 * H * (b + cb)) + 12 * T + 2 * case["rot"] + 8 * D * case["norms"]
        return {"bytes": moved, "flops": T * (Hq + H) * (3 * case["rot"] + 4 * D * case["norms"])}
    if case["op"] == "attn":
        new, keys = lengths(case)
        Hq, H, D = case["q_heads"], case["kv_heads"], case["dim"]
        seen = sum(n * k - n * (n - 1) // 2 for n, k in zip(new, keys))
        moved = 2 * sum(new) * Hq * D * SIZE[case["type"]] + 2 * sum(keys) * H * D * SIZE[case["cache"]]
        moved += 4 * sum(-(-k // case["page"]) for k in keys)
        return {"bytes": moved, "flops": 4 * D * Hq * seen}
    new, ids = adapter_lengths(case)
    n, rows, rank = case["n"], case["rows"], case["rank"]
    used, T = len({i for i in ids if i >= 0}), sum(new)
    with_one = sum(t for t, i in zip(new, ids) if i >= 0)
    moved = with_one * n * SIZE[case["type"]] + 8 * T * rows + used * rank * (n + rows) * SIZE[case["weights"]]
    return {"bytes": moved, "flops": 2 * with_one * rank * (n + rows)}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": exact_norm, "append": exact_append, "attn": exact_attn, "adapters": exact_adapters}[s["op"]](s)


def exact_norm(s):
    """The norm reads the stored (rounded) sum; the quants have no value in 64 bits, nor have scales rounded to f16."""
    total = s["x"].double() + (s["res"].double() if s["residual"] else 0.0)
    stored = total.to(s["x"].dtype).double()
    rows = stored / (stored.pow(2).mean(1, keepdim=True) + EPS).sqrt() * s["w"].double()
    scale = rows.abs().unflatten(1, (-1, s["qa"])).max(2).values / 127
    out = {"h": total, "d": None if s["f16_scale"] else scale, "values": None}
    if s["y"]:
        out["y"] = rows
    return out


def exact_append(s):
    half = s["rot"] // 2
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["pos"].double()[:, None] * s["freq"].double())

    def rotated(x, weight):
        x = x.double()
        if weight is not None:
            x = x * weight.double() / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
        z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn[:, None, :]
        return torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)

    k, v = s["k"].double(), s["v"].double()
    # places [page, offset] flattened, the cache seen as [place, head, dim]
    kp = k.permute(0, 2, 1, 3).flatten(0, 1).index_copy(0, s["slot"], rotated(s["new_k"], s["k_norm"]))
    vp = v.permute(0, 3, 1, 2).flatten(0, 1).index_copy(0, s["slot"], s["new_v"].double())
    k = kp.unflatten(0, (-1, s["page"])).permute(0, 2, 1, 3)
    v = vp.unflatten(0, (-1, s["page"])).permute(0, 2, 3, 1)
    return {"k": k, "v": v, "q": rotated(s["new_q"], s["q_norm"])}


def exact_attn(s):
    """Request by request and key head by key head."""
    cu, lens, page, D = s["cu"].tolist(), s["lens"].tolist(), s["page"], s["dim"]
    G = s["q_heads"] // s["kv_heads"]
    out = torch.zeros(s["new_q"].shape, dtype=torch.float64, device=DEV)
    for b, n_keys in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        pages = s["table"][b, :-(-n_keys // page)].long()
        last = n_keys - (hi - lo) + torch.arange(hi - lo, device=DEV)  # the last key each new token sees
        hidden = torch.arange(n_keys, device=DEV)[None, :] > last[:, None]
        for h in range(s["kv_heads"]):
            k = s["k"][pages, h].double().reshape(-1, D)[:n_keys]
            v = s["v"][pages, h].double().transpose(1, 2).reshape(-1, D)[:n_keys]
            for g in range(h * G, (h + 1) * G):
                logits = (s["new_q"][lo:hi, g].double() @ k.t()) * s["scale"]
                out[lo:hi, g] = torch.softmax(logits.masked_fill(hidden, -math.inf), 1) @ v
    return out


def exact_adapters(s):
    cu, out = s["cu"].tolist(), s["y"].double()
    for r, a in enumerate(s["ids"].tolist()):
        if a >= 0:
            t = slice(cu[r], cu[r + 1])
            out[t] += float(s["gain"][a]) * (s["b"][a].double() @ (s["a"][a].double() @ s["x"][t].double().t())).t()
    return out
