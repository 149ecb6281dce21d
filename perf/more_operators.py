"""Cases of the operators that stand around a decoder's layers, for timing them
and for comparing them with their plain forms:

  embed     rows of a token table, packed or dense, scaled (bq_embed): where a
            step begins
  matmul    a packed matrix times the 8-bit activations of any number of
            tokens, with bias, activation, gate and residual in its epilogue
            (bq_matmul): the products of a prompt or of a large batch
  gated     activation, gate and 8-bit activation in one pass (bq_gated_q8):
            between the gate / up products and the down product
  sample    the next token of each row of logits by temperature, top-k, top-p
            and min-p, from given random numbers (bq_sample): where a step ends

With ``own`` false, ``run`` computes the operator from elementary torch
operations in 32 bits (64 where a rounding border or a long sum asks for it);
with ``own`` true it makes the calls of this package.  ``exact`` evaluates the
definition in 64 bits.  Matrix and vocabulary sizes are those of the decode
token this repository benches (4096 and 12288 columns, 151936 tokens) or
generic.  Packed matrices are drawn in the layout that bq_pack writes.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
DEV = "cuda"
LEN = {"q1_0": 128, "q2_0": 64}  # weights of a block: 16 bytes and an f16 scale


def listed():
    return [
        # one decode token's row of the packed table that is also the LM head
        embed("embed_token", 1, 151936, 4096, "q1_0", "f32"),
        # a prompt of an odd number of tokens, ternary table, 16-bit rows
        embed("embed_prompt", 8191, 151936, 4096, "q2_0", "bf16"),
        # a few tokens more than the single products' sixteen columns, plain f32 output
        matmul("matmul_few", 24, 4096, 4096, "q1_0", 128, "f32"),
        # a large decode batch: gate of a gated layer, f32
        matmul("matmul_batch", 96, 12288, 4096, "q2_0", 128, "f32", act="silu"),
        # a prompt in the q8_0 block length, a bias, 16-bit output, ragged rows
        matmul("matmul_q8_0", 1000, 5000, 4096, "q1_0", 32, "bf16", bias=True),
        # a prompt's gate product with activation, times the up product's output
        matmul("matmul_gate", 2049, 12288, 4096, "q1_0", 128, "bf16", act="silu", mul=True),
        # the down product of a long prompt, added to the residual stream
        matmul("matmul_down", 4096, 4096, 12288, "q2_0", 128, "f32", res=True),
        # sixteen tokens between f32 products
        gated("gated_batch", 16, 12288, "f32", 128, "silu"),
        # a prompt in 16 bits, the q8_0 block length and scales, the values kept too
        gated("gated_prompt", 4099, 12288, "bf16", 32, "gelu", y=True, f16_scale=True),
        # one request's next token: latency
        sample("sample_token", 1, 151936, "f32", "mixed"),
        # a serving batch, every request its own filters
        sample("sample_batch", 192, 151936, "f32", "mixed"),
        # temperature only, from 16-bit logits (many equal ones) of a smaller vocabulary, some masked
        sample("sample_plain", 33, 32001, "bf16", "plain"),
    ]


def embed(name, tokens, count, n, table, type):
    return {"name": name, "op": "embed", "tokens": tokens, "count": count, "n": n, "table": table, "type": type}


def matmul(name, tokens, rows, cols, table, qa, type, act="none", bias=False, mul=False, res=False):
    return {"name": name, "op": "matmul", "tokens": tokens, "rows": rows, "cols": cols, "table": table, "qa": qa,
            "type": type, "act": act, "bias": bias, "mul": mul, "res": res}


def gated(name, tokens, n, type, qa, act, y=False, f16_scale=False):
    return {"name": name, "op": "gated", "tokens": tokens, "n": n, "type": type, "qa": qa, "act": act, "y": y,
            "f16_scale": f16_scale}


def sample(name, rows, vocab, type, filters):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "type": type, "filters": filters}


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("embed", "matmul", "matmul", "gated", "sample", "sample"))
    if op == "embed":
        table = rng.choice(("q1_0", "q2_0", "bf16", "f16", "f32"))
        block = LEN.get(table, 8)
        c = embed("", _log(rng, 1, 8191), _log(rng, 100, 151936), block * _log(rng, max(1, 64 // block), 8192 // block),
                  table, rng.choice(("f32", "f16", "bf16")))
        while c["tokens"] * c["n"] > 8191 * 4096:
            c["tokens"] = (c["tokens"] + 1) // 2
        while c["count"] * c["n"] > 151936 * 4096:
            c["count"] = (c["count"] + 1) // 2
    elif op == "matmul":
        qa = rng.choice((32, 64, 128, 128))
        c = matmul("", _log(rng, 1, 5000), _log(rng, 16, 14000), 128 * _log(rng, 1, 96), rng.choice(("q1_0", "q2_0")),
                   qa, rng.choice(("f32", "f16", "bf16")), rng.choice(("none", "none", "silu", "gelu", "relu2")),
                   rng.random() < 0.4, rng.random() < 0.3, rng.random() < 0.4)
        while c["tokens"] * c["rows"] * c["cols"] > 1e11:
            c["tokens"] = (c["tokens"] + 1) // 2
    elif op == "gated":
        qa = rng.choice((32, 64, 128))
        c = gated("", _log(rng, 1, 6000), qa * _log(rng, 1, 16384 // qa), rng.choice(("f32", "f16", "bf16")), qa,
                  rng.choice(("silu", "gelu", "relu2")), True, rng.random() < 0.3)
        c["y"] = c["f16_scale"] or rng.random() < 0.4
        while c["tokens"] * c["n"] > 4099 * 12288:
            c["tokens"] = (c["tokens"] + 1) // 2
    else:
        c = sample("", _log(rng, 1, 400), _log(rng, 16, 262144), rng.choice(("f32", "f16", "bf16")),
                   rng.choice(("mixed", "mixed", "plain")))
        while c["rows"] * c["vocab"] > 192 * 151936:
            c["rows"] = (c["rows"] + 1) // 2
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)

    def normal(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        x = torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, scale, generator=g)
        return x.add_(shift) if shift else x

    def uniform(*shape):
        return torch.empty(shape, device=DEV).uniform_(0.0, 1.0, generator=g)

    def packed(fmt, rows, cols):
        """The two planes of a packed matrix: tiles of 64 rows, 16 bytes a row and block; eight scales a row together."""
        blocks, tiles = cols // LEN[fmt], -(-rows // 64)
        gaps = 7 * ((tiles - 1) // 8) if fmt == "q2_0" else 0
        size = (tiles * blocks + gaps) * 1024
        bits = torch.randint(0, 256 if fmt == "q1_0" else 81, (size,), dtype=torch.uint8, device=DEV, generator=g)
        if fmt == "q2_0":  # four codes of 0, 1 or 2 a byte
            i = torch.arange(81, device=DEV)
            codes = (i % 3) | (i // 3 % 3) << 2 | (i // 9 % 3) << 4 | (i // 27) << 6
            bits = codes.to(torch.uint8)[bits.int()]
        scales = normal(tiles * -(-blocks // 8) * 512, scale=0.02).abs_().half()
        return bits, scales.view(torch.int16)

    if case["op"] == "embed":
        T, count, n = case["tokens"], case["count"], case["n"]
        if case["table"] in LEN:
            s["bits"], s["scales"] = packed(case["table"], count, n)
        else:
            s["dense"] = normal(count, n, dtype=DT[case["table"]], scale=0.02)
        s["ids"] = torch.randint(0, count, (T,), device=DEV, generator=g)
        s["scale"] = math.sqrt(n)
        s["out"] = torch.empty(T, n, dtype=DT[case["type"]], device=DEV)
    elif case["op"] == "matmul":
        T, rows, cols, qa, dt = case["tokens"], case["rows"], case["cols"], case["qa"], DT[case["type"]]
        s["bits"], s["scales"] = packed(case["table"], rows, cols)
        x = normal(T, cols // qa, qa)
        s["d"] = x.abs().amax(2) / 127.0
        s["q"] = (x / s["d"][..., None]).round_().to(torch.int8).view(T, cols)
        s["bias_in"] = normal(rows) if case["bias"] else None
        s["mul_in"] = normal(T, rows, dtype=dt) if case["mul"] else None
        s["res_in"] = normal(T, rows, dtype=dt, scale=2.0) if case["res"] else None
        s["y"] = torch.empty(T, rows, dtype=dt, device=DEV)
    elif case["op"] == "gated":
        T, n, qa, dt = case["tokens"], case["n"], case["qa"], DT[case["type"]]
        s["gate"], s["up"] = normal(T, n, dtype=dt, scale=2.0), normal(T, n, dtype=dt)
        s["q"] = torch.empty(T, n, dtype=torch.int8, device=DEV)
        s["d"] = torch.empty(T, n // qa, device=DEV)
        s["y_out"] = torch.empty(T, n, dtype=dt, device=DEV) if case["y"] else None
    else:
        B, V, mixed = case["rows"], case["vocab"], case["filters"] == "mixed"
        x = normal(B, V, scale=2.0)
        # a few tokens stand out, as in a model's logits
        few = torch.randint(0, V, (B, 40), device=DEV, generator=g)
        x.scatter_add_(1, few, 6.0 + 3.0 * normal(B, 40))
        if not mixed:
            x.masked_fill_(uniform(B, V) < 0.1, -math.inf)
        s["logits"] = x.to(DT[case["type"]])
        s["u"] = uniform(B)
        s["temperature"] = 0.4 + uniform(B)
        if mixed:  # each filter is off in some rows; one row in eight is greedy
            s["temperature"] *= uniform(B) > 0.125
            s["top_k"] = (4.0 ** (1.0 + 5.0 * uniform(B))).int() * (uniform(B) < 0.6)
            s["top_p"] = torch.where(uniform(B) < 0.6, 0.5 + 0.49 * uniform(B), 1.0)
            s["min_p"] = torch.where(uniform(B) < 0.3, 0.2 * uniform(B), 0.0)
        s["token"] = torch.empty(B, dtype=torch.int64, device=DEV)
        s["logprob"] = torch.empty(B, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"embed": run_embed, "matmul": run_matmul, "gated": run_gated, "sample": run_sample}[s["op"]](s)


def unpacked(s, rows, cols):
    """Codes (+1 / -1, or code - 1) and f32 scales of a packed matrix: [rows, blocks, weights], [rows, blocks]."""
    length = LEN[s["table"]]
    blocks, tiles = cols // length, -(-rows // 64)
    t = torch.arange(tiles, device=DEV)
    at = t * blocks + (7 * (t // 8) if s["table"] == "q2_0" else 0)
    at = at[:, None] + torch.arange(blocks, device=DEV)[None, :]
    words = s["bits"].view(torch.int32).view(-1, 64, 4)[at].permute(0, 2, 1, 3).reshape(tiles * 64, blocks, 4)[:rows]
    # word of weights k = 0, 1, ...: turned left by two bits
    each = length // 4
    shift = (torch.arange(each, device=DEV, dtype=torch.int32) * (32 // each) + 2) % 32
    code = (words[..., None] >> shift) & (1 if length == 128 else 3)
    code = (2 * code - 1 if length == 128 else code - 1).reshape(rows, blocks, length)
    scale = s["scales"].view(torch.float16).view(tiles, -1, 64, 8).permute(0, 2, 1, 3).reshape(tiles * 64, -1)
    return code, scale[:rows, :blocks].float()


def activated(x, act):
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    if act == "relu2":
        return torch.where(x > 0, x, torch.zeros_like(x)).square()
    return x


def run_embed(s):
    if own:
        import ternary_quantized_gemv_amd as bq
        table = s["dense"] if "dense" in s else bq.Weights(
            bq.BQ_Q1_0 if s["table"] == "q1_0" else bq.BQ_Q2_0, s["count"], s["n"], s["bits"], s["scales"])
        bq.bq_embed(table, s["ids"], s["out"], scale=s["scale"])
        return s["out"]
    if "dense" in s:
        return (s["dense"][s["ids"]].float() * s["scale"]).to(s["out"].dtype)
    # the rows' words and scales first: the table is far larger than what is read of it
    length = LEN[s["table"]]
    blocks = s["n"] // length
    tile, lane = s["ids"] // 64, s["ids"] % 64
    at = tile * blocks + (7 * (tile // 8) if s["table"] == "q2_0" else 0)
    at = at[:, None] + torch.arange(blocks, device=DEV)[None, :]
    words = s["bits"].view(torch.int32).view(-1, 64, 4)[at, lane[:, None]]
    each = length // 4
    shift = (torch.arange(each, device=DEV, dtype=torch.int32) * (32 // each) + 2) % 32
    code = (words[..., None] >> shift) & (1 if length == 128 else 3)
    code = (2 * code - 1 if length == 128 else code - 1).reshape(-1, blocks, length)
    d = s["scales"].view(torch.float16).view(-1, -(-blocks // 8), 64, 8)[tile, :, lane].reshape(-1, -(-blocks // 8) * 8)
    values = code.float() * d[:, :blocks, None].float()
    return (values.reshape(-1, s["n"]) * s["scale"]).to(s["out"].dtype)


def run_matmul(s):
    if own:
        import ternary_quantized_gemv_amd as bq
        w = bq.Weights(bq.BQ_Q1_0 if s["table"] == "q1_0" else bq.BQ_Q2_0, s["rows"], s["cols"], s["bits"], s["scales"])
        acts = {"none": bq.BQ_NONE, "silu": bq.BQ_SILU, "gelu": bq.BQ_GELU, "relu2": bq.BQ_RELU2}
        bq.bq_matmul(w, bq.Act(s["q"], s["d"], s["cols"], s["qa"], s["tokens"]), s["y"], bias=s["bias_in"],
                     act=acts[s["act"]], mul=s["mul_in"], res=s["res_in"])
        return s["y"]
    code, scale = unpacked(s, s["rows"], s["cols"])
    w = (code.float() * scale[..., None]).reshape(s["rows"], s["cols"])
    x = (s["q"].float().view(s["tokens"], -1, s["qa"]) * s["d"][..., None]).view(s["tokens"], s["cols"])
    y = torch.matmul(x, w.t())
    if s["bias"]:
        y = y + s["bias_in"]
    y = activated(y, s["act"])
    if s["mul"]:
        y = y * s["mul_in"].float()
    if s["res"]:
        y = y + s["res_in"].float()
    return y.to(s["y"].dtype)


def run_gated(s):
    T, n, qa = s["tokens"], s["n"], s["qa"]
    if own:
        import ternary_quantized_gemv_amd as bq
        acts = {"silu": bq.BQ_SILU, "gelu": bq.BQ_GELU, "relu2": bq.BQ_RELU2}
        bq.bq_gated_q8(s["gate"], s["up"], acts[s["act"]], qa, s["q"], s["d"], y=s["y_out"], f16_scale=s["f16_scale"])
        q, d, y = s["q"], s["d"], s["y_out"]
    else:
        v = (activated(s["gate"].double(), s["act"]) * s["up"].double()).float()  # next to a border: 64 bits
        blocks = v.view(T, n // qa, qa)
        d = blocks.abs().amax(2) / 127.0
        if s["f16_scale"]:
            d = d.half().float()
        ratio = blocks / torch.where(d == 0, torch.ones_like(d), d)[..., None]
        q = torch.where(ratio < 0, -1.0, 1.0) * torch.floor(ratio.abs().double() + 0.5).float()  # ties away from zero
        q = torch.where(d[..., None] == 0, torch.zeros_like(q), q.clamp_(-127, 127)).view(T, n)
        y = v.to(s["gate"].dtype) if s["y"] else None
    # the quants as the values that they stand for
    out = {"d": d, "values": (q.view(T, n // qa, qa) * d.view(T, n // qa, 1)).view(T, n)}
    if s["y"]:
        out["y"] = y
    return out


def run_sample(s):
    mixed = s["filters"] == "mixed"
    if own:
        import ternary_quantized_gemv_amd as bq
        filters = {"top_k": s["top_k"], "top_p": s["top_p"], "min_p": s["min_p"]} if mixed else {}
        bq.bq_sample(s["logits"], s["u"], s["token"], logprob=s["logprob"], temperature=s["temperature"], **filters)
        return {"token": s["token"], "logprob": s["logprob"]}
    # sums next to a border: 64 bits
    V = s["vocab"]
    x, order = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
    x, t = x.double(), s["temperature"].double()[:, None]
    greedy = t <= 0
    w = torch.exp((x - x[:, :1]) / torch.where(greedy, torch.ones_like(t), t))
    w = torch.where(greedy, (x == x[:, :1]).double(), w)
    sums = torch.cumsum(w, 1)
    mass = sums[:, -1:]
    if mixed:
        k = s["top_k"].long()[:, None]
        mass = sums.gather(1, torch.where(k > 0, k, V).clamp(max=V) - 1)
        p = s["top_p"].double()[:, None]
        nucleus = sums.gather(1, torch.searchsorted(sums, p * mass).clamp(max=V - 1))
        top = torch.where(w >= s["min_p"].double()[:, None], w, torch.zeros_like(w)).sum(1, keepdim=True)
        mass = torch.minimum(torch.where(p < 1, torch.minimum(nucleus, mass), mass), top)
    at = torch.searchsorted(sums, s["u"].double()[:, None] * mass, right=True).clamp(max=V - 1)
    at = torch.where(greedy, torch.zeros_like(at), at)
    logprob = torch.log(w.gather(1, at) / sums[:, -1:])
    return {"token": order.gather(1, at)[:, 0], "logprob": torch.where(greedy, 0.0, logprob)[:, 0].float()}


# ------------------------------------------------------------------ work
def row_bytes(table, n):
    return n // LEN[table] * 18 if table in LEN else n * SIZE[table]


def work(case):
    if case["op"] == "embed":
        T, n = case["tokens"], case["n"]
        # the rows that are read, at most the table's; ids; outputs
        moved = min(T, case["count"]) * row_bytes(case["table"], n) + 8 * T + T * n * SIZE[case["type"]]
        return {"bytes": moved, "flops": 2 * T * n}
    if case["op"] == "matmul":
        T, rows, cols = case["tokens"], case["rows"], case["cols"]
        moved = rows * row_bytes(case["table"], cols) + T * cols + 4 * T * (cols // case["qa"])
        moved += T * rows * SIZE[case["type"]] * (1 + case["mul"] + case["res"]) + 4 * rows * case["bias"]
        return {"bytes": moved, "flops": 2 * T * rows * cols}
    if case["op"] == "gated":
        T, n = case["tokens"], case["n"]
        moved = T * n * (SIZE[case["type"]] * (2 + case["y"]) + 1) + 4 * T * (n // case["qa"])
        return {"bytes": moved, "flops": 10 * T * n}
    B, V = case["rows"], case["vocab"]
    return {"bytes": B * V * SIZE[case["type"]] + B * (8 + 4 + 4 + 4 + 12 * (case["filters"] == "mixed")), "flops": 4 * B * V}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": exact_embed, "matmul": exact_matmul, "gated": exact_gated, "sample": exact_sample}[s["op"]](s)


def signed(payload, table):
    """Weights in 64 bits from blocks of 16 bytes ([..., 16]), byte by byte: byte b holds the weights whose bits stand
    two places to the left of where they are numbered, around the end of each 32-bit word."""
    wide = 128 // LEN[table]
    out = torch.empty(*payload.shape[:-1], LEN[table], dtype=torch.float64, device=DEV)
    for b in range(16):
        for part in range(8 // wide):
            k = (8 * (b % 4) + wide * part - 2) % 32 // wide + 32 // wide * (b // 4)
            c = payload[..., b] // 2 ** (wide * part) % 2 ** wide
            out[..., k] = c * 2.0 - 1.0 if wide == 1 else c - 1.0
    return out


def matrix(s, rows, cols):
    """The packed matrix in 64 bits, tile by tile."""
    length = LEN[s["table"]]
    blocks, tiles, eights = cols // length, [], -(-(cols // length) // 8)
    for t in range(-(-rows // 64)):
        first = t * blocks + (t // 8 * 7 if length == 64 else 0)
        w = signed(s["bits"].view(-1, 64, 16)[first:first + blocks].transpose(0, 1), s["table"])
        d = s["scales"].view(torch.float16).view(-1, 64, 8)[t * eights:(t + 1) * eights].double()
        tiles.append((w * d.transpose(0, 1).flatten(1)[:, :blocks, None]).flatten(1))
    return torch.cat(tiles)[:rows]


def smooth(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return x * torch.sigmoid(math.sqrt(8.0 / math.pi) * (x + 0.044715 * x ** 3))
    return x.clamp(min=0.0) ** 2 if act == "relu2" else x


def exact_embed(s):
    if "dense" in s:
        return torch.index_select(s["dense"].double(), 0, s["ids"]) * s["scale"]
    blocks, rows = s["n"] // LEN[s["table"]], []
    for tile, lane in zip((s["ids"] // 64).tolist(), (s["ids"] % 64).tolist()):
        first, eights = tile * blocks + (tile // 8 * 7 if s["table"] == "q2_0" else 0), -(-blocks // 8)
        rows.append((s["bits"].view(-1, 64, 16)[first:first + blocks, lane],
                     s["scales"].view(torch.float16).view(-1, 64, 8)[tile * eights:(tile + 1) * eights, lane].flatten()))
    payload, d = (torch.stack(x) for x in zip(*rows))
    return (signed(payload, s["table"]) * d[:, :blocks, None].double()).flatten(1) * s["scale"]


def exact_matmul(s):
    w = matrix(s, s["rows"], s["cols"])
    y = (s["q"].double().unflatten(1, (-1, s["qa"])) * s["d"].double().unsqueeze(2)).flatten(1) @ w.t()
    y = smooth(y + s["bias_in"].double() if s["bias"] else y, s["act"])
    y = y * s["mul_in"].double() if s["mul"] else y
    return y + s["res_in"].double() if s["res"] else y


def exact_gated(s):
    """The quants have no value in 64 bits, nor have scales rounded to f16."""
    v = smooth(s["gate"].double(), s["act"]) * s["up"].double()
    scale = v.abs().unflatten(1, (-1, s["qa"])).max(2).values / 127
    out = {"d": None if s["f16_scale"] else scale, "values": None}
    if s["y"]:
        out["y"] = v
    return out


def exact_sample(s):
    """Row by row: the kept tokens as a list, then the draw."""
    tokens, logprobs = [], []
    for r in range(s["rows"]):
        x, t = s["logits"][r].double(), float(s["temperature"][r])
        if t <= 0:
            tokens.append(int((x == x.max()).nonzero()[0]))
            logprobs.append(0.0)
            continue
        p = torch.softmax(x / t, 0)
        ranked = torch.argsort(x, descending=True, stable=True)
        kept = ranked
        if s["filters"] == "mixed":
            k, top_p = int(s["top_k"][r]), float(s["top_p"][r])
            kept = ranked[:k] if k > 0 else ranked
            if top_p < 1:
                share = torch.cumsum(p[kept], 0) / p[kept].sum()
                kept = kept[:int((share < top_p).sum()) + 1]
            kept = kept[p[kept] >= float(s["min_p"][r]) * p.max()]
        share = torch.cumsum(p[kept], 0)
        tokens.append(int(kept[int((share <= float(s["u"][r]) * share[-1]).sum())]))
        logprobs.append(float(torch.log_softmax(x / t, 0)[tokens[-1]]))
    return {"token": torch.tensor(tokens, device=DEV), "logprob": torch.tensor(logprobs, dtype=torch.float64, device=DEV)}
