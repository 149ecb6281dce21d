"""Stage many products on the GPU and run them as one decode-token sweep.

A convenience over the C ABI binding: packs each canonical matrix with bq_pack,
copies both planes to the device once, lays the float32 activation vectors end
to end in one device buffer (so one bq_quantize_act_q8 call quantizes them
all: quantization works block by block and every vector length is a multiple
of qa), and builds one bq_sweep plan.  A token is then two launches: the
quantizer over all activations and the sweep -- or one, sweep_fused(), whose
plan (bq_sweep_create_x) quantizes the f32 vectors inside the launch.
"""
from __future__ import annotations

import numpy as np

from . import (Act, BQ_Q1_0, GroupCall, Weights, bq_q1_0_matvec, bq_q2_0_matvec, bq_quantize_act_q8,
               bq_quantize_act_q8_f16, bq_sweep_create, bq_sweep_create_x, bq_token_sweep, BLOCK_LEN)

try:
    from . import (BQ_SILU, bq_adapters_add, bq_embed, bq_gated_q8, bq_kv_append, bq_matmul, bq_matmul_work_bytes,
                   bq_paged_attn, bq_rmsnorm_q8, bq_sample, bq_sample_work_bytes)
except ImportError:  # no torch: what lists the products works without it
    BQ_SILU = 1


class StagedSweep:
    def __init__(self, fmt: int, canon, shapes, x, qa: int = 128, keep_host: bool = True,
                 f16_scale: bool = False):
        """fmt: BQ_Q1_0 / BQ_Q2_0; canon: list of uint8 [rows, cols/QK, 18];
        shapes: list of (name, rows, cols); x: list of float32 [cols] (or one
        concatenated float32 array); f16_scale: quantize with f16-valued
        scales (bq_quantize_act_q8_f16, the q8_0 flavour)."""
        import torch

        self.fmt, self.qa, self.f16_scale = fmt, qa, f16_scale
        self.shapes = [(str(n), int(r), int(c)) for n, r, c in shapes]
        for _, _, cols in self.shapes:
            if cols % qa or cols % BLOCK_LEN[fmt]:
                raise ValueError("every cols must be a multiple of qa and of the block length")
        self.koff = np.concatenate([[0], np.cumsum([c for _, _, c in self.shapes])]).astype(np.int64)
        self.yoff = np.concatenate([[0], np.cumsum([r for _, r, _ in self.shapes])]).astype(np.int64)
        self.ktotal = int(self.koff[-1])
        self.rows_total = int(self.yoff[-1])
        self.weights = []
        self.weight_bytes = 0
        self.canon = [] if keep_host else None
        for c, (_, rows, cols) in zip(canon, self.shapes):
            self.weights.append(Weights.upload(fmt, c, rows, cols))
            self.weight_bytes += c.size
            if keep_host:
                self.canon.append(c)
        xa = np.concatenate([np.asarray(v, np.float32).ravel() for v in x]) if isinstance(x, (list, tuple)) \
            else np.asarray(x, np.float32).ravel()
        if xa.size != self.ktotal:
            raise ValueError("activation length does not match the shapes")
        self.x = xa
        self.xd = torch.from_numpy(xa).to("cuda")
        self.q = torch.empty(self.ktotal, dtype=torch.int8, device="cuda")
        self.d = torch.empty(self.ktotal // qa, dtype=torch.float32, device="cuda")
        self.y = torch.full((self.rows_total,), float("nan"), dtype=torch.float32, device="cuda")
        self.entries = []
        for i, (_, rows, cols) in enumerate(self.shapes):
            k0, k1 = int(self.koff[i]), int(self.koff[i + 1])
            a = Act(self.q[k0:k1], self.d[k0 // qa:k1 // qa], cols, qa, 1)
            self.entries.append((self.weights[i], a, self.y[int(self.yoff[i]):int(self.yoff[i + 1])]))
        self.plan = bq_sweep_create(self.entries)
        self.plan_x = None

    # ------------------------------------------------------------- running
    def quantize(self, stream=None):
        (bq_quantize_act_q8_f16 if self.f16_scale else bq_quantize_act_q8)(self.xd, self.qa, self.q, self.d, stream)

    def sweep(self, stream=None):
        bq_token_sweep(self.plan, stream)

    def run(self, stream=None):
        self.quantize(stream)
        self.sweep(stream)

    def sweep_fused(self, stream=None):
        """The token in one launch from the f32 activations (f32 scales only):
        the same bits in y as run()."""
        if self.f16_scale:
            raise ValueError("the in-launch quantizer writes f32 scales (the q8_0 flavour needs run())")
        if self.plan_x is None:
            ents = [(w, self.xd[int(self.koff[i]):int(self.koff[i + 1])], y) for i, (w, _, y) in enumerate(self.entries)]
            self.plan_x = bq_sweep_create_x(ents, self.qa)
        bq_token_sweep(self.plan_x, stream)

    # ----------------------------------------------------------- accounting
    def sweep_bytes(self) -> int:
        """Algorithmic bytes of one sweep launch: packed weights (18 bytes a
        block) + int8 quants + f32 activation scales read, f32 outputs written."""
        return self.weight_bytes + self.ktotal + 4 * (self.ktotal // self.qa) + 4 * self.rows_total

    def fused_bytes(self) -> int:
        """Algorithmic bytes of one sweep_fused launch: packed weights + the
        f32 activations read, f32 outputs written."""
        return self.weight_bytes + 4 * self.ktotal + 4 * self.rows_total

    def quantize_bytes(self) -> int:
        """Algorithmic bytes of the quantizer launch: f32 in, int8 + f32 scales out."""
        return 4 * self.ktotal + self.ktotal + 4 * (self.ktotal // self.qa)

    def output(self, i: int):
        return self.y[int(self.yoff[i]):int(self.yoff[i + 1])]

    def close(self):
        self.plan.destroy()
        if self.plan_x is not None:
            self.plan_x.destroy()


# ------------------------------------------------------------------ chain
def chain_groups(n_layers: int, lm_head: bool = True):
    """The dependency order of one decode token over the products of
    synth.decode_sweep_shapes(n_layers): per layer {q, k, v}, {o}, {gate, up},
    {down}, then {lm_head}.  Returns [(product indices, source index)]: the
    group's input is the output of product `source` (-1: the token's input
    vector).  The products' own data dependencies (attention, the gated
    activation) are replaced by the nearest output of the right length:
    o takes q's output, gate and up take o's, down takes up's, and the next
    layer (or the LM head) takes down's."""
    groups = []
    prev = -1
    for layer in range(n_layers):
        base = 7 * layer
        q, k, v, o, gate, up, down = range(base, base + 7)
        groups.append(([q, k, v], prev))
        groups.append(([o], q))
        groups.append(([gate, up], o))
        groups.append(([down], up))
        prev = down
    if lm_head:
        groups.append(([7 * n_layers], prev))
    return groups


class StagedChain:
    """One decode token as a chain of dependent launches over the groups of
    chain_groups(), all on one stream.  fused=True: one bq_group_matvec launch
    per group, which quantizes the group's input (the previous group's f32
    output) inside the kernel.  fused=False: a bq_quantize_act_q8 launch into
    an int8 buffer, then a sweep launch over the group's products."""

    def __init__(self, fmt: int, canon, shapes, x0, qa: int = 128, n_layers: int = None, fused: bool = True):
        import torch

        self.fmt, self.qa, self.fused = fmt, qa, fused
        self.shapes = [(str(n), int(r), int(c)) for n, r, c in shapes]
        n_layers = (len(self.shapes) - 1) // 7 if n_layers is None else n_layers
        self.groups = chain_groups(n_layers, lm_head=len(self.shapes) == 7 * n_layers + 1)
        self.yoff = np.concatenate([[0], np.cumsum([r for _, r, _ in self.shapes])]).astype(np.int64)
        self.weights = [Weights.upload(fmt, c, r, k) for c, (_, r, k) in zip(canon, self.shapes)]
        self.weight_bytes = int(sum(c.size for c in canon))
        self.x0 = torch.from_numpy(np.asarray(x0, np.float32).ravel()).to("cuda")
        self.y = torch.full((int(self.yoff[-1]),), float("nan"), dtype=torch.float32, device="cuda")
        self.stages = []
        for prods, src in self.groups:
            cols = self.shapes[prods[0]][2]
            if any(self.shapes[p][2] != cols for p in prods):
                raise ValueError("a group's products must share their input length")
            xin = self.x0 if src < 0 else self.output(src)
            if xin.numel() != cols:
                raise ValueError("a group's input length must match its products")
            if fused:
                self.stages.append(GroupCall([self.weights[p] for p in prods], xin, qa,
                                             [self.output(p) for p in prods]))
            else:
                q = torch.empty(cols, dtype=torch.int8, device="cuda")
                d = torch.empty(cols // qa, dtype=torch.float32, device="cuda")
                a = Act(q, d, cols, qa, 1)
                plan = bq_sweep_create([(self.weights[p], a, self.output(p)) for p in prods])
                self.stages.append((xin, q, d, plan))

    def output(self, i: int):
        return self.y[int(self.yoff[i]):int(self.yoff[i + 1])]

    def run(self, stream=None):
        if self.fused:
            for call in self.stages:
                call.launch(stream)
            return
        for xin, q, d, plan in self.stages:
            bq_quantize_act_q8(xin, self.qa, q, d, stream)
            bq_token_sweep(plan, stream)

    def launches(self) -> int:
        return len(self.stages) * (1 if self.fused else 2)

    def token_bytes(self) -> int:
        """Algorithmic bytes of one token: weights, every group's f32 input
        read once and every output written; unfused, also the int8 quants and
        scales written by the quantizer and read by each product."""
        n = 0
        for prods, _ in self.groups:
            cols = self.shapes[prods[0]][2]
            n += 4 * cols
            if not self.fused:
                n += cols + 4 * (cols // self.qa)                          # quantizer writes
                n += len(prods) * (cols + 4 * (cols // self.qa))           # products read the activation
        return self.weight_bytes + n + 4 * int(self.yoff[-1])

    def close(self):
        if not self.fused:
            for _, _, _, plan in self.stages:
                plan.destroy()
        self.stages = []


# --------------------------------------------------------------- products
class _Products:
    """Products of any number of tokens: 16 columns a call, or one bq_matmul
    from matmul_from tokens on, whose scratch is allocated here."""

    COLUMNS = 16  # activation columns of one product call

    def __init__(self, fmt: int, weights, qa: int, max_tokens: int, matmul_from, device):
        self.fmt, self.qa, self.matmul_from, self.work = fmt, qa, matmul_from, None
        if matmul_from is not None and max_tokens >= matmul_from:
            import torch
            # more tokens need more scratch
            need = max(bq_matmul_work_bytes(w, max_tokens, qa) for w in weights)
            self.work = torch.empty(need, dtype=torch.uint8, device=device)

    def wide(self, tokens: int) -> bool:
        return self.matmul_from is not None and tokens >= self.matmul_from

    def __call__(self, w, act, d, y, tokens: int, stream, res=None):
        """y = W x (+ res, with wide() only) for the first rows of act, d and y."""
        if self.wide(tokens):
            bq_matmul(w, Act(act[:tokens], d[:tokens], w.cols, self.qa, tokens), y[:tokens], res=res, work=self.work, stream=stream)
            return
        call = bq_q1_0_matvec if self.fmt == BQ_Q1_0 else bq_q2_0_matvec
        for c in range(0, tokens, self.COLUMNS):
            e = min(tokens, c + self.COLUMNS)
            call(w, Act(act[c:e], d[c:e], w.cols, self.qa, e - c), y[c:e], stream)


# --------------------------------------------------------------- attention
class StagedAttention:
    """The attention block of a decoder layer between its packed products, for
    the new tokens of any number of requests: residual addition, norm and
    8-bit activation; q, k and v products; their adapters; norm, rotation and
    cache; attention over the cache; quantizer; o product.  One token per
    request is a decode step, whole prompts and chunks of them run the same
    way (the products take up to 16 tokens, the columns of a call, at a time).

    All buffers hold max_tokens rows and are allocated here, on the cache's
    device, so that run() allocates nothing and can be captured into a graph;
    run() of two blocks on two streams need two objects.  In a padded batch
    (rows behind the last request, slot -1) the padding's rows of the output
    are finite where its rows of x are, and mean nothing.

    From matmul_from tokens on (None: never) a product is one bq_matmul instead
    of a call for every 16 tokens: the same numbers to f32 sums, where the
    calls give the same bits however many tokens there are."""

    COLUMNS = _Products.COLUMNS  # activation columns of one product call

    def __init__(self, fmt: int, canon, hidden: int, q_heads: int, cache, norm, freq, max_tokens: int, qa: int = 128,
                 q_norm=None, k_norm=None, adapters=None, eps: float = 1e-6, matmul_from: int | None = None):
        """canon: {"q", "k", "v", "o"} canonical matrices ([q_heads * dim or
        heads * dim, hidden] and [hidden, q_heads * dim]); cache: KVCache;
        norm: float32 [hidden]; adapters: {"q" / "k" / "v" / "o": Adapters}.
        All tensors are on the cache's device."""
        import torch

        self.device = cache.k.device
        self.fmt, self.hidden, self.q_heads, self.cache, self.qa, self.eps = fmt, hidden, q_heads, cache, qa, eps
        nq, nk = q_heads * cache.dim, cache.heads * cache.dim
        self.weights = {}
        for name, rows, cols in (("q", nq, hidden), ("k", nk, hidden), ("v", nk, hidden), ("o", hidden, nq)):
            if cols % qa or cols % BLOCK_LEN[fmt]:
                raise ValueError("every cols must be a multiple of qa and of the block length")
            self.weights[name] = Weights.upload(fmt, canon[name], rows, cols, device=self.device)
        self.norm, self.freq, self.q_norm, self.k_norm = norm, freq, q_norm, k_norm
        self.adapters = adapters or {}

        def rows(n, dtype=torch.float32):
            return torch.empty(max_tokens, n, dtype=dtype, device=self.device)

        self.h, self.normed = rows(hidden), rows(hidden)
        self.act, self.act_d = rows(hidden, torch.int8), rows(hidden // qa)
        self.q, self.k, self.v, self.o = rows(nq), rows(nk), rows(nk), rows(nq)
        # the attention leaves rows behind the last request as they were, and the quantizer takes finite values
        self.o.zero_()
        self.o_act, self.o_d, self.out = rows(nq, torch.int8), rows(nq // qa), rows(hidden)
        self.products = _Products(fmt, self.weights.values(), qa, max_tokens, matmul_from, self.device)

    def _product(self, name: str, act, d, y, tokens: int, stream):
        self.products(self.weights[name], act, d, y, tokens, stream)

    def run(self, x, res, pos, slot, cu, lens, table, max_new: int, max_keys: int, ids=None, work=None,
            adapter_work=None, stream=None):
        """x, res: float32 [tokens, hidden] (res: the residual stream, None for
        the first block); the rest as in bq_kv_append, bq_paged_attn and
        bq_adapters_add.  Returns (out, h): this block's output and the
        residual stream that it is to be added to.  With work and adapter_work
        given, nothing is allocated."""
        import torch

        with torch.cuda.device(self.device):  # whose stream the products take
            return self._run(x, res, pos, slot, cu, lens, table, max_new, max_keys, ids, work, adapter_work, stream)

    def _run(self, x, res, pos, slot, cu, lens, table, max_new, max_keys, ids, work, adapter_work, stream):
        T = x.shape[0]
        cache, dim = self.cache, self.cache.dim
        q, k, v, o, h, out = (b[:T] for b in (self.q, self.k, self.v, self.o, self.h, self.out))
        normed = self.normed[:T] if self.adapters else None
        bq_rmsnorm_q8(x, self.norm, self.eps, self.qa, self.act[:T], self.act_d[:T], res=res, h=h, y=normed, stream=stream)
        for name, y in (("q", q), ("k", k), ("v", v)):
            self._product(name, self.act, self.act_d, y, T, stream)
            if name in self.adapters:
                bq_adapters_add(self.adapters[name], normed, cu, ids, max_new, y, work=adapter_work, stream=stream)
        heads = (T, self.q_heads, dim)
        bq_kv_append(cache, k.view(T, cache.heads, dim), v.view(T, cache.heads, dim), pos, slot, self.freq, q=q.view(heads),
                     q_out=q.view(heads), q_norm=self.q_norm, k_norm=self.k_norm, eps=self.eps, stream=stream)
        bq_paged_attn(cache, q.view(heads), cu, lens, table, dim ** -0.5, max_new, max_keys, o.view(heads), work=work,
                      stream=stream)
        bq_quantize_act_q8(o.view(-1), self.qa, self.o_act[:T].view(-1), self.o_d[:T].view(-1), stream)
        self._product("o", self.o_act, self.o_d, out, T, stream)
        if "o" in self.adapters:
            bq_adapters_add(self.adapters["o"], o, cu, ids, max_new, out, work=adapter_work, stream=stream)
        return out, h


# --------------------------------------------------------------------- mlp
class StagedMLP:
    """The gated MLP of a decoder layer: residual addition, norm and 8-bit
    activation; gate and up products; activation, gate and 8-bit activation;
    down product.  Buffers and graphs as in StagedAttention."""

    def __init__(self, fmt: int, canon, hidden: int, inner: int, norm, max_tokens: int, act: int = BQ_SILU, qa: int = 128,
                 eps: float = 1e-6, matmul_from: int | None = 17, device="cuda"):
        """canon: {"gate", "up", "down"} canonical matrices ([inner, hidden]
        twice, [hidden, inner]); norm: float32 [hidden] on the device."""
        import torch

        self.device = torch.device(device)
        if self.device.index is None:  # the current one now, whichever is current when it runs
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.act_kind, self.qa, self.eps, self.norm = act, qa, eps, norm
        self.weights = {}
        for name, rows, cols in (("gate", inner, hidden), ("up", inner, hidden), ("down", hidden, inner)):
            if cols % qa or cols % BLOCK_LEN[fmt]:
                raise ValueError("every cols must be a multiple of qa and of the block length")
            self.weights[name] = Weights.upload(fmt, canon[name], rows, cols, device=self.device)
        self.products = _Products(fmt, self.weights.values(), qa, max_tokens, matmul_from, self.device)

        def rows(n, dtype=torch.float32):
            return torch.empty(max_tokens, n, dtype=dtype, device=self.device)

        self.h, self.act, self.act_d = rows(hidden), rows(hidden, torch.int8), rows(hidden // qa)
        self.gate, self.up, self.inner_act, self.inner_d = rows(inner), rows(inner), rows(inner, torch.int8), rows(inner // qa)
        self.out = rows(hidden)

    def run(self, x, res, stream=None):
        """x, res: float32 [tokens, hidden], whose sum is the residual stream
        (res None: x alone).  Returns (x, res) of the next block likewise: the
        down product and the residual stream in front of it, or, where the
        product is one bq_matmul, which adds it, their sum and None."""
        import torch

        T = x.shape[0]
        h, out, gate, up = (b[:T] for b in (self.h, self.out, self.gate, self.up))
        with torch.cuda.device(self.device):  # whose stream the products take
            bq_rmsnorm_q8(x, self.norm, self.eps, self.qa, self.act[:T], self.act_d[:T], res=res, h=h, stream=stream)
            self.products(self.weights["gate"], self.act, self.act_d, gate, T, stream)
            self.products(self.weights["up"], self.act, self.act_d, up, T, stream)
            bq_gated_q8(gate, up, self.act_kind, self.qa, self.inner_act[:T], self.inner_d[:T], stream=stream)
            wide = self.products.wide(T)
            self.products(self.weights["down"], self.inner_act, self.inner_d, out, T, stream, res=h if wide else None)
        return (out, None) if wide else (out, h)


# ----------------------------------------------------------------- decoder
class StagedDecoder:
    """A decoder from token ids to the next ids: rows of the token table, layers
    of a StagedAttention and a StagedMLP each, norm and head product of one row
    a request, and the draw.  A step runs any number of new tokens of any number
    of requests (prompts, chunks, one token each); its tokens can be the next
    step's ids where they lie, and a captured step replayed.  Buffers as in
    StagedAttention: steps on two streams at once need two objects, layers
    included, and the next step writes the returned tokens again.

    matmul_from here is of the head alone.  The layers have their own: 17 in
    StagedMLP, but None in StagedAttention, whose q, k, v and o products then
    take a prompt 16 tokens at a time; give it one for long prompts."""

    def __init__(self, table, layers, norm, head, max_tokens: int, max_requests: int, scale: float = 1.0, qa: int = 128,
                 eps: float = 1e-6, matmul_from: int | None = 17):
        """table: token table, Weights or a tensor [vocab, hidden]; layers:
        [(StagedAttention, StagedMLP)]; norm: float32 [hidden]; head: Weights
        [vocab, hidden] (the table's, where both are the same matrix)."""
        import torch

        self.table, self.layers, self.norm, self.head = table, list(layers), norm, head
        self.scale, self.qa, self.eps = scale, qa, eps
        self.device = norm.device
        hidden, vocab, B = head.cols, head.rows, max_requests

        def rows(n, count, dtype=torch.float32):
            return torch.empty(count, n, dtype=dtype, device=self.device)

        self.x = rows(hidden, max_tokens)
        self.last, self.last_res = rows(hidden, B), rows(hidden, B)
        self.act, self.act_d = rows(hidden, B, torch.int8), rows(hidden // qa, B)
        self.logits = rows(vocab, B)
        self.products = _Products(head.fmt, [head], qa, B, matmul_from, self.device)
        self.token = torch.empty(B, dtype=torch.int64, device=self.device)
        self.logprob = torch.empty(B, dtype=torch.float32, device=self.device)
        need = max(bq_sample_work_bytes(b, vocab) for b in range(1, B + 1))
        self.sample_work = torch.empty(need, dtype=torch.uint8, device=self.device)

    def run(self, ids, last, u, pos, slot, cu, lens, table, max_new: int, max_keys: int, adapter_ids=None, work=None,
            adapter_work=None, stream=None, **filters):
        """ids: int64 [tokens]; last: int64 [requests], the row of each request
        that its next token follows from; u: float32 [requests]; filters:
        temperature, top_k, top_p, min_p of bq_sample; the rest as in
        StagedAttention.run.  Returns (token, logprob) of the requests."""
        import torch

        T, B = ids.shape[0], last.shape[0]
        with torch.cuda.device(self.device):  # whose stream the products take
            x, res = self.x[:T], None
            bq_embed(self.table, ids, x, scale=self.scale, stream=stream)
            for attention, mlp in self.layers:
                x, res = attention.run(x, res, pos, slot, cu, lens, table, max_new, max_keys, ids=adapter_ids, work=work,
                                       adapter_work=adapter_work, stream=stream)
                x, res = mlp.run(x, res, stream=stream)
            bq_embed(x, last, self.last[:B], stream=stream)
            if res is not None:
                bq_embed(res, last, self.last_res[:B], stream=stream)
            bq_rmsnorm_q8(self.last[:B], self.norm, self.eps, self.qa, self.act[:B], self.act_d[:B],
                          res=None if res is None else self.last_res[:B], stream=stream)
            self.products(self.head, self.act, self.act_d, self.logits, B, stream)
            bq_sample(self.logits[:B], u, self.token[:B], logprob=self.logprob[:B], work=self.sample_work, stream=stream, **filters)
        return self.token[:B], self.logprob[:B]
