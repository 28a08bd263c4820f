"""A decoder layer served from its quantized weights: GPTQ's output and the 8-bit serving
operators used together.

``DecoderLayer.quantize`` runs the library's calibration path on the layer's inputs (Hessian,
factor, sweep at 2 to 4 bits; the inputs of the later projections are the quantized layer's own)
and keeps each projection as the e4m3 integers ``code - zero`` with GPTQ's step as the row scale,
which is exactly its ``W_hat``.  ``DecoderLayer.step`` then runs new tokens of a batch of
sequences through it:

    norm (8-bit out) -> q, k, v products -> append to the 8-bit cache -> attention over it
      -> 8-bit -> output product -> norm with the residual's addition (8-bit out)
      -> gate and up products -> SiLU(gate) * up -> 8-bit -> down product -> residual

``ExpertsLayer`` has experts in place of the one feed-forward block, each quantized on the tokens that
are routed to it, and a dense block that all tokens go through:

    norm -> router -> routing -> gate and up products of each token's experts, SiLU(gate) * up (8-bit out)
      -> their down products -> weighted sum + the dense block (gated product with 8-bit out, down product
      with the residual's addition)

Positions are not encoded (a rotation of q and k belongs between the products and the append).

    python -m post_weight_quantization_03_gb300.decoder [--hidden 1024 --mlp 2816 ...]
    python -m post_weight_quantization_03_gb300.decoder --experts 8 --top-k 2 [--mlp 704 ...]

quantizes a layer with random weights, serves a prompt and a few tokens, and compares the outputs
with the same layer in fp32 torch on the unquantized and on the quantized weights.
"""

from __future__ import annotations

import argparse
import math

from . import gptq


class Projection:
    """One linear layer as the block-scaled product takes it."""

    def __init__(self, codes, exps, scale):
        self.codes, self.exps, self.scale = codes, exps, scale

    @classmethod
    def from_gptq(cls, qpacked, scale, zero, d_in, bits):
        codes, exps = gptq.fp8_from_codes(qpacked, zero, d_in, bits)
        return cls(codes, exps, scale)

    def __call__(self, x, x_exps, x_scale=None, out_dtype=None):
        return gptq.fp8_matmul(x, x_exps, self.codes, self.exps, x_scale, self.scale, out_dtype)


class DecoderLayer:
    """Attention and a gated feed-forward block in 8-bit operands, with their norms."""

    NAMES = ("q", "k", "v", "o", "gate", "up", "down")

    def __init__(self, projections, norm1, norm2, heads, kv_heads, dim, eps=1e-6):
        self.p = projections
        self.norm1, self.norm2 = norm1, norm2
        self.heads, self.kv_heads, self.dim, self.eps = heads, kv_heads, dim, eps

    @classmethod
    def quantize(cls, weights, norm1, norm2, x, heads, kv_heads, bits=4, eps=1e-6, damp=0.01):
        """From the weights of the seven projections (a dict by NAMES, ``[d_out, d_in]``) and the
        calibration inputs ``x [seqs, tokens, hidden]`` (float16 or bfloat16)."""
        torch = gptq._torch()
        dim = weights["q"].shape[0] // heads
        layer = cls({}, norm1, norm2, heads, kv_heads, dim, eps)
        n_seq, tokens, hidden = x.shape

        def take(names, inputs):
            U, dead, _ = gptq.prepare(gptq.hessian(inputs), damp)
            outs = gptq.quantize_shared([weights[n] for n in names], U, bits, dead_mask=dead)
            for name, (qp, scale, zero, _) in zip(names, outs):
                layer.p[name] = Projection.from_gptq(qp, scale, zero, inputs.shape[1], bits)

        def norm(h, w):
            h = h.float()
            return (h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * w.float()).to(x.dtype)

        flat = x.reshape(-1, hidden)
        take(("q", "k", "v"), norm(flat, norm1))
        h = layer._calibrated_attention(take, x)
        take(("gate", "up"), norm(h, norm2))
        take(("down",), layer._gated(*gptq.rmsnorm_fp8(h, norm2, eps=eps)[:3], x.dtype))
        return layer

    def _calibrated_attention(self, take, x):
        """Quantizes the output projection on the quantized attention's outputs; the hidden states
        after it."""
        torch = gptq._torch()
        n_seq, tokens, hidden = x.shape
        blocks = -(-tokens // gptq.KV8_BLOCK)
        cache = gptq.kv8_cache(n_seq * blocks, self.kv_heads, self.dim, x.device)
        table = torch.arange(n_seq * blocks, dtype=torch.int32, device=x.device).view(n_seq, blocks)
        start = torch.zeros(n_seq, dtype=torch.int32, device=x.device)
        attended = self._attend(x, cache, table, start, start + tokens)
        take(("o",), attended)
        return x.reshape(-1, hidden) + self.p["o"](*gptq.fp8_quantize(attended), out_dtype=x.dtype)

    def _attend(self, x, cache, table, start, lengths):
        n_seq, new, hidden = x.shape
        codes, exps, rstd, _ = gptq.rmsnorm_fp8(x.reshape(-1, hidden), self.norm1, eps=self.eps)
        q, k, v = (self.p[n](codes, exps, rstd, x.dtype).view(n_seq, new, n_heads, self.dim)
                   for n, n_heads in (("q", self.heads), ("k", self.kv_heads), ("v", self.kv_heads)))
        gptq.kv8_append(cache, k, v, table, start)
        return gptq.kv8_attention(q, cache, table, lengths).view(n_seq * new, self.heads * self.dim)

    def _gated(self, codes, exps, rstd, dtype):
        torch = gptq._torch()
        gate, up = (self.p[n](codes, exps, rstd, dtype) for n in ("gate", "up"))
        return torch.nn.functional.silu(gate) * up

    def step(self, x, cache, table, start, lengths):
        """New tokens ``x [seqs, new, hidden]`` at ``start`` of each sequence; ``lengths`` is
        ``start + new``.  Returns the layer's outputs, with the cache brought up to date."""
        shape = x.shape
        flat = x.reshape(-1, shape[-1])
        o = self.p["o"](*gptq.fp8_quantize(self._attend(x, cache, table, start, lengths)),
                        out_dtype=x.dtype)
        codes, exps, rstd, h = gptq.rmsnorm_fp8(o, self.norm2, residual=flat, eps=self.eps)
        return self._feed_forward(codes, exps, rstd, h).view(shape)

    def _feed_forward(self, codes, exps, rstd, h):
        act = self._gated(codes, exps, rstd, h.dtype)
        return h + self.p["down"](*gptq.fp8_quantize(act), out_dtype=h.dtype)

    def dequantized(self):
        """The projections' weights in fp32 (W_hat)."""
        return {n: p.codes.float() * p.scale[:, None] for n, p in self.p.items()}


class ExpertsLayer(DecoderLayer):
    """A decoder layer whose feed-forward block is a set of experts beside a dense block.

    ``weights`` has, beside the dense layer's, ``router [experts, hidden]``, ``experts_gate`` and
    ``experts_up [experts, d, hidden]`` and ``experts_down [experts, hidden, d]``.  ``routing``: what
    ``moe_route`` takes beside the logits (top_k, scores, groups, ...)."""

    def __init__(self, *args, router=None, routing=None, **kw):
        super().__init__(*args, **kw)
        self.router, self.routing, self.experts = router, dict(routing or {"top_k": 1}), {}

    @classmethod
    def quantize(cls, weights, norm1, norm2, x, heads, kv_heads, bits=4, eps=1e-6, damp=0.01, routing=None):
        torch = gptq._torch()
        dim = weights["q"].shape[0] // heads
        layer = cls({}, norm1, norm2, heads, kv_heads, dim, eps, router=weights["router"].float(), routing=routing)

        def projections(named, inputs):
            U, dead, _ = gptq.prepare(gptq.hessian(inputs), damp)
            outs = gptq.quantize_shared([w for _, w in named], U, bits, dead_mask=dead)
            return {name: Projection.from_gptq(qp, scale, zero, inputs.shape[1], bits)
                    for (name, _), (qp, scale, zero, _) in zip(named, outs)}

        def take(names, inputs):
            layer.p.update(projections([(n, weights[n]) for n in names], inputs))

        def norm(h, w):
            h = h.float()
            return (h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * w.float()).to(x.dtype)

        take(("q", "k", "v"), norm(x.reshape(-1, x.shape[-1]), norm1))
        h = layer._calibrated_attention(take, x)
        normed = norm(h, norm2)
        take(("gate", "up"), normed)
        codes, exps, rstd, _ = gptq.rmsnorm_fp8(h, norm2, eps=eps)
        inner = gptq.fp8_gated(codes, exps, layer._of("gate"), layer._of("up"), rstd)
        take(("down",), _values(*inner).to(x.dtype))
        # each expert on the tokens that go to it, or on all where none does
        _, _, offsets, order = layer._route(h, rstd)
        begins, top_k = offsets.tolist(), layer.routing["top_k"]
        experts = range(len(begins) - 1)
        found = {n: [] for n in ("gate", "up", "down")}
        for e in experts:
            rows = order[begins[e]:begins[e + 1]].long() // top_k
            got = projections([(n, weights["experts_" + n][e]) for n in ("gate", "up")],
                              normed[rows] if len(rows) else normed)
            for n, p in got.items():
                found[n].append(p)
        layer.experts = {n: _stacked(found[n]) for n in ("gate", "up")}
        inner = _values(*gptq.fp8_experts_gated(codes, exps, layer.experts["gate"], layer.experts["up"], offsets,
                                                order, top_k, rstd)).to(x.dtype)
        for e in experts:
            rows = inner[begins[e]:begins[e + 1]]
            found["down"] += projections([("down", weights["experts_down"][e])],
                                         rows if len(rows) else inner[:begins[-1]]).values()
        layer.experts["down"] = _stacked(found["down"])
        return layer

    def _of(self, name):
        p = self.p[name]
        return p.codes, p.exps, p.scale

    def _route(self, h, rstd):
        """Routing by the normed hidden states."""
        logits = (h.float() * self.norm2.float()) @ self.router.t() * rstd[:, None]
        return gptq.moe_route(logits, **self.routing)

    def _feed_forward(self, codes, exps, rstd, h):
        _, weights, offsets, order = self._route(h, rstd)
        inner = gptq.fp8_gated(codes, exps, self._of("gate"), self._of("up"), rstd)
        dense = gptq.fp8_linear(*inner, *self._of("down")[:2], w_scale=self.p["down"].scale, residual=h,
                                out_dtype=h.dtype)
        inner = gptq.fp8_experts_gated(codes, exps, self.experts["gate"], self.experts["up"], offsets, order,
                                       self.routing["top_k"], rstd)
        down, down_exps, scale = self.experts["down"]
        y = gptq.fp8_experts(*inner, down, down_exps, offsets, order, scale, out_dtype=h.dtype)
        return gptq.moe_combine(y, weights, dense, out=dense)

    def dequantized(self):
        out = super().dequantized()
        out["router"] = self.router
        for n, (codes, _, scale) in self.experts.items():
            out["experts_" + n] = codes.float() * scale[..., None]
        return out


def _values(codes, exps):
    """The numbers that codes and exponents by 1 x 128 blocks stand for, in fp32."""
    torch = gptq._torch()
    scale = torch.ldexp(torch.ones((), device=codes.device), exps.int() - 127)
    return codes.float() * scale.repeat_interleave(gptq.FP8_BLOCK, 1)[:, :codes.shape[1]]


def _stacked(projections):
    """``(codes, exps, scale)`` of several experts' matrices of one shape, one after another."""
    torch = gptq._torch()

    def stack(ts, step):
        rows, d = ts[0].shape
        out = torch.zeros(len(ts), rows, -(-d // step) * step, dtype=torch.uint8, device=ts[0].device)[:, :, :d]
        for o, t in zip(out, ts):
            o.copy_(t.view(torch.uint8))
        return out

    codes = stack([p.codes for p in projections], 16).view(torch.float8_e4m3fn)
    return codes, stack([p.exps for p in projections], 4), torch.stack([p.scale for p in projections])


def experts_reference(weights, routing, g):
    """The experts' part of a layer for normed hidden states ``g [..., hidden]`` in fp32 torch, every
    expert for every token."""
    torch = gptq._torch()
    flat = g.reshape(-1, g.shape[-1])
    logits = flat @ weights["router"].float().t()
    ids, w, _, _ = gptq.moe_route(logits, **routing)
    mix = torch.zeros_like(logits).scatter_(1, ids.long(), w)
    act = torch.nn.functional.silu(torch.einsum("td,end->ten", flat, weights["experts_gate"].float())) \
        * torch.einsum("td,end->ten", flat, weights["experts_up"].float())
    return torch.einsum("ten,edn,te->td", act, weights["experts_down"].float(), mix).view(g.shape)


def reference(weights, norm1, norm2, x, heads, kv_heads, eps=1e-6, routing=None):
    """The layer in fp32 torch over whole sequences ``x [seqs, tokens, hidden]``."""
    torch = gptq._torch()
    n_seq, tokens, hidden = x.shape
    dim = weights["q"].shape[0] // heads

    def norm(h, w):
        return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * w.float()

    x = x.float()
    h = norm(x, norm1)
    q, k, v = ((h @ weights[n].float().t()).view(n_seq, tokens, -1, dim).transpose(1, 2)
               for n in ("q", "k", "v"))
    k, v = (t.repeat_interleave(heads // kv_heads, 1) for t in (k, v))
    s = q @ k.transpose(2, 3) * dim ** -0.5
    s = s.masked_fill(torch.ones(tokens, tokens, dtype=torch.bool, device=x.device).triu(1), -math.inf)
    a = (torch.softmax(s, -1) @ v).transpose(1, 2).reshape(n_seq, tokens, -1)
    h = x + a @ weights["o"].float().t()
    g = norm(h, norm2)
    act = torch.nn.functional.silu(g @ weights["gate"].float().t()) * (g @ weights["up"].float().t())
    out = h + act @ weights["down"].float().t()
    return out if routing is None else out + experts_reference(weights, routing, g)


def random_layer(hidden, mlp, heads, kv_heads, dim, seed=0, device="cuda", dtype=None, experts=0):
    """Weights and norms of a layer of this shape; ``experts``: of so many experts beside the dense
    block, all ``mlp`` wide."""
    torch = gptq._torch()
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    dtype = dtype or torch.bfloat16
    shapes = {"q": (heads * dim, hidden), "k": (kv_heads * dim, hidden), "v": (kv_heads * dim, hidden),
              "o": (hidden, heads * dim), "gate": (mlp, hidden), "up": (mlp, hidden),
              "down": (hidden, mlp)}
    if experts:
        shapes |= {"router": (experts, hidden), "experts_gate": (experts, mlp, hidden),
                   "experts_up": (experts, mlp, hidden), "experts_down": (experts, hidden, mlp)}
    weights = {n: (torch.randn(s, generator=g, device=device) / math.sqrt(s[-1])).to(dtype)
               for n, s in shapes.items()}
    norms = [(1 + 0.1 * torch.randn(hidden, generator=g, device=device)).to(dtype) for _ in range(2)]
    return weights, norms


def main(argv=None):
    torch = gptq._torch()
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--mlp", type=int, default=2816)
    ap.add_argument("--heads", type=int, default=8)
    ap.add_argument("--kv-heads", type=int, default=2)
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--bits", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=200)
    ap.add_argument("--tokens", type=int, default=20)
    ap.add_argument("--experts", type=int, default=0, help="experts beside the dense block (0: none)")
    ap.add_argument("--top-k", type=int, default=2, help="experts of a token")
    a = ap.parse_args(argv)
    weights, (n1, n2) = random_layer(a.hidden, a.mlp, a.heads, a.kv_heads, a.dim, experts=a.experts)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    calib = torch.randn(8, 512, a.hidden, generator=g, device="cuda").to(torch.bfloat16)
    routing = {"top_k": a.top_k} if a.experts else None
    if a.experts:
        layer = ExpertsLayer.quantize(weights, n1, n2, calib, a.heads, a.kv_heads, a.bits, routing=routing)
    else:
        layer = DecoderLayer.quantize(weights, n1, n2, calib, a.heads, a.kv_heads, a.bits)
    seqs, total = 2, a.prompt + a.tokens
    x = torch.randn(seqs, total, a.hidden, generator=g, device="cuda").to(torch.bfloat16)
    blocks = -(-total // gptq.KV8_BLOCK)
    cache = gptq.kv8_cache(seqs * blocks, a.kv_heads, a.dim)
    table = torch.arange(seqs * blocks, dtype=torch.int32, device="cuda").view(seqs, blocks)
    outs, at = [], 0
    for new in [a.prompt] + [1] * a.tokens:
        start = torch.full((seqs,), at, dtype=torch.int32, device="cuda")
        outs.append(layer.step(x[:, at:at + new], cache, table, start, start + new))
        at += new
    out = torch.cat(outs, 1).float()
    gptq.serving_status()
    for name, w in (("quantized", layer.dequantized()), ("original", weights)):
        want = reference(w, n1, n2, x, a.heads, a.kv_heads, routing=routing)
        print(f"against fp32 on the {name} weights: relative error "
              f"{float((out - want).norm() / want.norm()):.4f}")


if __name__ == "__main__":
    main()
