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

Positions are not encoded (a rotation of q and k belongs between the products and the append).

    python -m post_weight_quantization_03_gb300.decoder [--hidden 1024 --mlp 2816 ...]

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
        blocks = -(-tokens // gptq.KV8_BLOCK)
        cache = gptq.kv8_cache(n_seq * blocks, kv_heads, dim, x.device)
        table = torch.arange(n_seq * blocks, dtype=torch.int32, device=x.device).view(n_seq, blocks)
        start = torch.zeros(n_seq, dtype=torch.int32, device=x.device)
        attended = layer._attend(x, cache, table, start, start + tokens)
        take(("o",), attended)
        h = flat + layer.p["o"](*gptq.fp8_quantize(attended), out_dtype=x.dtype)
        take(("gate", "up"), norm(h, norm2))
        take(("down",), layer._gated(*gptq.rmsnorm_fp8(h, norm2, eps=eps)[:3], x.dtype))
        return layer

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
        act = self._gated(codes, exps, rstd, x.dtype)
        return (h + self.p["down"](*gptq.fp8_quantize(act), out_dtype=x.dtype)).view(shape)

    def dequantized(self):
        """The projections' weights in fp32 (W_hat)."""
        return {n: p.codes.float() * p.scale[:, None] for n, p in self.p.items()}


def reference(weights, norm1, norm2, x, heads, kv_heads, eps=1e-6):
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
    return h + act @ weights["down"].float().t()


def random_layer(hidden, mlp, heads, kv_heads, dim, seed=0, device="cuda", dtype=None):
    """Weights and norms of a layer of this shape."""
    torch = gptq._torch()
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    dtype = dtype or torch.bfloat16
    shapes = {"q": (heads * dim, hidden), "k": (kv_heads * dim, hidden), "v": (kv_heads * dim, hidden),
              "o": (hidden, heads * dim), "gate": (mlp, hidden), "up": (mlp, hidden),
              "down": (hidden, mlp)}
    weights = {n: (torch.randn(s, generator=g, device=device) / math.sqrt(s[1])).to(dtype)
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
    a = ap.parse_args(argv)
    weights, (n1, n2) = random_layer(a.hidden, a.mlp, a.heads, a.kv_heads, a.dim)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    calib = torch.randn(8, 512, a.hidden, generator=g, device="cuda").to(torch.bfloat16)
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
        want = reference(w, n1, n2, x, a.heads, a.kv_heads)
        print(f"against fp32 on the {name} weights: relative error "
              f"{float((out - want).norm() / want.norm()):.4f}")


if __name__ == "__main__":
    main()
