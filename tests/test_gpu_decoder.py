"""The decoder layer: GPTQ's output and the serving operators used together."""

import pytest
import torch

from post_weight_quantization_03_gb300 import build_lib, decoder, gptq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    gptq.load()
    torch.cuda.init()


@pytest.mark.parametrize("hidden,mlp,heads,kv_heads,dim,bits", [(256, 704, 4, 2, 64, 4), (512, 1000, 4, 1, 128, 3)])
def test_layer_served_in_steps(hidden, mlp, heads, kv_heads, dim, bits):
    weights, (n1, n2) = decoder.random_layer(hidden, mlp, heads, kv_heads, dim)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    calib = torch.randn(4, 256, hidden, generator=g, device="cuda").to(torch.bfloat16)
    layer = decoder.DecoderLayer.quantize(weights, n1, n2, calib, heads, kv_heads, bits)
    # each projection is exactly what the sweep quantized it to: integers times the row's step
    for p in layer.p.values():
        v = p.codes.float()
        assert torch.equal(v, v.round()) and float(v.abs().max()) <= 2 ** bits - 1
    seqs, total = 3, 150
    x = torch.randn(seqs, total, hidden, generator=g, device="cuda").to(torch.bfloat16)
    blocks = -(-total // 64)
    cache = gptq.kv8_cache(seqs * blocks, kv_heads, dim)
    table = torch.randperm(seqs * blocks, generator=g, device="cuda").to(torch.int32).view(seqs, blocks)
    outs, at = [], 0
    for new in (100, 1, 1, 40, 1, 7):
        start = torch.full((seqs,), at, dtype=torch.int32, device="cuda")
        outs.append(layer.step(x[:, at:at + new], cache, table, start, start + new))
        at += new
    assert at == total
    out = torch.cat(outs, 1).float()
    want = decoder.reference(layer.dequantized(), n1, n2, x, heads, kv_heads)
    # the added branches carry e4m3 operands: 2^-4 of an element at most, about 2^-5.3 of the norm for
    # each of the roundings on the way to an output (norm, cache twice, two inner operands), in
    # branches that are no larger than the residual they are added to
    assert float((out - want).norm() / want.norm()) < 5 ** 0.5 * 2 ** -5.3
    assert layer.step(x[:, :0], cache, table, start, start).shape == (seqs, 0, hidden)
