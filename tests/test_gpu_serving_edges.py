"""GPU tests of the 8-bit serving operators where their work meets: items that follow one another
in a CTA, softmaxes with a dominant token, magnitudes at the ends of a type's range.  Tolerances
are those of the operators' parity tests."""

import numpy as np
import pytest
import torch

from oracle import serving_oracle as SO
from post_weight_quantization_03_gb300 import gptq
from tests.test_gpu_serving import (DEV, DT, ULP, _cache, _check_attention, _dev_cache, _i32, _lib, _np,  # noqa: F401
                                    _randn, _table)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------
# Prompts: many short items, finished whole one after another by the same CTA
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("seqs,new,kv,group,longest", [(300, 64, 2, 4, 200), (500, 20, 2, 4, 140), (160, 100, 4, 1, 700)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("aligned", [True, False])
def test_prompts_of_many_short_items(seqs, new, kv, group, longest, d, dtype, aligned):
    # a tile's four warps leave an item one by one: what one of them writes or reads of the last
    # item must not meet what another has stored of the next
    rng = np.random.default_rng(seqs)
    lengths = rng.integers(new, longest + 1, seqs)
    n_blocks, mb = 64, -(-longest // 64)
    cache, table = _cache(seqs, n_blocks, kv, d), rng.integers(0, n_blocks, (seqs, mb)).astype(np.int32)
    dev, tab, length = _dev_cache(cache), _i32(table), _i32(lengths)
    heads = kv * group
    q = _randn(9, seqs, new, heads, d, dtype=dtype).to(DEV)
    pad = 8 if aligned else 1
    results = []
    for _ in range(6):
        out = torch.zeros(seqs, new, heads, d + pad, dtype=DT[dtype], device=DEV)[..., pad:]
        results.append(gptq.kv8_attention(q, dev, tab, length, out=out))
    for other in results[1:]:
        assert torch.equal(results[0], other)
    some = rng.permutation(seqs)[:8]
    _check_attention(results[0][some], q[some], cache, table[some], lengths[some])


# ---------------------------------------------------------------------------------------
# A dominant token (an attention sink) with a small value
# ---------------------------------------------------------------------------------------

def _sink_case(seqs, kv, new, group, d, tokens, weight, dtype, at):
    """Queries, cache and table of sequences with ``tokens`` tokens, of which token ``at`` takes
    ``weight`` of every row's softmax and has values of 1 %; the others' scores are a unit normal
    and their values have mean 0.5 and variance 1."""
    rng = np.random.default_rng(tokens + new)
    mb, kinds = -(-tokens // 64), min(seqs, 3)              # further sequences read the same blocks
    n = kinds * mb
    ones = rng.choice([-1.0, 1.0], d)                       # the direction that the queries share
    k = rng.standard_normal((n, kv, 64, d))
    v = 0.5 + rng.standard_normal((n, kv, d, 64))
    table = rng.permutation(n).reshape(kinds, mb).astype(np.int32)
    level = np.log(weight / (1 - weight)) + np.log(tokens) + 0.5
    pages = table[:, at // 64]
    k[pages, :, at % 64] = level / np.sqrt(d) * ones         # q = ones * sqrt(scores' variance)
    v[pages, :, :, at % 64] = 0.01 * rng.standard_normal((kinds, kv, d))
    cache = (SO.encode(k * 64), SO.encode(v * 64), np.full((n, kv), 121, np.uint8), np.full((n, kv), 121, np.uint8))
    q = ones + 0.02 * rng.standard_normal((seqs, new, kv * group, d))
    return torch.from_numpy(q).to(DT[dtype]), cache, table[np.arange(seqs) % kinds]


SINKS = [  # rows: one, eight, sixteen and thirty-two; long histories
    (1, 1, 1, 1, 128, 4000, 0.99), (1, 2, 1, 1, 64, 32768, 0.97), (2, 1, 1, 8, 64, 1000, 0.999), (1, 1, 1, 8, 128, 8000, 0.999),
    (1, 1, 1, 8, 64, 16000, 0.97), (1, 1, 1, 8, 64, 32768, 0.9), (1, 1, 2, 8, 64, 4000, 0.99), (1, 1, 2, 8, 128, 2000, 0.999),
    (1, 1, 2, 16, 64, 1000, 0.999), (1, 1, 4, 8, 64, 4000, 0.99), (1, 1, 4, 8, 64, 32768, 0.97), (1, 1, 2, 16, 64, 16000, 0.97),
    # long ones inside one share
    (160, 1, 1, 8, 128, 4000, 0.99), (160, 1, 2, 8, 64, 4000, 0.99), (160, 1, 4, 8, 64, 4000, 0.99), (152, 1, 1, 8, 64, 16000, 0.97),
    (152, 1, 4, 8, 64, 16000, 0.97),
    # short ones: dealt whole to CTAs and to groups
    (3, 2, 1, 8, 128, 1000, 0.999), (4, 1, 2, 8, 64, 500, 0.999), (3, 1, 4, 8, 64, 250, 0.999), (200, 1, 1, 4, 64, 180, 0.9999),
    (90, 2, 3, 4, 128, 250, 0.999), (170, 1, 4, 8, 64, 120, 0.999),
    # and one that leaves the others 2^-25 to 2^-28 each
    (1, 1, 1, 8, 64, 8000, 0.99995), (1, 1, 4, 8, 64, 8000, 0.99995),
]


@pytest.mark.parametrize("seqs,kv,new,group,d,tokens,weight", SINKS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("first", [True, False])
def test_attention_with_a_dominant_token(seqs, kv, new, group, d, tokens, weight, dtype, first):
    q, cache, table = _sink_case(seqs, kv, new, group, d, tokens, weight, dtype, 3 if first else tokens * 2 // 3)
    lengths = [tokens] * seqs
    dev = _dev_cache(cache)
    out = gptq.kv8_attention(q.to(DEV), dev, _i32(table), _i32(lengths), causal=False)
    assert torch.equal(out, gptq.kv8_attention(q.to(DEV), dev, _i32(table), _i32(lengths), causal=False))
    some = slice(0, 4)
    _check_attention(out[some], q[some], cache, table[some], lengths[some], causal=False)


@pytest.mark.parametrize("new,group", [(1, 8), (2, 8), (4, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attention_with_dominant_tokens_of_many_levels(new, group, dtype):
    # in every block a few tokens 2^10, 2^20, 2^30 above the rest, whose values are as small as they are large
    d, tokens = 64, 3000
    rng = np.random.default_rng(1)
    n = -(-tokens // 64)
    ones = rng.choice([-1.0, 1.0], d)
    level = rng.choice([0, 7, 14, 21], (n, 1, 64, 1), p=[0.9, 0.05, 0.03, 0.02])     # nats
    k = rng.standard_normal((n, 1, 64, d)) * 0.3 + level / np.sqrt(d) * ones
    v = (0.5 + rng.standard_normal((n, 1, 64, d))) * np.exp2(-10.0 * (level / 7) / 3)
    cache = (SO.encode(k * 64), SO.encode(v.transpose(0, 1, 3, 2).copy() * 64), np.full((n, 1), 121, np.uint8),
             np.full((n, 1), 121, np.uint8))
    table = rng.permutation(n).reshape(1, n).astype(np.int32)
    q = torch.from_numpy(ones + 0.02 * rng.standard_normal((1, new, group, d))).to(DT[dtype])
    out = gptq.kv8_attention(q.to(DEV), _dev_cache(cache), _i32(table), _i32([tokens]))
    _check_attention(out, q, cache, table, [tokens])


@pytest.mark.parametrize("new,group,d,tokens", [(1, 1, 128, 700), (1, 8, 128, 3000), (1, 8, 64, 100), (2, 8, 64, 3000), (4, 8, 64, 700),
                                                (4, 8, 128, 3000)])
@pytest.mark.parametrize("level", [10.0, 14.0, 17.0])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attention_behind_tokens_without_values(new, group, d, tokens, level, dtype):
    # in every block eight tokens that take nearly all of the weight and have no value at all
    rng = np.random.default_rng(int(level) + tokens)
    n = -(-tokens // 64)
    ones = rng.choice([-1.0, 1.0], d)
    k = rng.standard_normal((n, 1, 64, d))
    v = 0.5 + rng.standard_normal((n, 1, 64, d))
    k[:, :, 5::8] = level / np.sqrt(d) * ones
    v[:, :, 5::8] = 0
    cache = (SO.encode(k * 64), SO.encode(v.transpose(0, 1, 3, 2).copy() * 64), np.full((n, 1), 121, np.uint8),
             np.full((n, 1), 121 + 16, np.uint8))
    table = rng.permutation(n).reshape(1, n).astype(np.int32)
    q = torch.from_numpy(ones + 0.02 * rng.standard_normal((1, new, group, d))).to(DT[dtype])
    out = gptq.kv8_attention(q.to(DEV), _dev_cache(cache), _i32(table), _i32([tokens]))
    _check_attention(out, q, cache, table, [tokens])


# ---------------------------------------------------------------------------------------
# Norm: squares past fp32's range
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("rows,d", [(3, 40), (5, 4096), (2, 20000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top", [2.0 ** 50, 2.0 ** 58, 2.0 ** 63, 2.0 ** 64, 2.0 ** 100, 2.0 ** 125])
def test_norm_of_large_rows(rows, d, dtype, top):
    # rows of such elements, rows with one among ordinary ones, and ordinary rows beside them
    x = _randn(31, rows, d)
    x[0] = x[0] / x[0].abs().max() * top
    x[1, d // 3] = top
    x = x.to(DT[dtype])
    w = _randn(32, d, dtype=dtype) * 0.1
    c, e, rstd, h = gptq.rmsnorm_fp8(x.to(DEV), w.to(DEV), eps=1e-6)
    oc, oe, orstd, _ = SO.rmsnorm(_np(x), _np(w), None, 1e-6)
    np.testing.assert_allclose(_np(rstd), orstd, rtol=4e-6)
    np.testing.assert_array_equal(_np(c), oc)
    np.testing.assert_array_equal(_np(e), oe)
    y = rstd.double().cpu().numpy()[:, None] * SO.dequantize(_np(c), _np(e))
    want = _np(x).astype(np.float64) * orstd[:, None] * _np(w).astype(np.float64)
    assert np.all(np.abs(y - want) <= np.abs(want) / 15 + np.abs(want).max(1, keepdims=True) * 2.0 ** -17)


@pytest.mark.parametrize("where", ["x", "r"])
def test_norm_of_large_rows_in_place(where):
    # h replaces X or R; fp32, so that it is h itself
    x, r, w = _randn(1, 6, 700).to(DEV) * 2.0 ** 70, _randn(2, 6, 700).to(DEV) * 2.0 ** 69, _randn(3, 700).to(DEV) * 0.1
    want = gptq.rmsnorm_fp8(x, w, r)
    h = (x if where == "x" else r).clone()
    c, e = torch.empty(6, 704, dtype=torch.uint8, device=DEV), torch.empty(6, 8, dtype=torch.uint8, device=DEV)
    rstd = torch.zeros(6, device=DEV)
    p = gptq._ptr
    st = gptq.gptq_rmsnorm_fp8(p(h) if where == "x" else p(x), 2, 6, 700, 700, p(r) if where == "x" else p(h), 700, p(w), 2, 1e-6,
                               p(h), 700, p(c), 704, p(e), 8, p(rstd), gptq._stream(None))
    assert st == 0 and torch.equal(h, want[3]) and torch.equal(c[:, :700], want[0].view(torch.uint8))
    np.testing.assert_allclose(_np(rstd), SO.rmsnorm(_np(x), _np(w), _np(r), 1e-6)[2], rtol=4e-6)


@pytest.mark.parametrize("new,group,d,tokens", [(1, 1, 128, 3000), (1, 8, 64, 3000), (2, 8, 64, 3000), (1, 8, 128, 700), (2, 8, 128, 1500)])
@pytest.mark.parametrize("channels", [1, 8, 32])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attention_behind_tokens_with_values_in_few_channels(new, group, d, tokens, channels, dtype):
    # the other channels are the other tokens' alone, however large the first ones are
    rng = np.random.default_rng(channels + tokens)
    n = -(-tokens // 64)
    ones = rng.choice([-1.0, 1.0], d)
    k = rng.standard_normal((n, 1, 64, d))
    v = 0.5 + rng.standard_normal((n, 1, 64, d))
    k[:, :, 5::8] = 14.0 / np.sqrt(d) * ones
    v[:, :, 5::8, channels:] = 0
    cache = (SO.encode(k * 64), SO.encode(v.transpose(0, 1, 3, 2).copy() * 64), np.full((n, 1), 121, np.uint8),
             np.full((n, 1), 121 + 16, np.uint8))
    table = rng.permutation(n).reshape(1, n).astype(np.int32)
    q = torch.from_numpy(ones + 0.02 * rng.standard_normal((1, new, group, d))).to(DT[dtype])
    out = gptq.kv8_attention(q.to(DEV), _dev_cache(cache), _i32(table), _i32([tokens]))
    _check_attention(out, q, cache, table, [tokens])
