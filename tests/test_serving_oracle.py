"""Pins of the 8-bit serving oracle: the number format by hand, and the definitions against
direct computation on small inputs."""

import math

import numpy as np
import pytest
import torch

from oracle import serving_oracle as SO


def test_decode_table_is_e4m3():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(SO.TABLE, want)
    assert SO.TABLE[0x7E] == 448 and math.isnan(SO.TABLE[0x7F]) and SO.TABLE[1] == 2.0 ** -9


def test_encode_rounds_to_nearest_even():
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(4000, generator=g) * 30, torch.randn(2000, generator=g) * 1e-2,
                   torch.from_numpy((SO.TABLE[:126] + SO.TABLE[1:127]) / 2).float(),  # ties
                   torch.tensor([0.0, -0.0, 448.0, -448.0])]).clamp(-448, 448)
    np.testing.assert_array_equal(SO.encode(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert list(SO.encode([math.inf, -math.inf, math.nan])) == [0x7F] * 3


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0001, 1), (449.0, 1), (224.0, -1), (1.75, -8),
                                    (1.0, -8), (0.0, -96), (1e-45, -96), (3e38, 120)])
def test_block_exponent(amax, e):
    assert SO.block_exponent(amax) == e
    if amax > 0 and e > -96:
        assert amax / 2.0 ** e <= 448 and amax / 2.0 ** (e - 1) > 448


def test_quantize_blocks():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 300)) * 10.0 ** rng.uniform(-3, 3, (200, 1))
    for rb in (1, 128):
        c, e = SO.quantize(x, rb)
        assert e.shape == (200 if rb == 1 else 2, 3)
        step = 2.0 ** (np.repeat(np.repeat(e.astype(float), rb, 0), 128, 1)[:200, :300] - 127)
        assert np.all(np.abs(SO.dequantize(c, e, rb) - x) <= np.maximum(np.abs(x) / 16, step * 2.0 ** -10))


def test_append_one_at_a_time_keeps_values():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 1, 70, 2, 64))
    cache = (np.zeros((3, 2, 64, 64), np.uint8), np.zeros((3, 2, 64, 64), np.uint8),
             np.full((3, 2), 127, np.uint8), np.full((3, 2), 127, np.uint8))
    table = np.array([[2, 0]], np.int32)
    for t in range(70):
        cache = SO.kv_append(cache, k[:, t:t + 1], v[:, t:t + 1], table, np.array([t]))
    kc, vc, ke, ve = cache
    for h in range(2):
        got = SO.decode(kc[2, h]) * 2.0 ** (float(ke[2, h]) - 127)
        # a code is rounded again for each raise of the exponent, on the same grid or a coarser one
        assert np.all(np.abs(got - k[0, :64, h]) <= np.abs(k[0, :64, h]) / 8 + 2.0 ** (float(ke[2, h]) - 127 - 9))
        got = SO.decode(vc[0, h])[:, :6].T * 2.0 ** (float(ve[0, h]) - 127)
        assert np.all(np.abs(got - v[0, 64:, h]) <= np.abs(v[0, 64:, h]) / 8 + 2.0 ** (float(ve[0, h]) - 127 - 9))
    assert np.all(kc[1] == 0)


def test_attention_of_a_uniform_cache_is_the_mean():
    # equal keys: the softmax is uniform over the visible tokens, so the output is their mean
    kc = np.full((2, 1, 64, 64), SO.encode(1.0), np.uint8)
    vc = SO.encode(np.arange(2 * 64 * 64).reshape(2, 1, 64, 64) % 7 / 4.0)
    ones = np.full((2, 1), 127, np.uint8)
    q = np.random.default_rng(2).standard_normal((1, 3, 2, 64))
    table = np.array([[1, 0]], np.int32)
    out, _, _ = SO.kv_attention(q, (kc, vc, ones, ones), table, np.array([100]))
    V = np.concatenate([SO.decode(vc[1, 0]).T, SO.decode(vc[0, 0]).T])
    for t in range(3):
        np.testing.assert_allclose(out[0, t, 0], V[:98 + t].mean(0), rtol=1e-12)
    out, _, _ = SO.kv_attention(q, (kc, vc, ones, ones), table, np.array([2]))
    assert np.all(out[0, 0] == 0) and np.allclose(out[0, 2, 1], V[:2].mean(0))
    out, _, _ = SO.kv_attention(q, (kc, vc, ones, ones), np.array([[-1, 0]], np.int32), np.array([128]))
    np.testing.assert_allclose(out[0, 2, 1], V[64:].mean(0), rtol=1e-12)
