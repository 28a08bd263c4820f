"""GPU parity of the 8-bit serving operators against their 64-bit definitions.

Tolerances, from the arithmetic each operator is allowed:
  * codes, exponents, appended cache: equal bit for bit (the format's input u = h * w is defined
    in fp32, everything after it is exact or one defined rounding);
  * rstd: fp32 sums of d squares, at most ~64 of them in a row per thread plus a tree:
    64 * 2^-24 < 4e-6;
  * product: one rounding to the output type (half an ulp: 2^-9 bf16, 2^-12 f16 relative at most
    2^-8, 2^-11) plus fp32 accumulation over K in steps of 32 that may truncate:
    (K / 32 + 32) 2^-22 of the sum of the terms' magnitudes;
  * attention: probabilities held in 8 bits of significand or more (2^-8 of sum p |v|), scores
    exact up to fp32 sums and the exponential's own error (2^-18 of the largest sum of score
    terms, at most, on each exponent, twice), and the output's rounding.
"""

import math

import numpy as np
import pytest
import torch

from oracle import gptq_oracle as O
from oracle import serving_oracle as SO
from post_weight_quantization_03_gb300 import build_lib, gptq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ULP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    gptq.load()
    torch.cuda.init()


def _randn(seed, *shape, dtype="f32"):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DT[dtype])


def _np(t):
    t = t.detach().cpu()
    return (t.contiguous().view(torch.uint8) if t.dtype == F8 else t.float() if t.dtype == torch.bfloat16 else t).numpy()


def _padded(x, pad):
    """The matrix inside a wider one: rows that start off 16-byte boundaries for odd pads."""
    buf = torch.full((x.shape[0], x.shape[1] + pad), 7.0, dtype=x.dtype, device=DEV)
    buf[:, pad:] = x.to(DEV)
    return buf[:, pad:]


# ---------------------------------------------------------------------------------------
# Norm and quantizers
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("rows,d,dtype,wdtype,residual,pad", [
    (1, 1, "bf16", "bf16", True, 0), (3, 7, "f16", "f16", False, 0), (5, 128, "f32", "f32", True, 0),
    (2, 130, "bf16", "f32", True, 0), (33, 1000, "f16", "f32", True, 3), (7, 4096, "bf16", "bf16", True, 0),
    (4, 4099, "bf16", "bf16", True, 1), (3, 8192, "f32", "f32", False, 5), (2, 20000, "f16", "f16", True, 8),
    (300, 264, "bf16", "bf16", False, 8),
])
def test_norm(rows, d, dtype, wdtype, residual, pad):
    x = _randn(1, rows, d, dtype=dtype)
    x[:, ::5] *= 30
    r = _randn(2, rows, d, dtype=dtype) * 3 if residual else None
    w = (1 + 0.3 * _randn(3, d)).to(DT[wdtype])
    if rows > 2:
        x[1] = 0
        if r is not None:
            r[1] = 0
    c, e, rstd, h = gptq.rmsnorm_fp8(_padded(x, pad), w.to(DEV), _padded(r, pad) if residual else None, 1e-5)
    oc, oe, orstd, oh = SO.rmsnorm(_np(x), _np(w), None if r is None else _np(r), 1e-5)
    np.testing.assert_array_equal(_np(c), oc)
    np.testing.assert_array_equal(_np(e), oe)
    np.testing.assert_allclose(_np(rstd), orstd, rtol=4e-6)
    assert torch.equal(h.cpu(), torch.from_numpy(oh).to(DT[dtype]))


def test_norm_in_place_and_without_h():
    x, r = _randn(1, 9, 512, dtype="bf16").to(DEV), _randn(2, 9, 512, dtype="bf16").to(DEV)
    w = _randn(3, 512, dtype="bf16").to(DEV)
    c, e, rstd, h = gptq.rmsnorm_fp8(x, w, r)
    c2, e2, rstd2, none = gptq.rmsnorm_fp8(x, w, r, want_h=False)
    assert none is None and torch.equal(c.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(rstd, rstd2)
    hr = r.clone()
    c3, e3 = torch.empty_like(c), torch.empty(9, 4, dtype=torch.uint8, device=DEV)
    st = gptq.gptq_rmsnorm_fp8(gptq._ptr(x), 1, 9, 512, 512, gptq._ptr(hr), 512, gptq._ptr(w), 1, 1e-6, gptq._ptr(hr), 512,
                               gptq._ptr(c3), 512, gptq._ptr(e3), 4, gptq._ptr(rstd2), gptq._stream(None))
    assert st == 0 and torch.equal(hr, h) and torch.equal(c3.view(torch.uint8), c.view(torch.uint8)) and torch.equal(e3, e)


def test_norm_marks_what_is_not_finite():
    x = _randn(4, 4, 300, dtype="f32")
    x[1, 5], x[2, 200], x[2, 3] = math.inf, math.nan, -math.inf
    w = torch.ones(300)
    c, e, rstd, _ = gptq.rmsnorm_fp8(x.to(DEV), w.to(DEV))
    oc, oe, _, _ = SO.rmsnorm(_np(x), _np(w))
    np.testing.assert_array_equal(_np(c), oc)
    np.testing.assert_array_equal(_np(e), oe)
    assert _np(c)[1, 5] == _np(c)[2, 200] == 0x7F and float(rstd[1]) == 0 and math.isnan(float(rstd[2]))
    assert np.isfinite(_np(rstd)[[0, 3]]).all()


@pytest.mark.parametrize("rows,d,dtype,pad", [(1, 1, "f32", 0), (5, 127, "bf16", 0), (130, 300, "f16", 0), (256, 256, "f32", 1),
                                              (129, 4096, "bf16", 0), (64, 11008, "bf16", 8)])
@pytest.mark.parametrize("row_block", [1, 128])
def test_quantize(rows, d, dtype, pad, row_block):
    x = (_randn(5, rows, d) * torch.exp(3 * _randn(6, rows, 1))).to(DT[dtype])
    x[rows // 2, d // 3] = math.nan
    c, e = gptq.fp8_quantize(_padded(x, pad), row_block)
    oc, oe = SO.quantize(_np(x), row_block)
    np.testing.assert_array_equal(_np(c), oc)
    np.testing.assert_array_equal(_np(e), oe)


def test_quantize_extreme_magnitudes():
    x = torch.tensor([[3.4e38, 1.0], [1e-40, 1e-45], [448.0, -448.0], [2.0 ** -90, 2.0 ** -100], [449.0, 1e-3]])
    c, e = gptq.fp8_quantize(x.to(DEV))
    oc, oe = SO.quantize(x.numpy())
    np.testing.assert_array_equal(_np(c), oc)
    np.testing.assert_array_equal(_np(e), oe)


def test_norm_of_no_rows():
    c, e, rstd, h = gptq.rmsnorm_fp8(torch.empty(0, 64, device=DEV), torch.ones(64, device=DEV))
    assert c.shape == (0, 64) and rstd.shape == (0,)


# ---------------------------------------------------------------------------------------
# Product
# ---------------------------------------------------------------------------------------

def _fp8_matrix(seed, rows, d, row_block, spread=2.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, d)) * np.exp2(np.rint(rng.standard_normal((1, d)) * spread))
    codes, exps = SO.quantize(x, row_block)
    return codes, exps


def _dev_codes(codes, fill=0x7F):
    """Codes in a 16-byte pitch, NaN in the padding (which must not be read into a result)."""
    rows, d = codes.shape
    buf = torch.full((rows, -(-d // 16) * 16 + 16), fill, dtype=torch.uint8, device=DEV)
    buf[:, :d] = torch.from_numpy(codes).to(DEV)
    return buf.view(F8)[:, :d]


def _dev_exps(exps):
    rows, kb = exps.shape
    buf = torch.full((rows, -(-kb // 4) * 4 + 4), 255, dtype=torch.uint8, device=DEV)
    buf[:, :kb] = torch.from_numpy(exps).to(DEV)
    return buf[:, :kb]


def _check_product(out, want, mag, k):
    tol = ULP[out.dtype] * np.abs(want) + (k / 32 + 32) * 2.0 ** -22 * mag + 1e-30
    got = out.double().cpu().numpy()
    worst = np.max(np.abs(got - want) / tol)
    assert worst <= 1, worst


PRODUCTS = [
    (1, 1, 1), (1, 128, 128), (3, 130, 200), (16, 256, 512), (17, 257, 1000), (1, 513, 4096), (8, 128, 11008), (33, 384, 640),
    (64, 100, 129), (65, 256, 2048), (127, 129, 257), (128, 128, 128), (130, 640, 384), (255, 500, 700), (257, 1024, 1152),
    (300, 2000, 96), (513, 300, 4112), (2, 64, 28672), (48, 128, 16),
]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_product(m, n, k, dtype):
    a, ae = _fp8_matrix(m + k, m, k, 1)
    w, we = _fp8_matrix(n + k + 1, n, k, 128)
    rng = np.random.default_rng(7)
    ra, rw = rng.uniform(0.01, 0.1, m).astype(np.float32), rng.uniform(0.01, 0.1, n).astype(np.float32)
    if dtype == "f16":
        ra, rw = ra / np.float32(k), rw   # inside the type's range
    want, mag = SO.matmul(a, ae, w, we, ra, rw)
    out = gptq.fp8_matmul(_dev_codes(a), _dev_exps(ae), _dev_codes(w), _dev_exps(we), torch.from_numpy(ra).to(DEV),
                          torch.from_numpy(rw).to(DEV), out_dtype=DT[dtype])
    _check_product(out, want, mag, k) if dtype == "bf16" else _check_product_f16(out, want, mag, k)


def _check_product_f16(out, want, mag, k):
    tol = ULP[out.dtype] * np.abs(want) + (k / 32 + 32) * 2.0 ** -22 * mag + 2.0 ** -25  # subnormal half step
    assert np.max(np.abs(out.double().cpu().numpy() - want) / tol) <= 1


def test_product_without_scales_into_a_wider_output_and_repeats():
    m, n, k = 70, 300, 1500
    a, ae = _fp8_matrix(1, m, k, 1, 0.5)
    w, we = _fp8_matrix(2, n, k, 128, 0.5)
    want, mag = SO.matmul(a, ae, w, we)
    for pad in (1, 4):
        buf = torch.full((m, n + 5), 3.0, dtype=torch.bfloat16, device=DEV)
        args = (_dev_codes(a), _dev_exps(ae), _dev_codes(w), _dev_exps(we))
        out = gptq.fp8_matmul(*args, out=buf[:, pad:pad + n])
        _check_product(out, want, mag, k)
        assert (buf[:, :pad] == 3).all() and (buf[:, pad + n:] == 3).all()
        again = gptq.fp8_matmul(*args)
        assert torch.equal(out, again)


def test_product_wide_exponents_and_zero_blocks():
    # neighbouring blocks of K up to 2^60 apart, whole blocks of zeros, columns that cancel
    m, n, k = 20, 140, 1024
    a, ae = _fp8_matrix(3, m, k, 1, 0.5)
    w, we = _fp8_matrix(4, n, k, 128, 0.5)
    rng = np.random.default_rng(5)
    ae = (127 + rng.integers(-30, 31, ae.shape)).astype(np.uint8)
    we = (127 + rng.integers(-30, 31, we.shape)).astype(np.uint8)
    a[:, 128:256], w[:, 512:640] = 0, 0
    ae[:, 1], we[:, 4] = 31, 31
    want, mag = SO.matmul(a, ae, w, we)
    out = gptq.fp8_matmul(_dev_codes(a), _dev_exps(ae), _dev_codes(w), _dev_exps(we))
    _check_product(out, want, mag, k)


@pytest.mark.parametrize("m", [5, 300])
def test_product_nan_stays_in_its_row_and_column(m):
    n, k = 200, 400
    a, ae = _fp8_matrix(8, m, k, 1)
    w, we = _fp8_matrix(9, n, k, 128)
    a[3, 77], w[150, 399] = 0x7F, 0xFF
    out = gptq.fp8_matmul(_dev_codes(a), _dev_exps(ae), _dev_codes(w), _dev_exps(we)).float().cpu().numpy()
    bad = np.isnan(out)
    assert bad[3].all() and bad[:, 150].all() and bad.sum() == n + m - 1


def test_product_of_no_tokens():
    w, we = _fp8_matrix(9, 64, 128, 128)
    a, ae = torch.empty(0, 128, dtype=F8, device=DEV), torch.empty(0, 4, dtype=torch.uint8, device=DEV)[:, :1]
    assert gptq.fp8_matmul(a, ae, _dev_codes(w), _dev_exps(we)).shape == (0, 64)


@pytest.mark.parametrize("bits,m,d", [(2, 5, 33), (3, 130, 300), (4, 64, 256), (4, 257, 1000)])
def test_gptq_codes_are_served_exactly(bits, m, d):
    # codes, zeros and steps as the sweep writes them; x exact in e4m3
    rng = np.random.default_rng(bits)
    codes = rng.integers(0, 2 ** bits, (m, d)).astype(np.uint8)
    zero = rng.integers(0, 2 ** bits, m).astype(np.int32)
    scale = rng.uniform(0.001, 0.01, m).astype(np.float32)
    packed = O.pack_codes(codes, bits).view(np.int32)
    c, e = gptq.fp8_from_codes(torch.from_numpy(packed).to(DEV), torch.from_numpy(zero).to(DEV), d, bits)
    np.testing.assert_array_equal(SO.decode(_np(c)), codes.astype(float) - zero[:, None])
    assert (_np(e) == 127).all() and e.shape == (-(-m // 128), -(-d // 128))
    x, xe = _fp8_matrix(10, 6, d, 1, 0.5)
    out = gptq.fp8_matmul(_dev_codes(x), _dev_exps(xe), c, e, w_scale=torch.from_numpy(scale).to(DEV))
    w_hat = scale.astype(np.float64)[:, None] * (codes.astype(float) - zero[:, None])
    xv = SO.dequantize(x, xe)
    _check_product(out, xv @ w_hat.T, np.abs(xv) @ np.abs(w_hat).T, d)


# ---------------------------------------------------------------------------------------
# Cache: append
# ---------------------------------------------------------------------------------------

def _cache(seed, n_blocks, kv, d, spread=1):
    """Random valid codes everywhere and exponents a few powers of two apart."""
    rng = np.random.default_rng(seed)
    k = SO.encode(rng.standard_normal((n_blocks, kv, 64, d)) * 100)
    v = SO.encode(rng.standard_normal((n_blocks, kv, d, 64)) * 100)
    ke, ve = (np.uint8(127 - 7) + rng.integers(-spread, spread + 1, (n_blocks, kv)).astype(np.int8).view(np.uint8) for _ in range(2))
    return k, v, ke.astype(np.uint8), ve.astype(np.uint8)


def _dev_cache(cache):
    k, v, ke, ve = (torch.from_numpy(t.copy()).to(DEV) for t in cache)
    return k.view(F8), v.view(F8), ke, ve


def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32), device=DEV)


def _table(rng, seqs, blocks, n_blocks):
    return rng.permutation(n_blocks)[:seqs * blocks].reshape(seqs, blocks).astype(np.int32)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("new,starts", [(1, [0, 63, 64, 130]), (5, [60, 0, 61, 5]), (64, [0, 1, 64, 100]), (200, [3, 0, 64, 56])])
def test_append(d, dtype, new, starts):
    rng = np.random.default_rng(new)
    kv, n_blocks, mb = 3, 24, 5
    cache, table = _cache(new, n_blocks, kv, d), _table(rng, 4, mb, n_blocks)
    k, v = _randn(1, 4, new, kv, d, dtype=dtype), _randn(2, 4, new, kv, d, dtype=dtype)
    k[1] *= 100
    v[2] *= 1000                      # raises the exponents of what is there
    v[3] *= 1e-3                      # does not
    dev = _dev_cache(cache)
    gptq.kv8_append(dev, k.to(DEV), v.to(DEV), _i32(table), _i32(starts))
    want = SO.kv_append(cache, _np(k), _np(v), table, starts)
    for got, w in zip(dev, want):
        np.testing.assert_array_equal(_np(got), w)
    gptq.kv8_append(dev, k.to(DEV), v.to(DEV), _i32(table), _i32(starts))  # the same tokens again
    again = SO.kv_append(want, _np(k), _np(v), table, starts)
    for got, w in zip(dev, again):
        np.testing.assert_array_equal(_np(got), w)


def test_append_strided_unaligned_and_dropped():
    d, kv = 128, 2
    rng = np.random.default_rng(3)
    cache, table = _cache(3, 10, kv, d), _table(rng, 3, 2, 10)
    table[1, 0], table[2, 1] = -1, 10                      # no such blocks
    qkv = _randn(4, 3, 70, kv, 2 * d + 1, dtype="bf16").to(DEV)   # rows off 16 bytes
    k, v = qkv[..., :d], qkv[..., d + 1:]
    dev = _dev_cache(cache)
    starts = [100, 10, -5]                                 # past the table's end; a negative start
    gptq.kv8_append(dev, k, v, _i32(table), _i32(starts))
    want = SO.kv_append(cache, _np(k), _np(v), table, starts)
    for got, w in zip(dev, want):
        np.testing.assert_array_equal(_np(got), w)


def test_append_marks_tokens_that_are_not_finite():
    d, kv = 64, 2
    cache, table = _cache(5, 4, kv, d), np.array([[2, 1]], np.int32)
    k, v = _randn(1, 1, 80, kv, d), _randn(2, 1, 80, kv, d)
    v[0, 7, 1, 3], v[0, 70, 0, 0], k[0, 9, 0, 5] = math.inf, math.nan, -math.inf
    dev = _dev_cache(cache)
    gptq.kv8_append(dev, k.to(DEV), v.to(DEV), _i32(table), _i32([20]))
    want = SO.kv_append(cache, _np(k), _np(v), table, [20])
    for got, w in zip(dev, want):
        np.testing.assert_array_equal(_np(got), w)
    q = _randn(3, 1, 80, 2 * kv, d, dtype="bf16")
    out = gptq.kv8_attention(q.to(DEV), dev, _i32(table), _i32([100])).float().cpu().numpy()
    nan = np.isnan(out).all(-1)[0]
    assert np.array_equal(np.isnan(out).any(-1)[0], nan)
    t = np.arange(80)
    assert np.array_equal(nan[:, 0], t >= 9) and np.array_equal(nan[:, 2], t >= 7)


# ---------------------------------------------------------------------------------------
# Cache: attention
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("seqs,new,group,length,dtype", [(2, 1, 4, 150, "bf16"), (2, 1, 4, 150, "f16"), (2, 1, 8, 4000, "bf16"),
                                                         (1, 70, 8, 200, "bf16"), (1, 70, 8, 200, "f16"), (1, 300, 4, 2000, "bf16")])
def test_attention_queries_that_are_not_finite(seqs, new, group, length, dtype):
    # a row of queries with an infinity or a NaN in it has no softmax: it becomes NaN, and only it
    kv, d, mb = 2, 64, -(-length // 64)
    cache, table = _cache(11, seqs * mb, kv, d), np.arange(seqs * mb, dtype=np.int32).reshape(seqs, mb)
    q = _randn(12, seqs, new, kv * group, d, dtype=dtype)
    clean = gptq.kv8_attention(q.to(DEV), _dev_cache(cache), _i32(table), _i32([length] * seqs))
    bad = np.zeros((seqs, new, kv * group), bool)
    for i, x in enumerate((math.inf, -math.inf, math.nan)):
        at = (i % seqs, (37 * i) % new, (3 * i + 1) % (kv * group))
        q[at + (5 + 20 * i,)] = x
        bad[at] = True
    out = gptq.kv8_attention(q.to(DEV), _dev_cache(cache), _i32(table), _i32([length] * seqs))
    nan = torch.isnan(out)
    assert np.array_equal(_np(nan.all(-1)), bad) and np.array_equal(_np(nan.any(-1)), bad)
    ok = torch.from_numpy(~bad).to(DEV)
    assert torch.equal(out[ok], clean[ok])


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("top", [2.0 ** -110, 2.0 ** -60, 2.0 ** 60, 2.0 ** 100, 2.0 ** 121, 3.3e38])
def test_attention_queries_at_the_ends_of_their_range(new, top):
    cache, table = _cache(13, 3, 1, 64), np.array([[2, 0, 1]], np.int32)
    q = _randn(14, 1, new, 8, 64).double()
    q = (q / q.abs().amax(-1, keepdim=True) * top).to(torch.bfloat16)
    out = gptq.kv8_attention(q.to(DEV), _dev_cache(cache), _i32(table), _i32([180]), scale=0.5 / top)
    _check_attention(out, q, cache, table, [180], scale=0.5 / top)


def _check_attention(out, q, cache, table, lengths, **kw):
    want, mag, terms = SO.kv_attention(_np(q), cache, table, lengths, **kw)
    tol = ULP[out.dtype] * np.abs(want) + (2.0 ** -8 + 2 * 2.0 ** -18 * max(terms, 1.0)) * mag + 1e-7
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - want) / tol)
    assert worst <= 1, worst


ATTENTION = [  # seqs, new, kv heads, group, dim, lengths, blocks of the table
    (1, 1, 1, 1, 128, [1], 1), (2, 1, 2, 1, 64, [0, 64], 1), (3, 1, 2, 4, 128, [63, 65, 700], 12), (2, 1, 1, 8, 64, [128, 1000], 16),
    (2, 1, 2, 16, 128, [300, 5], 5), (1, 1, 1, 7, 128, [3000], 47), (2, 2, 2, 3, 128, [100, 257], 5), (1, 4, 2, 8, 64, [777], 13),
    (2, 3, 1, 20, 128, [2, 400], 7), (1, 64, 2, 2, 128, [64], 1), (2, 65, 1, 4, 64, [65, 300], 5), (1, 200, 2, 4, 128, [200], 4),
    (2, 130, 2, 1, 128, [40, 513], 9), (1, 33, 1, 16, 64, [1111], 18), (3, 17, 1, 5, 128, [17, 16, 0], 2), (1, 300, 1, 3, 64, [1500], 24),
]


@pytest.mark.parametrize("seqs,new,kv,group,d,lengths,mb", ATTENTION)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attention(seqs, new, kv, group, d, lengths, mb, dtype):
    rng = np.random.default_rng(new + d)
    n_blocks = seqs * mb + 2
    cache, table = _cache(new, n_blocks, kv, d), _table(rng, seqs, mb, n_blocks)
    q = _randn(9, seqs, new, kv * group, d, dtype=dtype)
    dev = _dev_cache(cache)
    out = gptq.kv8_attention(q.to(DEV), dev, _i32(table), _i32(lengths))
    _check_attention(out, q, cache, table, lengths)
    assert torch.equal(out, gptq.kv8_attention(q.to(DEV), dev, _i32(table), _i32(lengths)))
    full = gptq.kv8_attention(q.to(DEV), dev, _i32(table), _i32(lengths), scale=0.05, causal=False)
    _check_attention(full, q, cache, table, lengths, scale=0.05, causal=False)


@pytest.mark.parametrize("seqs,new,kv,group,d,longest", [
    (5, 1, 3, 4, 128, 5000), (40, 1, 2, 8, 64, 1500), (7, 2, 1, 8, 128, 3000), (3, 4, 2, 8, 64, 2500), (200, 1, 1, 2, 64, 1300),
    (3, 40, 2, 4, 128, 3000), (30, 9, 1, 4, 64, 1200),
    # more items than there are CTAs, of a few blocks each
    (200, 1, 2, 4, 64, 300), (170, 1, 1, 1, 128, 1000), (90, 3, 4, 4, 128, 400), (80, 8, 4, 4, 64, 250), (700, 1, 2, 2, 64, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attention_many_lengths(seqs, new, kv, group, d, longest, dtype):
    # more blocks than are dealt whole: items cut by the shares, empty sequences between them
    rng = np.random.default_rng(seqs)
    lengths = rng.integers(0, longest + 1, seqs)
    lengths[0], lengths[seqs // 2], lengths[-1] = longest, 0, 1
    n_blocks, mb = 64, -(-longest // 64)
    cache, table = _cache(new, n_blocks, kv, d), rng.integers(0, n_blocks, (seqs, mb)).astype(np.int32)
    q = _randn(9, seqs, new, kv * group, d, dtype=dtype)
    out = gptq.kv8_attention(q.to(DEV), _dev_cache(cache), _i32(table), _i32(lengths))
    _check_attention(out, q, cache, table, lengths)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("new", [1, 50])
def test_attention_scales(new, scale):
    cache, table = _cache(3, 6, 2, 64), np.array([[3, 1, 5, 0]], np.int32)
    q = _randn(4, 1, new, 8, 64, dtype="bf16")
    out = gptq.kv8_attention(q.to(DEV), _dev_cache(cache), _i32(table), _i32([230]), scale=scale)
    _check_attention(out, q, cache, table, [230], scale=scale)


@pytest.mark.parametrize("new,group", [(1, 8), (100, 4)])
def test_attention_ignores_what_is_past_the_length(new, group):
    d, kv, length = 128, 2, 330
    cache = _cache(1, 8, kv, d)
    table = np.array([[5, 2, 7, 0, 1, 3, 6, 4]], np.int32)
    q = _randn(2, 1, new, kv * group, d, dtype="bf16")
    clean = gptq.kv8_attention(q.to(DEV), _dev_cache(cache), _i32(table), _i32([length]))
    dirty = tuple(t.copy() for t in cache)
    dirty[0][3, :, length % 64:] = 0x7F                    # NaN codes and exponents
    dirty[1][3, :, :, length % 64:] = 0xFF
    for t in dirty[:2]:
        t[[6, 4]] = 0x7F
    dirty[2][[6, 4]], dirty[3][[6, 4]] = 255, 255
    out = gptq.kv8_attention(q.to(DEV), _dev_cache(dirty), _i32(table), _i32([length]))
    assert torch.equal(out, clean)
    _check_attention(out, q, cache, table, [length])


@pytest.mark.parametrize("new,group", [(1, 4), (70, 2)])
def test_attention_over_blocks_that_are_not_there(new, group):
    d, kv = 64, 2
    cache = _cache(1, 6, kv, d)
    table = np.array([[-1, 3, 6, 0, -7, 1], [-1, -1, -1, -1, -1, -1]], np.int32)
    q = _randn(2, 2, new, kv * group, d, dtype="f16")
    out = gptq.kv8_attention(q.to(DEV), _dev_cache(cache), _i32(table), _i32([380, 380]))
    _check_attention(out, q, cache, table, [380, 380])
    assert (out[1] == 0).all()


@pytest.mark.parametrize("new,group", [(1, 4), (90, 4)])
def test_attention_peaked_scores_and_uneven_blocks(new, group):
    # scores up to hundreds, blocks whose value exponents are 2^20 apart
    d, kv = 128, 1
    k, v, ke, ve = _cache(4, 9, kv, d)
    ke = (ke.astype(int) + 4).astype(np.uint8)
    ve = (ve.astype(int) + np.array([0, -10, 10, 3, -3, 5, 0, 1, -10])[:, None]).astype(np.uint8)
    cache, table = (k, v, ke, ve), np.arange(9, dtype=np.int32)[None, ::-1].copy()
    q = _randn(2, 1, new, kv * group, d, dtype="bf16") * 4
    out = gptq.kv8_attention(q.to(DEV), _dev_cache(cache), _i32(table), _i32([570]))
    want, mag, terms = SO.kv_attention(_np(q), cache, table, [570])
    # a block's probabilities are rounded in units of the largest block value of the row
    top = float(SO.TABLE[:0x7F].max()) * 2.0 ** (float(ve.max()) - 127) * 2.0 ** -17
    tol = ULP[out.dtype] * np.abs(want) + (2.0 ** -8 + 2.0 ** -17 * terms) * mag + top
    assert np.max(np.abs(out.double().cpu().numpy() - want) / tol) <= 1


def test_attention_strided_tensors_on_another_stream():
    d, kv, group, new = 128, 2, 4, 40
    cache = _cache(1, 8, kv, d)
    table = np.array([[5, 2, 7], [0, 1, 3]], np.int32)
    wide = _randn(3, 2, new, kv * group + 3, d + 8, dtype="bf16").to(DEV)
    odd = _randn(3, 2, new, kv * group, d + 1, dtype="bf16").to(DEV)
    tab = torch.full((2, 5), 10 ** 9, dtype=torch.int32, device=DEV)
    tab[:, :3] = _i32(table)
    s = torch.cuda.Stream()
    dev = _dev_cache(cache)
    s.wait_stream(torch.cuda.current_stream())
    for q in (wide[:, :, 3:, 8:], odd[..., 1:], wide[:, :, 3:, 8:].expand(2, new, kv * group, d)):
        buf = torch.zeros(2, kv * group, new, d + 2, dtype=torch.bfloat16, device=DEV)
        out = buf.transpose(1, 2)[..., 2:]
        s.wait_stream(torch.cuda.current_stream())
        gptq.kv8_attention(q, dev, tab[:, :3], _i32([150, 77]), out=out, stream=s)
        s.synchronize()
        _check_attention(out, q, cache, table, [150, 77])
        assert (buf[..., :2] == 0).all()
    one = wide[:1, :1, 3:, 8:].expand(2, new, kv * group, d)          # broadcast queries
    out = gptq.kv8_attention(one, dev, tab[:, :3], _i32([150, 77]))
    _check_attention(out, one, cache, table, [150, 77])


@pytest.mark.parametrize("new", [1, 80])
def test_attention_past_32_bit_offsets(new):
    d, kv, group = 128, 8, 2
    n_blocks = 66000                                        # 4.3e9 bytes of keys and of values
    small, table = _cache(6, 4, kv, d), np.array([[0, 1, 2, 3]], np.int32)
    at = torch.tensor([65999, 65600, 32800, 0], device=DEV)
    big = [torch.empty(n_blocks, *t.shape[1:], dtype=torch.uint8, device=DEV) for t in small]
    for t, b in zip(small, big):
        b[at] = torch.from_numpy(t).to(DEV)
    cache = (big[0].view(F8), big[1].view(F8), big[2], big[3])
    q = _randn(2, 1, new, kv * group, d, dtype="bf16")
    out = gptq.kv8_attention(q.to(DEV), cache, at[None].int(), _i32([240]))
    _check_attention(out, q, small, table, [240])
    k, v = _randn(3, 1, 3, kv, d, dtype="bf16"), _randn(4, 1, 3, kv, d, dtype="bf16")
    gptq.kv8_append(cache, k.to(DEV), v.to(DEV), at[None].int(), _i32([62]))
    want = SO.kv_append(small, _np(k), _np(v), table, [62])
    for got, w in zip(big, want):
        np.testing.assert_array_equal(got[at].cpu().numpy(), w)


def test_attention_of_nothing():
    cache = _dev_cache(_cache(1, 2, 1, 64))
    q = torch.empty(0, 1, 2, 64, dtype=torch.bfloat16, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    assert gptq.kv8_attention(q, cache, torch.empty(0, 2, dtype=torch.int32, device=DEV), none).shape == q.shape
    q = _randn(1, 2, 3, 2, 64, dtype="bf16").to(DEV)
    out = gptq.kv8_attention(q, cache, torch.empty(2, 0, dtype=torch.int32, device=DEV), _i32([5, 5]))
    assert (out == 0).all()


def test_calls_in_a_graph():
    d, kv, heads = 128, 2, 8
    cache = _dev_cache(_cache(1, 8, kv, d))
    table, start, lengths = _i32([[5, 2, 7]]), _i32([100]), _i32([101])
    k, v, q = (_randn(i, 1, 1, h, d, dtype="bf16").to(DEV) for i, h in ((1, kv), (2, kv), (3, heads)))
    x, w = _randn(4, 1, heads * d, dtype="bf16").to(DEV), torch.ones(heads * d, dtype=torch.bfloat16, device=DEV)
    W, We = gptq.fp8_quantize(_randn(5, 640, heads * d, dtype="bf16").to(DEV), 128)

    def step():
        gptq.kv8_append(cache, k, v, table, start)
        o = gptq.kv8_attention(q, cache, table, lengths)
        c, e, r, h = gptq.rmsnorm_fp8(o.view(1, -1), w, x)
        return o, gptq.fp8_matmul(c, e, W, We, a_scale=r)

    want = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for t in got:
        t.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
