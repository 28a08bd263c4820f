"""GPU parity of the feed-forward operators (products with an epilogue, routing to experts, the experts'
products and their sum) against their 64-bit definitions.

Tolerances, from the arithmetic each operator is allowed:
  * a product before its epilogue: e_z = (K / 32 + 32) 2^-22 of the sum of the terms' magnitudes, as
    for the plain product;
  * an activation: its slope (at most 1.13) times that, and 2^-20 of its argument (fp32 exponential,
    quotient, error function);
  * an output: one rounding of half a step (2^-8 bf16, 2^-11 f16; half the smallest step 2^-25 for f16);
  * gated codes: half a step of e4m3 (2^-4 of the value, 2^-10 of the block's scale for its smallest);
    a block's exponent is that of a largest magnitude within the value's tolerance;
  * ids, offsets, order: equal; weights: fp32 exponentials and a sum of up to 1024 scores: 2^-17;
  * combine: fp32 sums of k terms: (k + 1) 2^-24 of the magnitudes, and the output's rounding.
"""

import gc
import math

import numpy as np
import pytest
import torch

from oracle import serving_oracle as SO
from post_weight_quantization_03_gb300 import build_lib, gptq
from tests.test_gpu_serving import DEV, DT, ULP, _dev_codes, _dev_exps, _fp8_matrix, _np, _padded, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    gptq.load()
    torch.cuda.init()
    yield
    gc.collect()   # frames of expected errors hold tensors: others' tests look at what is allocated


def _dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _weights(seed, n, k, scale=True, bias=False, spread=0.5):
    """(codes, exps, scale, bias) on the host."""
    w, we = _fp8_matrix(seed, n, k, 128, spread)
    rng = np.random.default_rng(seed + 1)
    rw = (rng.uniform(0.5, 1.5, n) / math.sqrt(k)).astype(np.float32) if scale else None
    return w, we, rw, rng.standard_normal(n).astype(np.float32) if bias else None


def _on_dev(w):
    return _dev_codes(w[0]), _dev_exps(w[1]), _dev(w[2]), _dev(w[3])


def _experts_on_dev(ws):
    """One matrix for each expert, in pitches of their own."""
    codes = torch.stack([_dev_codes(w[0]).view(torch.uint8) for w in ws])
    pitch = -(-codes.shape[2] // 16) * 16
    buf = torch.full((len(ws), codes.shape[1], pitch + 16), 0x7F, dtype=torch.uint8, device=DEV)
    buf[:, :, :codes.shape[2]] = codes
    exps = torch.stack([_dev_exps(w[1]) for w in ws])
    ebuf = torch.full((len(ws), exps.shape[1], -(-exps.shape[2] // 4) * 4 + 4), 255, dtype=torch.uint8, device=DEV)
    ebuf[:, :, :exps.shape[2]] = exps
    stack = [None if ws[0][i] is None else torch.stack([_dev(w[i]) for w in ws]) for i in (2, 3)]
    return buf.view(torch.float8_e4m3fn)[:, :, :codes.shape[2]], ebuf[:, :, :exps.shape[2]], *stack


def _z_tol(mag, k):
    return (k / 32 + 32) * 2.0 ** -22 * mag


def _check16(out, want, tol):
    half = 2.0 ** -25 if out.dtype == torch.float16 else 1e-30
    got = out.double().cpu().numpy()
    worst = np.max(np.abs(got - want) / (ULP[out.dtype] * np.abs(want) + tol + half), initial=0.0)
    assert worst <= 1, worst


def _check_codes(codes, exps, want, tol):
    """Codes [rows, n] and exponents against values that may be off by tol before they are rounded."""
    c, e = SO.decode(_np(codes)), _np(exps).astype(int) - 127
    rows, n = want.shape
    nb = -(-n // 128)
    pad = np.zeros((rows, nb * 128 - n))
    w, t = np.concatenate([want, pad], 1).reshape(rows, nb, 128), np.concatenate([tol, pad], 1).reshape(rows, nb, 128)
    lo = np.vectorize(SO.block_exponent)(np.maximum(np.abs(w) - t, 0).max(2))
    hi = np.vectorize(SO.block_exponent)((np.abs(w) + t).max(2))
    assert (lo <= e).all() and (e <= hi).all()
    scale = np.repeat(2.0 ** e, 128, 1)[:, :n]
    worst = np.max(np.abs(c * scale - want) / (2.0 ** -4 * np.abs(want) + 2.0 ** -10 * scale + 1.0625 * tol), initial=0.0)
    assert worst <= 1, worst


def _want_linear(a, ae, w, ra, act, r, k):
    z, mag = SO.linear(a, ae, w[0], w[1], ra, w[2], w[3])
    tol = 1.13 * _z_tol(mag, k) + 2.0 ** -20 * np.abs(z)
    x = SO.activate(z, act)
    return (x, tol) if r is None else (x + r, tol + 2.0 ** -23 * (np.abs(x) + np.abs(r)))


def _want_gated(a, ae, gate, up, ra, act, k):
    g, gm = SO.linear(a, ae, gate[0], gate[1], ra, gate[2], gate[3])
    u, um = SO.linear(a, ae, up[0], up[1], ra, up[2], up[3])
    x = SO.activate(g, act)
    gt, ut = 1.13 * _z_tol(gm, k) + 2.0 ** -20 * np.abs(g), _z_tol(um, k)
    return x * u, gt * np.abs(u) + ut * np.abs(x) + gt * ut + 2.0 ** -23 * np.abs(x * u) + 1e-37


SIZES = [(1, 1, 1), (1, 128, 128), (3, 130, 200), (16, 256, 512), (17, 257, 1000), (1, 513, 4096), (8, 128, 11008), (33, 384, 640),
         (64, 100, 129), (127, 129, 257), (130, 640, 384), (255, 500, 700), (257, 1024, 1152), (300, 2000, 96), (513, 300, 4112),
         (2, 64, 28672), (48, 128, 16)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype,act,bias,residual", [("bf16", None, False, True), ("f16", "gelu", True, False), ("bf16", "silu", True, True),
                                                     ("f16", "relu", False, False)])
def test_linear(m, n, k, dtype, act, bias, residual):
    a, ae = _fp8_matrix(m + k, m, k, 1, 0.5)
    w = _weights(n + k, n, k, bias=bias)
    ra = np.random.default_rng(7).uniform(0.1, 1, m).astype(np.float32)
    r = _randn(8, m, n, dtype=dtype) if residual else None
    want, tol = _want_linear(a, ae, w, ra, act, None if r is None else r.double().numpy(), k)
    codes, exps, rw, b = _on_dev(w)
    out = gptq.fp8_linear(_dev_codes(a), _dev_exps(ae), codes, exps, _dev(ra), rw, b, act, None if r is None else _padded(r, n % 3),
                          out_dtype=DT[dtype])
    assert out.dtype == DT[dtype]
    _check16(out, want, tol)


@pytest.mark.parametrize("m,n,k", [(1, 200, 512), (40, 300, 1500), (300, 257, 384)])
def test_linear_onto_its_residual_in_a_wider_buffer_and_again(m, n, k):
    a, ae = _fp8_matrix(1, m, k, 1, 0.5)
    w = _weights(2, n, k, scale=False)
    args = (_dev_codes(a), _dev_exps(ae), *_on_dev(w)[:2])
    for pad in (1, 4):
        r = _randn(3, m, n + 5, dtype="bf16")
        buf = r.to(DEV)
        want, tol = _want_linear(a, ae, w, None, None, r[:, pad:pad + n].double().numpy(), k)
        out = gptq.fp8_linear(*args, residual=buf[:, pad:pad + n], out=buf[:, pad:pad + n])
        _check16(out, want, tol)
        assert torch.equal(buf[:, :pad].cpu(), r[:, :pad]) and torch.equal(buf[:, pad + n:].cpu(), r[:, pad + n:])
        assert torch.equal(out, gptq.fp8_linear(*args, residual=r[:, pad:pad + n].to(DEV)))


@pytest.mark.parametrize("m", [15, 16, 17, 100, 111, 112, 113, 150, 224, 239, 240, 241, 400, 480, 700])
def test_tiles_of_every_size(m):
    n, k = 130, 300
    a, ae = _fp8_matrix(m, m, k, 1, 0.5)
    w = _weights(1, n, k)
    dev = _on_dev(w)
    want, tol = _want_linear(a, ae, w, None, "relu", None, k)
    _check16(gptq.fp8_linear(_dev_codes(a), _dev_exps(ae), dev[0], dev[1], None, dev[2], act="relu"), want, tol)
    want, tol = _want_gated(a, ae, w, w, None, "silu", k)
    _check_codes(*gptq.fp8_gated(_dev_codes(a), _dev_exps(ae), dev, dev), want, tol)


def test_linear_without_an_epilogue_is_the_product():
    for m, n, k in ((1, 513, 4096), (70, 300, 1500), (515, 1000, 640)):
        a, ae = _fp8_matrix(1, m, k, 1, 0.5)
        w = _on_dev(_weights(2, n, k))
        args = (_dev_codes(a), _dev_exps(ae), w[0], w[1])
        plain = gptq.fp8_matmul(*args, w_scale=w[2]).float()
        # (both within a rounding, and the sums' order, of one value)
        assert torch.allclose(gptq.fp8_linear(*args, w_scale=w[2]).float(), plain, rtol=2.0 ** -7, atol=1e-4 * float(plain.abs().max()))


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("act,bias", [("silu", False), ("gelu", True)])
def test_gated(m, n, k, act, bias):
    a, ae = _fp8_matrix(m + k, m, k, 1, 0.5)
    gate, up = _weights(n + k, n, k, bias=bias), _weights(n + k + 9, n, k, bias=bias)
    ra = np.random.default_rng(7).uniform(0.1, 1, m).astype(np.float32)
    want, tol = _want_gated(a, ae, gate, up, ra, act, k)
    codes, exps = gptq.fp8_gated(_dev_codes(a), _dev_exps(ae), _on_dev(gate), _on_dev(up), _dev(ra), act)
    assert codes.shape == (m, n) and exps.shape == (m, -(-n // 128))
    _check_codes(codes, exps, want, tol)
    again = gptq.fp8_gated(_dev_codes(a), _dev_exps(ae), _on_dev(gate), _on_dev(up), _dev(ra), act)
    assert torch.equal(codes.view(torch.uint8), again[0].view(torch.uint8)) and torch.equal(exps, again[1])


@pytest.mark.parametrize("m", [5, 300])
def test_nan_stays_in_its_row_and_column(m):
    n, k = 200, 400
    a, ae = _fp8_matrix(8, m, k, 1)
    gate, up = _weights(9, n, k), _weights(10, n, k)
    a[3, 77], up[0][150, 399] = 0x7F, 0xFF
    codes, exps = gptq.fp8_gated(_dev_codes(a), _dev_exps(ae), _on_dev(gate), _on_dev(up))
    bad = np.isnan(SO.decode(_np(codes)))
    assert bad[3].all() and bad[:, 150].all() and bad.sum() == n + m - 1
    assert (_np(exps)[3] == 127 + SO.E_MIN).all()
    out = gptq.fp8_linear(_dev_codes(a), _dev_exps(ae), *_on_dev(up)[:2], act="relu").float().cpu().numpy()
    bad = np.isnan(out)
    assert bad[3].all() and bad[:, 150].all() and bad.sum() == n + m - 1


def test_gated_of_products_that_overflow():
    # act(G) * U past fp32's range is not finite: the NaN code, and no part of its block's exponent
    a, ae = np.full((2, 128), 0x7E, np.uint8), np.full((2, 1), 127 + 60, np.uint8)     # 448 * 2^60
    ae[1] = 127
    gate = np.full((3, 128), 0x38, np.uint8), np.full((1, 1), 127, np.uint8), np.array([1, 2.0 ** -70, 0], np.float32), None
    codes, exps = gptq.fp8_gated(_dev_codes(a), _dev_exps(ae), _on_dev(gate), _on_dev(gate), act=None)
    z = 448.0 * 128
    v = SO.decode(_np(codes)) * 2.0 ** (_np(exps).astype(int) - 127)
    assert math.isnan(v[0, 0]) and v[0, 2] == 0 and abs(v[0, 1] / (z * 2.0 ** -10) ** 2 - 1) <= 2.0 ** -4
    assert abs(v[1, 0] / z ** 2 - 1) <= 2.0 ** -4 and v[1, 2] == 0


def test_products_of_no_tokens():
    w = _on_dev(_weights(9, 64, 128))
    a, ae = torch.empty(0, 128, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(0, 4, dtype=torch.uint8, device=DEV)[:, :1]
    assert gptq.fp8_linear(a, ae, w[0], w[1]).shape == (0, 64)
    codes, exps = gptq.fp8_gated(a, ae, w, w)
    assert codes.shape == (0, 64) and exps.shape == (0, 1)
    ids, weights, offsets, order = gptq.moe_route(torch.empty(0, 5, device=DEV), 2)
    assert ids.shape == (0, 2) and offsets.tolist() == [0] * 6 and order.shape == (0,)
    experts = _experts_on_dev([_weights(9, 64, 128)] * 5)
    codes, exps = gptq.fp8_experts_gated(a, ae, experts, experts, offsets, order, 2)
    assert codes.shape == (0, 64)
    assert gptq.moe_combine(torch.empty(0, 9, device=DEV), weights).shape == (0, 9)


# ---------------------------------------------------------------------------------------
# Routing
# ---------------------------------------------------------------------------------------

def _check_route(logits, top_k, bias=None, **kw):
    """Against the oracle; logits on the host in the type that is handed over."""
    got = gptq.moe_route(logits.to(DEV), top_k, None if bias is None else bias.to(DEV), **kw)
    if kw.get("groups", 1) == 1:
        kw = {k: v for k, v in kw.items() if k not in ("top_groups", "group_top")}
    else:
        kw = {"group_top": 2, "top_groups": kw["groups"], **kw}
    ids, weights, offsets, order = SO.route(logits.double().numpy(), top_k, None if bias is None else bias.double().numpy(), **kw)
    np.testing.assert_array_equal(got[0].cpu().numpy(), ids)
    np.testing.assert_allclose(got[1].cpu().numpy(), weights, rtol=2.0 ** -17, atol=1e-37)
    np.testing.assert_array_equal(got[2].cpu().numpy(), offsets)
    np.testing.assert_array_equal(got[3].cpu().numpy(), order)
    return got


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (1, 64, 6), (2, 7, 7), (5, 32, 32), (31, 60, 4), (32, 256, 8), (33, 256, 8),
                                                  (1, 300, 5), (70, 512, 10), (9, 1024, 32), (333, 160, 6), (1000, 33, 3), (2049, 128, 2),
                                                  (5000, 8, 2), (40000, 16, 3)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_route(tokens, experts, top_k, dtype):
    logits = (2 * _randn(1, tokens, experts)).to(DT[dtype])     # 16-bit logits have equals
    _check_route(logits, top_k)
    bias = 0.2 * _randn(2, experts)
    if tokens <= 5000:
        _check_route(logits, top_k, scores="sigmoid", renormalize=False, scale=2.5)
        _check_route(logits, top_k, bias=bias, scores="sigmoid", scale=0.5)
        _check_route(logits, top_k, bias=0.01 * bias, renormalize=False)


@pytest.mark.parametrize("tokens,experts,groups,top_groups,group_top,top_k", [
    (1, 8, 2, 1, 1, 4), (17, 64, 8, 3, 2, 6), (333, 160, 8, 3, 1, 6), (1500, 256, 8, 4, 2, 8), (40, 96, 32, 5, 2, 15), (3, 30, 30, 7, 1, 7),
    (20, 1024, 4, 2, 2, 9), (50, 45, 5, 5, 2, 3)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_route_by_groups(tokens, experts, groups, top_groups, group_top, top_k, scores):
    logits = 1.5 * _randn(3, tokens, experts)
    for bias in (None, 0.1 * _randn(4, experts)):
        _check_route(logits, top_k, bias, scores=scores, groups=groups, top_groups=top_groups, group_top=group_top)


def test_route_of_equals_takes_the_lowest_index():
    logits = torch.zeros(70, 100)
    got = _check_route(logits, 5)
    assert (got[0].cpu() == torch.arange(5)).all()
    _check_route(logits, 5, torch.zeros(100), scores="sigmoid")
    _check_route(logits, 5, torch.zeros(100), groups=10, top_groups=3, group_top=2)
    logits[:, 50:] = -0.0
    _check_route(logits, 7)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_route_where_fp32_does_not_tell(scores):
    # choices within 1e-9 of one another: the bias makes up for the score but for a little
    rng = np.random.default_rng(5)
    x = rng.standard_normal((200, 64)).astype(np.float32)
    s = 1 / (1 + np.exp(-x[0].astype(np.float64))) if scores == "sigmoid" else np.exp(x[0].astype(np.float64)) / np.exp(x[0].astype(np.float64)).sum()
    x[:] = x[0]
    bias = (0.75 - s).astype(np.float32)                          # what rounding the bias leaves is what decides
    _check_route(torch.from_numpy(x), 8, torch.from_numpy(bias), scores=scores)
    _check_route(torch.from_numpy(x), 6, torch.from_numpy(bias), scores=scores, groups=8, top_groups=3, group_top=2)
    # saturated: the same in fp32, not in fp64
    y = torch.linspace(17, 30, 64).repeat(3, 1).flip(1)
    _check_route(y, 8, torch.zeros(64), scores="sigmoid")


@pytest.mark.parametrize("experts,groups", [(64, 8), (32, 8), (256, 8), (16, 8), (128, 32), (45, 5), (64, 2), (300, 4)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_route_between_groups_that_are_equal_or_nearly(experts, groups, scores, group_top):
    # every group has the same logits in an order of its own; the bias tells them apart by 1e-9, or not at all
    rng = np.random.default_rng(experts + groups)
    size = experts // groups
    x = np.stack([np.concatenate([rng.permutation(v) for _ in range(groups)]) for v in rng.standard_normal((60, size))])
    logits = torch.from_numpy(x.astype(np.float32))
    kw = dict(scores=scores, groups=groups, top_groups=max(1, groups // 2), group_top=min(group_top, size))
    top_k = min(4, size * kw["top_groups"])
    _check_route(logits, top_k, **kw)
    _check_route(logits, top_k, torch.zeros(experts), **kw)
    _check_route(logits, top_k, torch.from_numpy((1e-9 * rng.standard_normal(experts)).astype(np.float32)), **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kw", [dict(), dict(scores="sigmoid"), dict(groups=4, top_groups=2, group_top=2), dict(renormalize=False)])
def test_route_masks(dtype, kw):
    lowest = torch.finfo(DT[dtype]).min
    logits = _randn(6, 80, 24).to(DT[dtype])
    logits[0, :] = -math.inf
    logits[1, :] = math.nan
    logits[2, 3:] = -math.inf                                      # three are left
    logits[3, ::2] = math.nan
    logits[4, :] = lowest
    logits[5, 1:] = lowest
    logits[6, 5], logits[6, 7] = math.inf, math.inf
    logits[7, :20] = -math.inf
    logits[9, :] = torch.finfo(DT[dtype]).max if dtype == "f16" else 1e30
    logits[10:60] = -math.inf                                      # padding
    _check_route(logits, 5, **kw)
    bias = 0.1 * _randn(7, 24)
    bias[4], bias[5] = math.nan, math.inf
    _check_route(logits, 5, bias, **kw)
    if dtype != "f16":
        _check_route(torch.where(torch.isfinite(logits), logits * 0 - 90 - 3 * _randn(8, 80, 24).to(DT[dtype]), logits), 4, **kw)


@pytest.mark.parametrize("mask", [-math.inf, math.nan])
@pytest.mark.parametrize("by", ["bias", "logit"])
@pytest.mark.parametrize("tokens", [1, 70])
def test_route_with_an_expert_left_out_of_the_choice_or_of_the_sum(mask, by, tokens):
    """Weights written out: a bias leaves an expert out of the choice alone, a logit out of the softmax's sum too."""
    logits, bias = torch.tensor([[1.0, 2.0, 3.0]]).repeat(tokens, 1), torch.zeros(3)
    (bias if by == "bias" else logits[0])[2] = mask
    ids, weights, offsets, _ = gptq.moe_route(logits.to(DEV), 2, bias.to(DEV), renormalize=False)
    assert ids[0].tolist() == [1, 0] and (by == "logit" or offsets.tolist() == [0, tokens, 2 * tokens, 2 * tokens])
    want = [0.24472847105479764, 0.09003057317038045] if by == "bias" else [0.7310585786300049, 0.2689414213699951]
    np.testing.assert_allclose(weights[0].cpu().numpy(), want, rtol=2.0 ** -20)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts", [24, 60, 256])
def test_route_by_biases_of_any_size(scores, experts):
    """Biases up to the largest numbers of the type, whose sums in a group pass them; masks by its lowest."""
    logits = _randn(11, 40, experts)
    big = torch.finfo(torch.float32).max
    rng = np.random.default_rng(experts)
    for values in ([-big, 0.0, 0.1], [-big, -0.9 * big, -0.7 * big, -0.8 * big], [big, 0.9 * big, 0.7 * big, 0.8 * big], [-big, big], [-big],
                   [1e30, 1.1e30, -1e30], [1e-40, -1e-40, 0.0]):
        bias = torch.from_numpy(rng.choice(np.array(values, np.float32), experts))
        _check_route(logits, 3, bias, scores=scores)
        for groups, top in ((4, 2), (12 if experts < 256 else 32, 3)):
            for group_top in (1, 2):
                _check_route(logits, 3, bias, scores=scores, groups=groups, top_groups=top, group_top=group_top)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups", [(8, 4), (64, 32), (45, 5), (96, 8)])
@pytest.mark.parametrize("uneven", [False, True])
def test_route_by_groups_whose_sums_cancel(scores, experts, groups, uneven):
    """The two largest of a group with biases of opposite signs: their sum is small, what rounding them leaves is not."""
    rng = np.random.default_rng(experts + uneven)
    logits = torch.from_numpy((1.5 * rng.standard_normal((1500, experts))).astype(np.float32))
    for size in (1e2, 1e3, 1e4, 1e5, 1e6):
        of_group = size * (3e-3 ** rng.random(groups) if uneven else np.ones(groups))
        bias = np.repeat(-of_group[:, None], experts // groups, 1)
        bias[:, 0] = of_group
        _check_route(logits, 2, torch.from_numpy(bias.reshape(-1).astype(np.float32)), scores=scores, groups=groups, top_groups=1, group_top=2)


def test_route_of_a_view_and_on_another_stream():
    logits = _randn(9, 100, 70)
    wide = torch.full((100, 90), math.nan, device=DEV)
    wide[:, 3:73] = logits.to(DEV)
    want = [t.cpu() for t in gptq.moe_route(logits.to(DEV), 4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gptq.moe_route(wide[:, 3:73], 4, stream=side)
    side.synchronize()
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))


# ---------------------------------------------------------------------------------------
# Experts
# ---------------------------------------------------------------------------------------

def _routes(seed, tokens, experts, top_k, dropped=False, favour=None):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((tokens, experts))
    if favour is not None:
        x[:, favour] += 100
    ids = np.argsort(-x, 1)[:, :top_k].astype(np.int32)
    if dropped:
        ids[rng.random(ids.shape) < 0.3] = -1
    return (ids, *SO.plan(ids, experts))


EXPERTS = [(1, 8, 2, 200, 300), (1, 4, 4, 128, 128), (3, 16, 1, 130, 257), (7, 5, 5, 96, 640), (40, 64, 6, 64, 200), (130, 3, 2, 384, 512),
           (300, 2, 1, 129, 96), (513, 8, 3, 100, 384), (64, 1, 1, 257, 129), (700, 40, 4, 256, 128)]


@pytest.mark.parametrize("tokens,experts,top_k,n,k", EXPERTS)
@pytest.mark.parametrize("kind", ["spread", "dropped", "one"])
def test_experts_gated(tokens, experts, top_k, n, k, kind):
    ids, offsets, order = _routes(tokens, tokens, experts, top_k, kind == "dropped", experts // 2 if kind == "one" else None)
    a, ae = _fp8_matrix(tokens + k, tokens, k, 1, 0.5)
    ra = np.random.default_rng(7).uniform(0.1, 1, tokens).astype(np.float32)
    bias = kind == "dropped"
    gate, up = [_weights(10 + i, n, k, bias=bias) for i in range(experts)], [_weights(500 + i, n, k, bias=bias) for i in range(experts)]
    codes, exps = gptq.fp8_experts_gated(_dev_codes(a), _dev_exps(ae), _experts_on_dev(gate), _experts_on_dev(up), _dev(offsets), _dev(order),
                                         top_k, _dev(ra), "silu")
    assert codes.shape == (tokens * top_k, n) and exps.shape == (tokens * top_k, -(-n // 128))
    for e in range(experts):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            t = order[lo:hi] // top_k
            want, tol = _want_gated(a[t], ae[t], gate[e], up[e], ra[t], "silu", k)
            _check_codes(codes[lo:hi], exps[lo:hi], want, tol)


def test_experts_of_every_second_matrix():
    n, k, tokens = 130, 300, 40
    ws = [_weights(10 + i, n, k, bias=True) for i in range(8)]
    stack = _experts_on_dev(ws)
    some = (stack[0][1::2], stack[1][1::2], stack[2][1::2].contiguous(), stack[3][1::2].contiguous())
    alone = _experts_on_dev(ws[1::2])
    _, offsets, order = _routes(1, tokens, 4, 2)
    a, ae = _fp8_matrix(2, tokens, k, 1, 0.5)
    args = (_dev(offsets), _dev(order))
    got = gptq.fp8_experts_gated(_dev_codes(a), _dev_exps(ae), some, some, *args, 2)
    want = gptq.fp8_experts_gated(_dev_codes(a), _dev_exps(ae), alone, alone, *args, 2)
    assert np.array_equal(_np(got[0]), _np(want[0])) and np.array_equal(_np(got[1]), _np(want[1]))
    rows = (_dev_codes(np.repeat(a, 2, 0)), _dev_exps(np.repeat(ae, 2, 0)))
    assert torch.equal(gptq.fp8_experts(*rows, *some[:2], *args, some[2], some[3]), gptq.fp8_experts(*rows, *alone[:2], *args, alone[2], alone[3]))


@pytest.mark.parametrize("n", [1, 100])
def test_weights_of_one_row_of_blocks_in_any_pitch(n):
    k, experts, tokens = 300, 4, 20
    a, ae = _fp8_matrix(2, tokens, k, 1, 0.5)
    A = _dev_codes(a), _dev_exps(ae)
    ws = [_weights(10 + i, n, k) for i in range(experts)]
    codes, exps, scale, _ = _experts_on_dev(ws)
    _, offsets, order = _routes(1, tokens, experts, 1)
    plan = _dev(offsets), _dev(order)

    def call(c, e):
        return gptq.fp8_experts(*A, c, e, *plan, scale)

    want, one = call(codes, exps), gptq.fp8_linear(*A, codes[0], exps[0], w_scale=scale[0])
    # the step from a matrix's only row to the next has no meaning: it may pass the one between matrices
    across = torch.full((1, experts, 8), 255, dtype=torch.uint8, device=DEV).transpose(0, 1)[:, :, :3].copy_(exps)
    assert across.stride(1) > across.stride(0) and torch.equal(call(codes, across), want)
    if n == 1:
        rows = torch.zeros(1, experts, 320, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).transpose(0, 1)[:, :, :k]
        rows.view(torch.uint8).copy_(codes.view(torch.uint8))
        assert rows.stride(1) > rows.stride(0) and torch.equal(call(rows, exps), want)
    # exponents that end with their storage, as a clone of one row does
    short = torch.full((4 * experts - 1,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(call(codes, short.as_strided((experts, 1, 3), (4, 3, 1)).copy_(exps)), want)
    alone = exps[0].clone()
    assert alone.untyped_storage().nbytes() == 3 and torch.equal(gptq.fp8_linear(*A, codes[0], alone, w_scale=scale[0]), one)
    w = codes[0], exps[0], scale[0]
    for m in (1, tokens):
        x, xe = A[0][:m], A[1][:m]
        got, again = (gptq.fp8_gated(x, t, (w[0], u, w[2]), (w[0], u, w[2])) for t, u in ((xe, w[1]), (xe.clone() if m == 1 else xe, alone)))
        assert np.array_equal(_np(got[0]), _np(again[0])) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("tokens", [15, 16, 17, 31, 48, 65, 80, 96, 97, 104, 111, 112, 113, 150, 220, 224, 240, 241, 330, 336, 448, 670, 1000])
def test_experts_tiles_of_every_size(tokens):
    """One expert of `tokens` rows and a second of a few: tiles of all sizes, and rows at every place in them."""
    n, k, few = 130, 300, 5
    a, ae = _fp8_matrix(tokens, tokens + few, k, 1, 0.5)
    order = np.random.default_rng(tokens).permutation(tokens + few).astype(np.int32)
    order[:tokens].sort()
    order[tokens:].sort()
    offsets = np.array([0, tokens, tokens + few], np.int32)
    ws = [_weights(1, n, k), _weights(2, n, k)]
    dev = _experts_on_dev(ws)
    codes, exps = gptq.fp8_experts_gated(_dev_codes(a), _dev_exps(ae), dev, dev, _dev(offsets), _dev(order), 1)
    out = gptq.fp8_experts(_dev_codes(a), _dev_exps(ae), dev[0], dev[1], _dev(offsets), _dev(order), dev[2])
    for e, (lo, hi) in enumerate(((0, tokens), (tokens, tokens + few))):
        t = order[lo:hi]
        want, tol = _want_gated(a[t], ae[t], ws[e], ws[e], None, "silu", k)
        _check_codes(codes[lo:hi], exps[lo:hi], want, tol)
        want, tol = _want_linear(a[lo:hi], ae[lo:hi], ws[e], None, None, None, k)
        _check16(out[torch.from_numpy(t.astype(np.int64)).to(DEV)], want, tol)


@pytest.mark.parametrize("tokens,experts,top_k,n,k", EXPERTS)
@pytest.mark.parametrize("kind,dtype,act,bias", [("spread", "bf16", None, False), ("dropped", "f16", None, True), ("one", "bf16", "relu", False)])
def test_experts_out(tokens, experts, top_k, n, k, kind, dtype, act, bias):
    ids, offsets, order = _routes(tokens, tokens, experts, top_k, kind == "dropped", experts // 2 if kind == "one" else None)
    rows = tokens * top_k
    a, ae = _fp8_matrix(tokens + k, rows, k, 1, 0.5)
    w = [_weights(10 + i, n, k, bias=bias) for i in range(experts)]
    codes, exps, scale, b = _experts_on_dev(w)
    buf = torch.full((rows, n + 3), 7.0, dtype=DT[dtype], device=DEV)
    out = gptq.fp8_experts(_dev_codes(a), _dev_exps(ae), codes, exps, _dev(offsets), _dev(order), scale, b, act, out=buf[:, 2:2 + n])
    assert (buf[:, :2] == 7).all() and (buf[:, 2 + n:] == 7).all()
    for e in range(experts):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            want, tol = _want_linear(a[lo:hi], ae[lo:hi], w[e], None, act, None, k)
            _check16(out[torch.from_numpy(order[lo:hi].astype(np.int64)).to(DEV)], want, tol)
    unnamed = np.setdiff1d(np.arange(rows), order[:offsets[-1]])
    assert (out[torch.from_numpy(unnamed).to(DEV)] == 7).all()


def test_experts_with_a_plan_that_makes_no_sense():
    # offsets out of range or falling, orders that name nothing: no write outside, the sound part is right
    tokens, experts, top_k, n, k = 40, 6, 2, 200, 256
    rows = tokens * top_k
    a, ae = _fp8_matrix(1, tokens, k, 1, 0.5)
    w = _experts_on_dev([_weights(10 + i, n, k) for i in range(experts)])
    _, offsets, order = _routes(2, tokens, experts, top_k)
    want, we = gptq.fp8_experts_gated(_dev_codes(a), _dev_exps(ae), w, w, _dev(offsets), _dev(order), top_k)
    bad = order.copy()
    bad[[0, 7, 70]] = -5, 10 ** 9, rows
    for offs in ([0, 10 ** 6, 20, 30, 40, 50, -7], [-20, 5, 5, 90, 95, 60, 10 ** 9], [0, 0, 0, 0, 0, 0, 0], [5, 4, 3, 2, 1, 0, 0]):
        offs = np.array(offs, np.int32)
        codes, exps = gptq.fp8_experts_gated(_dev_codes(a), _dev_exps(ae), w, w, _dev(offs), _dev(bad), top_k)
        out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device=DEV)
        gptq.fp8_experts(_dev_codes(np.repeat(a, 2, 0)), _dev_exps(np.repeat(ae, 2, 0)), w[0], w[1], _dev(offs), _dev(bad), out=out)
    codes, exps = gptq.fp8_experts_gated(_dev_codes(a), _dev_exps(ae), w, w, _dev(offsets), _dev(bad), top_k)
    good = np.setdiff1d(np.arange(rows), [0, 7, 70])
    assert np.array_equal(_np(codes)[good], _np(want)[good]) and np.array_equal(_np(exps)[good], _np(we)[good])
    assert (_np(codes)[[0, 7, 70]] == 0).all()
    gptq.serving_status()


# ---------------------------------------------------------------------------------------
# Combine
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("tokens,top_k,d,pad", [(1, 1, 1, 0), (1, 6, 4096, 0), (3, 2, 130, 1), (33, 8, 1000, 4), (5, 32, 257, 8), (9, 9, 20000, 0),
                                                (1000, 3, 64, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
def test_combine(tokens, top_k, d, pad, dtype, residual):
    y, r = _randn(1, tokens * top_k, d, dtype=dtype), _randn(2, tokens, d, dtype=dtype) if residual else None
    w = torch.softmax(_randn(3, tokens, top_k), -1)
    if top_k > 1:
        w[tokens // 2, 1] = 0
        y[tokens // 2 * top_k + 1] = math.nan                        # not read
    want, mag = SO.combine(y.double().numpy(), w.numpy(), None if r is None else r.double().numpy())
    out = gptq.moe_combine(_padded(y, pad), w.to(DEV), None if r is None else _padded(r, pad))
    tol = (top_k + 1) * 2.0 ** -24 * mag
    if dtype == "f32":
        assert np.max(np.abs(out.double().cpu().numpy() - want) / (tol + 2.0 ** -24 * np.abs(want) + 1e-40)) <= 1
    else:
        _check16(out, want, tol)
    if residual:
        buf = r.to(DEV)
        assert torch.equal(gptq.moe_combine(y.to(DEV), w.to(DEV), buf, out=buf), out) and buf.data_ptr() != out.data_ptr()


# ---------------------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("tokens,experts,top_k,d,n", [(1, 8, 2, 256, 200), (50, 8, 2, 256, 200), (300, 16, 4, 384, 130)])
def test_a_block_of_experts(tokens, experts, top_k, d, n):
    """Norm, routing, the experts and their sum, against fp64 on the operands that each step was given."""
    x = _randn(1, tokens, d, dtype="bf16").to(DEV)
    norm = (1 + 0.1 * _randn(2, d)).to(torch.bfloat16).to(DEV)
    router = (_randn(3, experts, d) / math.sqrt(d)).to(DEV)
    gate, up, down = ([_weights(s + i, *shape) for i in range(experts)] for s, shape in ((10, (n, d)), (200, (n, d)), (400, (d, n))))
    codes, exps, rstd, h = gptq.rmsnorm_fp8(x, norm)
    ids, weights, offsets, order = gptq.moe_route(x.float() @ router.t(), top_k, renormalize=False)
    inner, inner_e = gptq.fp8_experts_gated(codes, exps, _experts_on_dev(gate), _experts_on_dev(up), offsets, order, top_k, rstd)
    dw = _experts_on_dev(down)
    out = gptq.moe_combine(gptq.fp8_experts(inner, inner_e, dw[0], dw[1], offsets, order, dw[2]), weights, x)
    gptq.serving_status()
    a = SO.dequantize(_np(codes), _np(exps)) * rstd.double().cpu().numpy()[:, None]
    mats = [[SO.dequantize(w[0], w[1], 128) * w[2].astype(np.float64)[:, None] for w in ws] for ws in (gate, up, down)]
    want = x.double().cpu().numpy()
    branch = np.zeros_like(want)
    for t in range(tokens):
        for j in range(top_k):
            e = int(ids[t, j])
            branch[t] += float(weights[t, j]) * ((SO.activate(a[t] @ mats[0][e].T, "silu") * (a[t] @ mats[1][e].T)) @ mats[2][e].T)
    # the inner rows are rounded to e4m3 (2^-4 of an element at most: 2^-5.3 of the norm, with which the
    # product's error goes), the experts' outputs and the sum to bf16
    got = out.double().cpu().numpy()
    assert np.linalg.norm(got - (want + branch)) <= 2.0 ** -4.3 * np.linalg.norm(branch) + 2.0 ** -8 * np.linalg.norm(want)
