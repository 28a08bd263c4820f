"""The feed-forward operators as programs use them: in graphs, on several streams at once, between guard
bytes, in a layer of experts, and where a device wait runs out."""

import ctypes
import gc
import math
import time

import numpy as np
import pytest
import torch

from oracle import serving_oracle as SO
from post_weight_quantization_03_gb300 import build_lib, decoder, gptq
from tests.test_gpu_canaries import PAT, Guarded
from tests.test_gpu_feed_forward import (_check16, _check_codes, _dev, _experts_on_dev, _on_dev, _routes, _want_gated, _want_linear,
                                         _weights)
from tests.test_gpu_serving import DEV, DT, _dev_codes, _dev_exps, _fp8_matrix, _np, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    gptq.load()
    torch.cuda.init()
    yield
    gc.collect()   # frames of expected errors hold tensors: others' tests look at what is allocated


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _u8(t):
    return t.view(torch.uint8)


class _Block:
    """A block of experts on operands of its own."""

    def __init__(self, seed, tokens, experts, top_k, d, n):
        self.top_k = top_k
        self.x = _randn(seed, tokens, d, dtype="bf16").to(DEV)
        self.norm = (1 + 0.1 * _randn(seed + 1, d)).to(torch.bfloat16).to(DEV)
        self.router = (_randn(seed + 2, experts, d) / math.sqrt(d)).to(DEV)
        self.gate, self.up, self.down = (
            _experts_on_dev([_weights(s + i, *shape) for i in range(experts)]) for s, shape in ((10, (n, d)), (200, (n, d)), (400, (d, n))))

    def __call__(self, stream=None):
        codes, exps, rstd, _ = gptq.rmsnorm_fp8(self.x, self.norm, stream=stream)
        logits = self.x.float() @ self.router.t() if stream is None else self.logits
        ids, w, offsets, order = gptq.moe_route(logits, self.top_k, stream=stream)
        inner = gptq.fp8_experts_gated(codes, exps, self.gate, self.up, offsets, order, self.top_k, rstd, stream=stream)
        y = gptq.fp8_experts(*inner, self.down[0], self.down[1], offsets, order, self.down[2], stream=stream)
        return gptq.moe_combine(y, w, self.x, stream=stream)


@pytest.mark.parametrize("tokens", [1, 20, 300])
def test_a_captured_block_follows_its_inputs(tokens):
    block = _Block(1, tokens, 8, 2, 256, 200)
    other = _randn(50, tokens, 256, dtype="bf16").to(DEV)
    first = block().clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block()
    graph.replay()
    assert torch.equal(out, first)
    before = block.x.clone()
    block.x.copy_(other)
    want = block().clone()
    graph.replay()
    assert torch.equal(out, want) and not torch.equal(out, first)
    block.x.copy_(before)
    graph.replay()
    assert torch.equal(out, first)
    gptq.serving_status()


def test_blocks_on_two_streams_at_once():
    blocks = [_Block(1, 40, 8, 2, 256, 200), _Block(7, 333, 16, 4, 384, 130)]
    want = [b().clone() for b in blocks]
    for b in blocks:
        b.logits = b.x.float() @ b.router.t()
    streams = [torch.cuda.Stream() for _ in blocks]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for i, (b, s) in enumerate(zip(blocks, streams)):
            got[i].append(b(s))
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert all(torch.equal(o, w) for o in outs)
    gptq.serving_status()


class _Few:
    """Products of a few tokens, whose tiles are shared by clusters of CTAs."""

    def __init__(self, seed, m, n, k, experts):
        a, ae = _fp8_matrix(seed, m, k, 1, 0.5)
        self.a = _dev_codes(a), _dev_exps(ae)
        self.w = _on_dev(_weights(seed + 1, n, k))
        self.r = _randn(seed + 2, m, n, dtype="bf16").to(DEV)
        _, offsets, order = _routes(seed, m, experts, 2)
        self.plan = _dev(offsets), _dev(order)
        self.ew = _experts_on_dev([_weights(seed + 3 + i, n, k) for i in range(experts)])
        self.rows = _dev_codes(np.repeat(a, 2, 0)), _dev_exps(np.repeat(ae, 2, 0))

    def __call__(self, stream=None):
        kw = dict(stream=stream)
        return [_u8(t) for t in (
            gptq.fp8_linear(*self.a, *self.w[:2], w_scale=self.w[2], residual=self.r, **kw),
            gptq.fp8_matmul(*self.a, *self.w[:2], w_scale=self.w[2], **kw),
            *gptq.fp8_gated(*self.a, self.w, self.w, **kw),
            *gptq.fp8_experts_gated(*self.a, self.ew, self.ew, *self.plan, 2, **kw),
            gptq.fp8_experts(*self.rows, *self.ew[:2], *self.plan, self.ew[2], **kw))]


def test_products_of_few_tokens_on_three_streams_at_once():
    sets = [_Few(1, 1, 512, 4096, 4), _Few(20, 8, 640, 2048, 8), _Few(40, 3, 130, 8192, 3)]
    want = [[t.clone() for t in s()] for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        got.append((i % 3, sets[i % 3](streams[i % 3])))
    torch.cuda.synchronize()
    for i, outs in got:
        assert all(torch.equal(o, w) for o, w in zip(outs, want[i]))
    gptq.serving_status()


def test_two_graphs_replayed_at_once():
    sets = [_Few(1, 1, 512, 4096, 4), _Few(20, 8, 640, 2048, 8)]
    blocks = [_Block(1, 40, 8, 2, 256, 200), _Block(7, 333, 16, 4, 384, 130)]
    want = [[t.clone() for t in s()] + [b().clone()] for s, b in zip(sets, blocks)]
    graphs, outs = [], []
    for s, b in zip(sets, blocks):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s() + [b()])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(o, w))
    gptq.serving_status()


def test_offsets_that_pass_32_bits():
    """Outputs, token rows and experts' weights of more than 2^31 bytes: what lies past them is right."""
    n, k, m = 4112, 32, 540_000
    w = _on_dev(_weights(3, n, k))
    a, ae = _fp8_matrix(1, 64, k, 1, 0.5)
    last = _dev_codes(a), _dev_exps(ae)
    codes, exps = torch.zeros(m, k, dtype=torch.uint8, device=DEV), torch.full((m, 4), 127, dtype=torch.uint8, device=DEV)
    codes[-64:], exps[-64:, :1] = _u8(last[0]), last[1]
    many = codes.view(torch.float8_e4m3fn), exps[:, :1]
    # (K is one block: the sums of few rows and of many are the same numbers)
    small = gptq.fp8_linear(*last, *w[:2], w_scale=w[2])
    out = gptq.fp8_linear(*many, *w[:2], w_scale=w[2])
    assert torch.equal(out[-64:], small) and not out[:1000].any()
    gptq.fp8_linear(*many, *w[:2], w_scale=w[2], residual=out, out=out)
    small = gptq.fp8_linear(*last, *w[:2], w_scale=w[2], residual=small)
    assert torch.equal(out[-64:], small)
    gptq.moe_combine(out, torch.ones(m, 1, device=DEV), out, out=out)
    assert torch.equal(out[-64:], 2 * small) and not out[:1000].any()
    del out
    c, e = gptq.fp8_gated(*many, w, w)
    c2, e2 = gptq.fp8_gated(*last, w, w)
    assert torch.equal(_u8(c[-64:]), _u8(c2)) and torch.equal(e[-64:], e2)
    # the last of those rows by index
    ws = [_weights(30 + i, 130, n) for i in range(2)]
    order = torch.full((m,), -1, dtype=torch.int32, device=DEV)
    order[:64] = torch.arange(m - 1, m - 65, -1)
    got = gptq.fp8_experts_gated(c, e, _experts_on_dev(ws), _experts_on_dev(ws), _dev(np.array([0, 40, 64], np.int32)), order, 1)
    rows, rows_e = _np(c2)[::-1], _np(e2)[::-1]
    for i, at in ((0, slice(0, 40)), (1, slice(40, 64))):
        _check_codes(got[0][at], got[1][at], *_want_gated(rows[at], rows_e[at], ws[i], ws[i], None, "silu", n))
    del c, e, got, codes, exps, many
    # the last of 700 matrices of 2048 x 2048 bytes
    experts, d = 700, 2048
    stack = torch.zeros(experts, d, d, dtype=torch.uint8, device=DEV)
    stack_e = torch.full((experts, 16, 16), 127, dtype=torch.uint8, device=DEV)
    hw = _weights(5, d, d, scale=False)
    stack[-1], stack_e[-1] = _u8(_dev_codes(hw[0])), _dev_exps(hw[1])
    a, ae = _fp8_matrix(9, 20, d, 1, 0.5)
    offsets = np.zeros(experts + 1, np.int32)
    offsets[-1] = 20
    y = gptq.fp8_experts(_dev_codes(a), _dev_exps(ae), stack.view(torch.float8_e4m3fn), stack_e, _dev(offsets), _dev(np.arange(20, dtype=np.int32)))
    _check16(y, *_want_linear(a, ae, hw, None, None, None, d))
    gptq.serving_status()


@pytest.mark.parametrize("tokens,experts", [(0, 8), (1, 7), (33, 300)])
@pytest.mark.parametrize("inference", [False, True])
def test_outputs_of_a_call_do_not_share_memory(tokens, experts, inference):
    logits = _randn(1, tokens, experts).to(DEV)
    a, ae = _fp8_matrix(2, max(tokens, 1), 300, 1, 0.5)
    w = _on_dev(_weights(3, 130, 300))
    with torch.inference_mode(inference):
        outs = [*gptq.moe_route(logits, 3), *gptq.fp8_gated(_dev_codes(a)[:tokens], _dev_exps(ae)[:tokens], w, w)]
        want = [t.clone() for t in outs]
        for i, t in enumerate(outs):
            _u8(t).fill_(0x11)
            assert all(torch.equal(_u8(x), _u8(y)) for x, y in zip(outs[i + 1:], want[i + 1:]))
        assert [t.is_inference() for t in outs] == [inference] * 6 and not any(t.requires_grad for t in outs)
    assert all((_u8(t) == 0x11).all() for t in outs)
    assert [t.dtype for t in outs] == [torch.int32, torch.float32, torch.int32, torch.int32, torch.float8_e4m3fn, torch.uint8]
    assert [tuple(t.shape) for t in outs] == [(tokens, 3), (tokens, 3), (experts + 1,), (3 * tokens,), (tokens, 130), (tokens, 2)]


def test_calls_repeat():
    a, ae = _fp8_matrix(3, 500, 512, 1, 0.5)
    w = [_weights(10 + i, 384, 512) for i in range(8)]
    _, offsets, order = _routes(4, 500, 8, 2)
    ew = _experts_on_dev(w)
    args = (_dev_codes(a), _dev_exps(ae), ew, ew, _dev(offsets), _dev(order), 2)
    c, e = gptq.fp8_experts_gated(*args)
    for _ in range(5):
        c2, e2 = gptq.fp8_experts_gated(*args)
        assert torch.equal(_u8(c), _u8(c2)) and torch.equal(e, e2)


# ---------------------------------------------------------------------------------------
# Guard bytes
# ---------------------------------------------------------------------------------------

def _struct(w, experts=False):
    codes, exps, scale, bias = w
    st, es = codes.stride(), exps.stride()
    return gptq.Fp8Weights(codes.data_ptr(), st[-2], st[0] if experts else 0, exps.data_ptr(), es[-2], es[0] if experts else 0,
                           None if scale is None else scale.data_ptr(), None if bias is None else bias.data_ptr())


def _ok(st):
    assert st == 0, gptq.gptq_status_str(st)


@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (3, 130, 200), (17, 257, 1000), (130, 640, 384), (300, 1999, 96), (1, 512, 4096)])
def test_products_write_their_rows_alone(m, n, k):
    a, ae = _fp8_matrix(m + k, m, k, 1, 0.5)
    w = _on_dev(_weights(n + k, n, k, bias=True))
    A, AE = _dev_codes(a), _dev_exps(ae)
    ws = gptq.workspace(256, DEV)
    tail = (_p(ws), 256, gptq._stream(None))
    for extra in (0, 3, 4):
        out = Guarded(m * (n + extra) * 2)
        r = _randn(1, m, n + 1, dtype="bf16").to(DEV)
        _ok(gptq.gptq_fp8_linear(_p(A), A.stride(0), _p(AE), AE.stride(0), None, _struct(w), 2, _p(r), n + 1, m, n, k, out.ptr, 1, n + extra,
                                 *tail))
        assert out.intact() and bool((out.view(torch.uint8, (m, (n + extra) * 2))[:, n * 2:] == PAT).all())
        ldc, lde = -(-n // 16) * 16 + 16 * (extra > 0), -(-(-(-n // 128)) // 4) * 4 + 4 * (extra > 0)
        codes, exps = Guarded(m * ldc), Guarded(m * lde)
        _ok(gptq.gptq_fp8_gated(_p(A), A.stride(0), _p(AE), AE.stride(0), None, _struct(w), _struct(w), 2, m, n, k, codes.ptr, ldc, exps.ptr,
                                lde, *tail))
        assert codes.intact() and exps.intact()
        assert bool((codes.view(torch.uint8, (m, ldc))[:, n:] == PAT).all())
        assert bool((exps.view(torch.uint8, (m, lde))[:, -(-n // 128):] == PAT).all())


@pytest.mark.parametrize("tokens,experts,top_k,n,k", [(1, 4, 2, 200, 300), (40, 16, 4, 130, 256), (300, 3, 1, 257, 128)])
def test_experts_write_their_rows_alone(tokens, experts, top_k, n, k):
    rows = tokens * top_k
    _, offsets, order = _routes(1, tokens, experts, top_k, dropped=True)
    a, ae = _fp8_matrix(2, rows, k, 1, 0.5)
    w = _experts_on_dev([_weights(10 + i, n, k) for i in range(experts)])
    A, AE, O, R = _dev_codes(a), _dev_exps(ae), _dev(offsets), _dev(order)
    ws = gptq.workspace(256, DEV)
    tail = (_p(ws), 256, gptq._stream(None))
    ldc, lde, nb = -(-n // 16) * 16 + 16, -(-(-(-n // 128)) // 4) * 4 + 4, -(-n // 128)
    codes, exps, out = Guarded(rows * ldc), Guarded(rows * lde), Guarded(rows * (n + 3) * 2)
    _ok(gptq.gptq_fp8_experts_gated(_p(A), A.stride(0), _p(AE), AE.stride(0), None, _struct(w, True), _struct(w, True), 2, experts, _p(O), _p(R),
                                    top_k, tokens, n, k, codes.ptr, ldc, exps.ptr, lde, *tail))
    _ok(gptq.gptq_fp8_experts(_p(A), A.stride(0), _p(AE), AE.stride(0), _struct(w, True), 0, experts, _p(O), _p(R), rows, n, k, out.ptr, 1, n + 3,
                              *tail))
    used = int(offsets[-1])
    assert codes.intact() and exps.intact() and out.intact()
    c, e = codes.view(torch.uint8, (rows, ldc)), exps.view(torch.uint8, (rows, lde))
    assert bool((c[:, n:] == PAT).all()) and bool((c[used:] == PAT).all()) and bool((e[:, nb:] == PAT).all()) and bool((e[used:] == PAT).all())
    o = out.view(torch.uint8, (rows, (n + 3) * 2))
    unnamed = torch.from_numpy(np.setdiff1d(np.arange(rows), order[:used])).to(DEV)
    assert bool((o[:, n * 2:] == PAT).all()) and bool((o[unnamed] == PAT).all())


def _bad_plans(rng, experts, rows):
    """Offsets that fall, are out of range or both."""
    sorted_ = np.sort(rng.integers(0, rows + 1, experts + 1))
    wild = sorted_.copy()
    wild[rng.integers(0, experts + 1, 2)] = 2 ** 31 - 1, -2 ** 31
    yield from (np.zeros(experts + 1), sorted_[::-1], sorted_ + rows // 3, sorted_ - rows // 3, wild, rng.integers(-rows, 2 * rows, experts + 1),
                np.where(np.arange(experts + 1) < experts, sorted_, -7))


@pytest.mark.parametrize("tokens,experts,top_k,n,k", [(1, 4, 2, 200, 300), (40, 6, 2, 200, 256), (300, 40, 2, 130, 384), (400, 3, 3, 257, 128)])
def test_experts_by_a_plan_that_makes_no_sense(tokens, experts, top_k, n, k):
    """Offsets are limited to the rows there are and read as increasing; an order that names no row of A stands for
    zeros, one that names no row of the output for none.  What no position names stays as it was."""
    rows = tokens * top_k
    rng = np.random.default_rng(tokens)
    hw = [_weights(10 + i, n, k) for i in range(experts)]
    w = _experts_on_dev(hw)
    a, ae = _fp8_matrix(2, tokens, k, 1, 0.5)
    x, xe = _fp8_matrix(3, rows, k, 1, 0.5)
    A, AE, X, XE = _dev_codes(a), _dev_exps(ae), _dev_codes(x), _dev_exps(xe)
    ws = gptq.workspace(256, DEV)
    tail = (_p(ws), 256, gptq._stream(None))
    ldc, lde, nb = -(-n // 16) * 16 + 16, -(-(-(-n // 128)) // 4) * 4 + 4, -(-n // 128)
    for offsets in _bad_plans(rng, experts, rows):
        offsets = offsets.astype(np.int32)
        order = rng.permutation(rows).astype(np.int32)
        for at, bad in zip(rng.permutation(rows), (-5, 10 ** 9, rows, -2 ** 31, 2 ** 31 - 1)):
            order[at] = bad
        O, R = _dev(offsets), _dev(order)
        codes, exps, out = Guarded(rows * ldc), Guarded(rows * lde), Guarded(rows * (n + 3) * 2)
        _ok(gptq.gptq_fp8_experts_gated(_p(A), A.stride(0), _p(AE), AE.stride(0), None, _struct(w, True), _struct(w, True), 2, experts, _p(O),
                                        _p(R), top_k, tokens, n, k, codes.ptr, ldc, exps.ptr, lde, *tail))
        _ok(gptq.gptq_fp8_experts(_p(X), X.stride(0), _p(XE), XE.stride(0), _struct(w, True), 0, experts, _p(O), _p(R), rows, n, k, out.ptr, 1,
                                  n + 3, *tail))
        assert codes.intact() and exps.intact() and out.intact()
        c, e = codes.view(torch.uint8, (rows, ldc)), exps.view(torch.uint8, (rows, lde))
        o = out.view(torch.uint8, (rows, (n + 3) * 2))
        assert bool((c[:, n:] == PAT).all()) and bool((e[:, nb:] == PAT).all()) and bool((o[:, n * 2:] == PAT).all())
        begins = np.maximum.accumulate(np.clip(offsets.astype(np.int64), 0, rows))
        none = np.r_[0:begins[0], begins[-1]:rows]
        assert bool((c[_dev(none)] == PAT).all()) and bool((e[_dev(none)] == PAT).all())
        named = order[begins[0]:begins[-1]]
        unnamed = np.setdiff1d(np.arange(rows), named)
        assert bool((o[_dev(unnamed)] == PAT).all())
        values = o[:, :n * 2].contiguous().view(torch.bfloat16)
        for i in range(experts):
            at = np.arange(begins[i], begins[i + 1])
            if len(at) == 0:
                continue
            token = order[at].astype(np.int64) // top_k
            there = (token >= 0) & (token < tokens)
            token = np.where(there, token, 0)
            z = np.where(there[:, None], a[token], 0).astype(np.uint8)
            _check_codes(c[_dev(at)][:, :n].view(torch.float8_e4m3fn), e[_dev(at)][:, :nb], *_want_gated(z, ae[token], hw[i], hw[i], None, "silu", k))
            at = at[(order[at] >= 0) & (order[at] < rows)]
            if len(at):
                want, tol = _want_linear(x[at], xe[at], hw[i], None, None, None, k)
                _check16(values[_dev(order[at].astype(np.int64))], want, tol)
    gptq.serving_status()


@pytest.mark.parametrize("tokens,experts,top_k,d", [(1, 7, 3, 5), (33, 100, 8, 130), (3000, 17, 2, 64), (9000, 64, 4, 8)])
def test_routing_and_combine_write_their_rows_alone(tokens, experts, top_k, d):
    logits = _randn(1, tokens, experts).to(DEV)
    ids, w = Guarded(tokens * top_k * 4), Guarded(tokens * top_k * 4)
    offsets, order = Guarded((experts + 1) * 4), Guarded(tokens * top_k * 4)
    need = gptq.gptq_moe_route_workspace_bytes(tokens, experts, top_k)
    ws = Guarded(need)
    _ok(gptq.gptq_moe_route(_p(logits), 2, experts, tokens, experts, top_k, None, 1, 1, 1, 1, 1, 1.0, ids.ptr, w.ptr, offsets.ptr, order.ptr,
                            ws.ptr, need, gptq._stream(None)))
    assert all(g.intact() for g in (ids, w, offsets, order, ws))
    y, out = _randn(2, tokens * top_k, d, dtype="bf16").to(DEV), Guarded(tokens * (d + 3) * 2)
    _ok(gptq.gptq_moe_combine(_p(y), 1, d, tokens, top_k, d, w.ptr, None, 0, out.ptr, d + 3, gptq._stream(None)))
    assert out.intact() and bool((out.view(torch.uint8, (tokens, (d + 3) * 2))[:, d * 2:] == PAT).all())


# ---------------------------------------------------------------------------------------
# Waits that run out
# ---------------------------------------------------------------------------------------

TIMEOUT, BUDGET = 4, 50_000_000


@pytest.mark.parametrize("experts,tokens,top_k,n,k", [(0, 1, 1, 256, 4096), (0, 300, 1, 2000, 512), (4, 1, 2, 256, 2048), (8, 500, 2, 640, 1024)])
@pytest.mark.parametrize("copy", [0, 3])
def test_a_wait_that_gives_up(experts, tokens, top_k, n, k, copy):
    rows = tokens * top_k
    a, ae = _fp8_matrix(1, tokens, k, 1, 0.5)
    A, AE = _dev_codes(a), _dev_exps(ae)
    w = _experts_on_dev([_weights(10 + i, n, k) for i in range(experts)]) if experts else _on_dev(_weights(10, n, k))
    _, offsets, order = _routes(1, tokens, max(experts, 1), top_k) if experts else (None, None, None)
    O, R = (_dev(offsets), _dev(order)) if experts else (None, None)
    ws = gptq.workspace(256, DEV)
    codes = torch.zeros(rows, -(-n // 16) * 16, dtype=torch.uint8, device=DEV)
    exps = torch.zeros(rows, -(-n // 512) * 4, dtype=torch.uint8, device=DEV)

    def regular():
        if experts:
            return gptq.fp8_experts_gated(A, AE, w, w, O, R, top_k, ws=ws)
        return gptq.fp8_gated(A, AE, w, w, ws=ws)

    want = regular()
    gptq.serving_status()
    t = time.monotonic()
    st = gptq.gptq_debug_fp8_gated_lost_copy(_p(A), A.stride(0), _p(AE), AE.stride(0), _struct(w, bool(experts)), _struct(w, bool(experts)), 2,
                                             experts, _p(O), _p(R), top_k, tokens, n, k, _p(codes), codes.stride(0), _p(exps), exps.stride(0),
                                             copy, BUDGET, _p(ws), 256, gptq._stream(None))
    assert st == TIMEOUT and time.monotonic() - t < 5
    with pytest.raises(gptq.GptqError, match="TIMEOUT"):
        gptq.serving_status()
    gptq.serving_status()
    again = regular()
    assert torch.equal(_u8(again[0]), _u8(want[0])) and torch.equal(again[1], want[1])
    assert gptq.gptq_workspace_status(_p(ws), gptq._stream(None)) == 0


# ---------------------------------------------------------------------------------------
# A layer of experts
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("hidden,mlp,experts,routing", [
    (256, 200, 4, dict(top_k=2)), (256, 128, 8, dict(top_k=3, scores="sigmoid", groups=4, top_groups=2, scale=1.5)),
    (512, 96, 12, dict(top_k=1, renormalize=False))])
def test_a_layer_of_experts(hidden, mlp, experts, routing):
    heads, kv_heads, dim = 4, 2, 64
    weights, (n1, n2) = decoder.random_layer(hidden, mlp, heads, kv_heads, dim, experts=experts)
    calib = _randn(3, 2, 160, hidden, dtype="bf16").to(DEV)
    layer = decoder.ExpertsLayer.quantize(weights, n1, n2, calib, heads, kv_heads, 4, routing=routing)
    for codes, exps, scale in layer.experts.values():
        v = codes.float()
        assert codes.shape[0] == experts and torch.equal(v, v.round()) and float(v.abs().max()) <= 15 and bool((exps == 127).all())
    # the feed-forward part on hidden states given to it, against fp32 on the same weights
    h = _randn(4, 90, hidden, dtype="bf16").to(DEV)
    codes, exps, rstd, _ = gptq.rmsnorm_fp8(h, n2, eps=layer.eps)
    got = layer._feed_forward(codes, exps, rstd, h).float()
    w = layer.dequantized()
    g = h.float() * torch.rsqrt(h.float().square().mean(-1, keepdim=True) + layer.eps) * n2.float()
    dense = (torch.nn.functional.silu(g @ w["gate"].t()) * (g @ w["up"].t())) @ w["down"].t()
    branch = dense + decoder.experts_reference(w, routing, g)
    # operands of e4m3 on the way: 2^-5.3 of the norm each for the normed rows (which count twice, in both
    # factors) and the inner ones
    err = float((got - (h.float() + branch)).norm())
    assert err <= 3 ** 0.5 * 2 ** -5.3 * float(branch.norm()) + 2.0 ** -8 * float(h.float().norm())
    # a whole layer in steps
    seqs, total = 2, 70
    x = _randn(5, seqs, total, hidden, dtype="bf16").to(DEV)
    cache = gptq.kv8_cache(seqs * 2, kv_heads, dim)
    table = torch.arange(seqs * 2, dtype=torch.int32, device=DEV).view(seqs, 2)
    at = 0
    for new in (50, 1, 1, 18):
        start = torch.full((seqs,), at, dtype=torch.int32, device=DEV)
        out = layer.step(x[:, at:at + new], cache, table, start, start + new)
        assert out.shape == (seqs, new, hidden) and bool(torch.isfinite(out.float()).all())
        at += new
    gptq.serving_status()


def test_the_decoder_command_runs_experts(capsys):
    decoder.main(["--hidden", "256", "--mlp", "256", "--heads", "4", "--dim", "64", "--prompt", "40", "--tokens", "3", "--experts", "4"])
    assert "quantized weights" in capsys.readouterr().out
