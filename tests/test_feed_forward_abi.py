"""Refusals of the feed-forward calls: arguments that fail validation return before the GPU is touched
(so this runs without one), and the helpers raise for what the kernels would read as something else."""

import ctypes
import gc

import pytest

from post_weight_quantization_03_gb300 import build_lib, gptq

P = ctypes.c_void_p
AT = 256 * 1024
FAKE, ODD = P(AT), P(AT + 8)   # never dereferenced
INV, UNSUP, WS = 1, 6, 7


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    gptq.load()
    yield
    gc.collect()   # frames of expected errors hold tensors: others' tests look at what is allocated


def _call(fn, base, **kw):
    a = dict(base)
    assert set(kw) <= set(a)
    a.update(kw)
    return fn(*a.values())


def _w(**kw):
    a = dict(codes=AT, ld=304, next_codes=304 * 200, exps=AT, ld_exps=4, next_exps=8, scale=None, bias=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return gptq.Fp8Weights(*a.values())


LINEAR = dict(a=FAKE, lda=304, ae=FAKE, ldae=4, ra=None, w=_w(), act=0, residual=FAKE, ldr=200, m=5, n=200, k=300, out=FAKE, odtype=1,
              ldo=200, ws=FAKE, ws_bytes=1 << 30, stream=None)
GATED = dict(a=FAKE, lda=304, ae=FAKE, ldae=4, ra=None, gate=_w(), up=_w(), act=2, m=5, n=200, k=300, codes=FAKE, ldc=208, exps=FAKE, lde=4,
             ws=FAKE, ws_bytes=1 << 30, stream=None)
EXPERTS = dict(a=FAKE, lda=304, ae=FAKE, ldae=4, w=_w(), act=0, n_experts=8, offsets=FAKE, order=FAKE, rows=10, n=200, k=300, out=FAKE,
               odtype=1, ldo=200, ws=FAKE, ws_bytes=1 << 30, stream=None)
EXPERTS_GATED = dict(a=FAKE, lda=304, ae=FAKE, ldae=4, ra=None, gate=_w(), up=_w(), act=2, n_experts=8, offsets=FAKE, order=FAKE, top_k=2,
                     n_tokens=5, n=200, k=300, codes=FAKE, ldc=208, exps=FAKE, lde=4, ws=FAKE, ws_bytes=1 << 30, stream=None)
ROUTE = dict(logits=FAKE, dtype=1, ld=64, n_tokens=50, n_experts=64, top_k=6, bias=None, scores=0, groups=8, top_groups=3, group_top=2,
             renormalize=1, scale=1.0, ids=FAKE, weights=FAKE, offsets=FAKE, order=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=None)
COMBINE = dict(y=FAKE, dtype=1, ldy=100, n_tokens=5, top_k=2, d=100, weights=FAKE, residual=FAKE, ldr=100, out=FAKE, ldo=100, stream=None)

A_FAULTS = [dict(a=None), dict(a=ODD), dict(lda=300), dict(lda=288), dict(ae=None), dict(ldae=3), dict(n=0), dict(k=0), dict(act=-1), dict(act=4)]
W_FAULTS = [dict(codes=None), dict(codes=AT + 8), dict(ld=300), dict(ld=288), dict(exps=None), dict(exps=AT + 2), dict(ld_exps=2),
            dict(ld_exps=5), dict(scale=AT + 2), dict(bias=AT + 1)]
NEXT_FAULTS = [dict(next_codes=304 * 199), dict(next_codes=304 * 200 + 8), dict(next_exps=4), dict(next_exps=10), dict(next_codes=0)]
WS_FAULTS = [dict(ws=None), dict(ws=ODD), dict(ws_bytes=16)]


@pytest.mark.parametrize("kw", A_FAULTS + [dict(m=-1), dict(odtype=2), dict(ldo=199), dict(out=None), dict(out=P(AT + 1)), dict(ldr=199),
                                           dict(residual=P(AT + 1)), dict(ra=P(AT + 2)), dict(w=None)] + [dict(w=_w(**f)) for f in W_FAULTS])
def test_linear_refuses(kw):
    assert _call(gptq.gptq_fp8_linear, LINEAR, **kw) == INV


@pytest.mark.parametrize("kw", A_FAULTS + [dict(m=-1), dict(ldc=200), dict(ldc=192), dict(codes=None), dict(codes=ODD), dict(exps=None), dict(lde=1),
                                           dict(gate=None), dict(up=None)] + [dict(gate=_w(**f)) for f in W_FAULTS]
                         + [dict(up=_w(**f)) for f in W_FAULTS])
def test_gated_refuses(kw):
    assert _call(gptq.gptq_fp8_gated, GATED, **kw) == INV


@pytest.mark.parametrize("kw", A_FAULTS + [dict(rows=-1), dict(n_experts=0), dict(offsets=None), dict(order=None), dict(offsets=P(AT + 2)),
                                           dict(order=P(AT + 1)), dict(out=None), dict(odtype=2), dict(ldo=100), dict(w=None)]
                         + [dict(w=_w(**f)) for f in W_FAULTS + NEXT_FAULTS])
def test_experts_refuses(kw):
    assert _call(gptq.gptq_fp8_experts, EXPERTS, **kw) == INV


@pytest.mark.parametrize("kw", A_FAULTS + [dict(n_tokens=-1), dict(top_k=0), dict(n_experts=0), dict(offsets=None), dict(order=None),
                                           dict(codes=None), dict(ldc=201), dict(gate=None), dict(up=None)]
                         + [dict(gate=_w(**f)) for f in W_FAULTS + NEXT_FAULTS] + [dict(up=_w(**f)) for f in NEXT_FAULTS])
def test_experts_gated_refuses(kw):
    assert _call(gptq.gptq_fp8_experts_gated, EXPERTS_GATED, **kw) == INV


def test_products_refuse_workspaces_and_sizes():
    for fn, base, rows in ((gptq.gptq_fp8_linear, LINEAR, "m"), (gptq.gptq_fp8_gated, GATED, "m"), (gptq.gptq_fp8_experts, EXPERTS, "rows"),
                           (gptq.gptq_fp8_experts_gated, EXPERTS_GATED, "n_tokens")):
        for kw in WS_FAULTS:
            assert _call(fn, base, **kw) == WS
        assert _call(fn, base, **{rows: (1 << 22) + 1}) == UNSUP
    assert _call(gptq.gptq_fp8_experts, EXPERTS, n_experts=1025) == UNSUP
    assert _call(gptq.gptq_fp8_experts_gated, EXPERTS_GATED, top_k=33) == UNSUP
    assert _call(gptq.gptq_fp8_experts_gated, EXPERTS_GATED, n_tokens=1 << 22, top_k=2) == UNSUP
    wide = _w(ld=1 << 21, ld_exps=1 << 14)
    assert _call(gptq.gptq_fp8_linear, LINEAR, w=wide, k=(1 << 20) + 1, lda=1 << 21, ldae=1 << 14) == UNSUP
    assert gptq.gptq_fp8_linear_workspace_bytes(1, 1, 1) >= 256 and gptq.gptq_fp8_linear_workspace_bytes(-1, 1, 1) == 0
    assert gptq.gptq_fp8_linear_workspace_bytes(1, 0, 1) == gptq.gptq_fp8_linear_workspace_bytes(1, 1, 0) == 0


@pytest.mark.parametrize("kw,st", [
    (dict(dtype=7), INV), (dict(n_tokens=-1), INV), (dict(n_experts=0), INV), (dict(ld=63), INV), (dict(top_k=0), INV), (dict(top_k=25), INV),
    (dict(scores=2), INV), (dict(groups=0), INV), (dict(groups=7), INV), (dict(top_groups=0), INV), (dict(top_groups=9), INV),
    (dict(group_top=0), INV), (dict(group_top=3), INV), (dict(groups=64, top_groups=64, group_top=2), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(logits=None), INV), (dict(logits=P(AT + 1)), INV), (dict(ids=None), INV), (dict(weights=None), INV),
    (dict(offsets=None), INV), (dict(order=None), INV), (dict(bias=P(AT + 2)), INV), (dict(order=P(AT + 2)), INV),
    (dict(ws=None), WS), (dict(ws=ODD), WS), (dict(ws_bytes=16), WS),
    (dict(groups=64, top_groups=64, group_top=1), UNSUP), (dict(n_experts=2048, ld=2048), UNSUP), (dict(n_tokens=1 << 22), UNSUP),
    (dict(groups=1, top_groups=1, top_k=33), UNSUP)])
def test_route_refuses(kw, st):
    assert _call(gptq.gptq_moe_route, ROUTE, **kw) == st


def test_route_workspace_sizes():
    size = gptq.gptq_moe_route_workspace_bytes
    assert size(0, 8, 2) >= 256 and size(8192, 256, 8) % 256 == 0 and size(8192, 256, 8) >= 2 * 64 * 256
    assert size(-1, 8, 2) == size(1, 0, 1) == size(1, 1025, 1) == size(1, 8, 0) == size(1, 64, 33) == size(1 << 22, 8, 2) == 0


@pytest.mark.parametrize("kw,st", [
    (dict(dtype=5), INV), (dict(n_tokens=-1), INV), (dict(top_k=0), INV), (dict(d=0), INV), (dict(ldy=99), INV), (dict(ldr=99), INV),
    (dict(ldo=99), INV), (dict(y=None), INV), (dict(weights=None), INV), (dict(out=None), INV), (dict(y=P(AT + 1)), INV),
    (dict(weights=P(AT + 2)), INV), (dict(residual=P(AT + 1)), INV), (dict(out=P(AT + 1)), INV),
    (dict(top_k=33), UNSUP), (dict(n_tokens=(1 << 21) + 1), UNSUP), (dict(d=1 << 21, ldy=1 << 21, ldr=1 << 21, ldo=1 << 21), UNSUP)])
def test_combine_refuses(kw, st):
    assert _call(gptq.gptq_moe_combine, COMBINE, **kw) == st


def test_helpers_refuse():
    torch = pytest.importorskip("torch")
    f8, u8, i32 = torch.float8_e4m3fn, torch.uint8, torch.int32

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype)

    a, ae, w, we = empty(4, 256, dtype=f8), empty(4, 2, dtype=u8), empty(130, 256, dtype=f8), empty(2, 2, dtype=u8)
    ew, ewe = empty(3, 130, 256, dtype=f8), empty(3, 2, 2, dtype=u8)
    offsets, order = empty(4, dtype=i32), empty(8, dtype=i32)
    for call in (lambda: gptq.fp8_linear(a, ae, w, we), lambda: gptq.fp8_gated(a, ae, (w, we), (w, we)),
                 lambda: gptq.fp8_experts(a, ae, ew, ewe, offsets, order[:4]),
                 lambda: gptq.fp8_experts_gated(a, ae, (ew, ewe), (ew, ewe), offsets, order, 2),
                 lambda: gptq.moe_route(empty(4, 8), 2), lambda: gptq.moe_combine(empty(8, 16), empty(4, 2, dtype=torch.float32))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for bad in (lambda: gptq.moe_route(empty(4, 8), 2, scores="other"), lambda: gptq.moe_route(empty(8), 2),
                lambda: gptq.moe_route(empty(4, 8), 2, bias=torch.zeros(7)), lambda: gptq.moe_combine(empty(7, 16), empty(4, 2, dtype=torch.float32)),
                lambda: gptq.moe_combine(empty(8, 16), empty(4, 2)), lambda: gptq.fp8_linear(a, ae[:, :1], w, we),
                lambda: gptq.moe_combine(empty(8, 16), empty(4, 2, dtype=torch.float32), residual=empty(4, 15))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        gptq.moe_combine(empty(8, 16), empty(4, 2, dtype=torch.float32), residual=empty(4, 16, dtype=torch.float16))
    with pytest.raises(TypeError):
        gptq.fp8_linear(empty(4, 256), ae, w, we)


@pytest.mark.gpu
def test_helpers_refuse_what_does_not_match():
    import torch
    dev = "cuda:0"
    f8, u8, i32 = torch.float8_e4m3fn, torch.uint8, torch.int32

    def empty(*shape, dtype):
        return torch.empty(*shape, dtype=dtype, device=dev)

    a, ae, w, we = empty(4, 256, dtype=f8), empty(4, 4, dtype=u8)[:, :2], empty(130, 256, dtype=f8), empty(2, 4, dtype=u8)[:, :2]
    ew, ewe = empty(3, 130, 256, dtype=f8), empty(3, 2, 4, dtype=u8)[:, :, :2]
    offsets, order = empty(4, dtype=i32), empty(8, dtype=i32)
    plan = (offsets, order)
    calls = [lambda: gptq.fp8_linear(a, ae, w, we, act="tanh"), lambda: gptq.fp8_linear(a, ae, w[:, :128], we),
             lambda: gptq.fp8_linear(a, ae, w, we[:1]), lambda: gptq.fp8_linear(a, ae, ew, ewe), lambda: gptq.fp8_linear(a, ae, w.cpu(), we),
             lambda: gptq.fp8_linear(a, ae, w, we, bias=torch.zeros(129, device=dev)), lambda: gptq.fp8_linear(a, ae, w, we, bias=torch.zeros(130)),
             lambda: gptq.fp8_linear(a, ae, w, we, residual=torch.zeros(4, 129, dtype=torch.bfloat16, device=dev)),
             lambda: gptq.fp8_gated(a, ae, (w,), (w, we)), lambda: gptq.fp8_gated(a, ae, (w, we), (w[:129], we)),
             lambda: gptq.fp8_experts_gated(a, ae, (ew, ewe), (ew[:2], ewe[:2]), *plan, 2),
             lambda: gptq.fp8_experts_gated(a, ae, (ew, ewe), (ew, ewe), offsets, order[:7], 2),
             lambda: gptq.fp8_experts_gated(a, ae, (ew, ewe), (ew, ewe), offsets, order, 0),
             lambda: gptq.fp8_experts(a, ae, ew, ewe, offsets.cpu(), order[:4]), lambda: gptq.fp8_experts(a, ae, w, we, offsets, order[:4]),
             lambda: gptq.moe_route(torch.zeros(4, 8, device=dev), 9), lambda: gptq.moe_route(torch.zeros(4, 8, device=dev), 0)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(str(i))
    for call in (lambda: gptq.fp8_experts(a, ae, ew, ewe, offsets.long(), order[:4]), lambda: gptq.fp8_linear(a, ae, w.view(u8), we),
                 lambda: gptq.fp8_linear(a, ae, w, we, residual=torch.zeros(4, 130, device=dev)),
                 lambda: gptq.moe_route(torch.zeros(4, 8, dtype=i32, device=dev), 2)):
        with pytest.raises(TypeError):
            call()
    for kw in (dict(top_k=5, groups=4, top_groups=2), dict(top_k=2, groups=3), dict(top_k=2, groups=4, top_groups=5), dict(top_k=1, groups=8),
               dict(top_k=2, scale=float("inf"))):
        with pytest.raises(gptq.GptqError, match="INVALID_ARG"):
            gptq.moe_route(torch.zeros(4, 8, device=dev), **kw)


@pytest.mark.gpu
def test_helpers_refuse_workspaces_that_do_not_hold_their_elements():
    import torch
    dev = "cuda:0"
    f8, u8 = torch.float8_e4m3fn, torch.uint8
    a, ae = torch.zeros(4, 256, dtype=u8, device=dev).view(f8), torch.zeros(4, 4, dtype=u8, device=dev)[:, :2]
    w, we = torch.zeros(130, 256, dtype=u8, device=dev).view(f8), torch.zeros(2, 4, dtype=u8, device=dev)[:, :2]
    one = torch.zeros(1, dtype=u8, device=dev).expand(1 << 20)          # a million elements in one byte
    offsets, order = torch.zeros(2, dtype=torch.int32, device=dev), torch.zeros(4, dtype=torch.int32, device=dev)
    for call in (lambda: gptq.fp8_linear(a, ae, w, we, ws=one), lambda: gptq.fp8_gated(a, ae, (w, we), (w, we), ws=one),
                 lambda: gptq.fp8_experts_gated(a, ae, (w[None], we[None]), (w[None], we[None]), offsets, order, 1, ws=one),
                 lambda: gptq.fp8_experts(a, ae, w[None], we[None], offsets, order, ws=one),
                 lambda: gptq.moe_route(torch.zeros(400, 8, device=dev), 2, ws=one)):
        with pytest.raises(ValueError, match="contiguous"):
            call()
    assert gptq.moe_route(torch.zeros(400, 8, device=dev), 2, ws=torch.zeros(1 << 16, dtype=u8, device=dev))[0].shape == (400, 2)
    gptq.fp8_linear(a, ae, w, we, ws=torch.zeros(256, dtype=u8, device=dev))
    torch.cuda.synchronize()
