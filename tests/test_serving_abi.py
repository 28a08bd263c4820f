"""Refusals of the 8-bit serving calls: arguments that fail validation return before the GPU is
touched (so this runs without one)."""

import ctypes

import pytest

from post_weight_quantization_03_gb300 import build_lib, gptq

P = ctypes.c_void_p
FAKE, ODD = P(256 * 1024), P(256 * 1024 + 8)   # never dereferenced
INV, UNSUP, WS = 1, 6, 7


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    gptq.load()


def _call(fn, base, **kw):
    a = dict(base)
    assert set(kw) <= set(a)
    a.update(kw)
    return fn(*a.values())


NORM = dict(X=FAKE, xdtype=1, rows=4, d=300, ldx=300, R=FAKE, ldr=300, weight=FAKE, wdtype=1,
            eps=1e-6, H=FAKE, ldh=300, codes=FAKE, ldc=304, exps=FAKE, lde=4, rstd=FAKE, stream=None)


@pytest.mark.parametrize("kw", [
    dict(xdtype=9), dict(wdtype=0), dict(rows=-1), dict(d=0), dict(ldx=299), dict(ldr=299), dict(ldh=299),
    dict(eps=-1.0), dict(eps=float("nan")), dict(X=None), dict(weight=None), dict(codes=None), dict(exps=None),
    dict(rstd=None), dict(ldc=300), dict(ldc=288), dict(codes=ODD), dict(lde=3), dict(lde=0),
    dict(exps=P(256 * 1024 + 2)), dict(X=P(256 * 1024 + 1))])
def test_norm_refuses(kw):
    assert _call(gptq.gptq_rmsnorm_fp8, NORM, **kw) == INV


def test_norm_limits_and_empty():
    assert _call(gptq.gptq_rmsnorm_fp8, NORM, d=(1 << 20) + 16, ldx=1 << 21, ldr=1 << 21, ldh=1 << 21, ldc=1 << 21,
                 lde=1 << 14) == UNSUP
    assert _call(gptq.gptq_rmsnorm_fp8, NORM, rows=0, X=None, codes=None, exps=None, rstd=None) == 0


QUANT = dict(X=FAKE, xdtype=1, rows=4, d=300, ldx=300, row_block=1, codes=FAKE, ldc=304, exps=FAKE, lde=4, stream=None)
CODES = dict(qpacked=FAKE, bits=4, zero=FAKE, d_out=4, d_in=300, codes=FAKE, ldc=304, exps=FAKE, lde=4, stream=None)


@pytest.mark.parametrize("kw", [dict(xdtype=3), dict(row_block=2), dict(row_block=0), dict(rows=-1), dict(d=0),
                                dict(ldx=10), dict(X=None), dict(ldc=303), dict(lde=2), dict(codes=ODD)])
def test_quantize_refuses(kw):
    assert _call(gptq.gptq_fp8_quantize, QUANT, **kw) == INV


@pytest.mark.parametrize("kw,st", [(dict(bits=5), INV), (dict(bits=8), UNSUP), (dict(d_out=0), INV), (dict(d_in=0), INV),
                                   (dict(qpacked=None), INV), (dict(zero=None), INV), (dict(ldc=290), INV),
                                   (dict(lde=6), INV)])
def test_from_codes_refuses(kw, st):
    assert _call(gptq.gptq_fp8_from_codes, CODES, **kw) == st


MM = dict(a=FAKE, lda=304, ae=FAKE, ldae=4, ra=None, w=FAKE, ldw=304, we=FAKE, ldwe=4, rw=None, m=5, n=200, k=300,
          out=FAKE, odtype=1, ldo=200, ws=FAKE, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,st", [
    (dict(m=-1), INV), (dict(n=0), INV), (dict(k=0), INV), (dict(odtype=2), INV), (dict(odtype=7), INV),
    (dict(ldo=199), INV), (dict(lda=300), INV), (dict(ldw=288), INV), (dict(ldae=3), INV), (dict(ldwe=0), INV),
    (dict(a=None), INV), (dict(w=None), INV), (dict(ae=None), INV), (dict(we=None), INV), (dict(out=None), INV),
    (dict(a=ODD), INV), (dict(w=ODD), INV), (dict(ra=P(256 * 1024 + 2)), INV), (dict(rw=P(256 * 1024 + 1)), INV),
    (dict(ws=None), WS), (dict(ws=ODD), WS), (dict(ws_bytes=16), WS),
    (dict(k=(1 << 20) + 1, lda=1 << 21, ldw=1 << 21, ldae=1 << 14, ldwe=1 << 14), UNSUP),
    (dict(n=(1 << 22) + 1, ldo=1 << 23), UNSUP)])
def test_matmul_refuses(kw, st):
    assert _call(gptq.gptq_fp8_matmul, MM, **kw) == st


def test_workspace_sizes():
    assert gptq.gptq_fp8_matmul_workspace_bytes(1, 4096, 4096) >= 256
    assert gptq.gptq_fp8_matmul_workspace_bytes(1, 0, 4096) == 0
    assert gptq.gptq_kv8_attention_workspace_bytes(2, 1, 8, 2, 128, 10) >= 256
    for bad in ((-1, 1, 8, 2, 128, 10), (2, -1, 8, 2, 128, 10), (2, 1, 8, 3, 128, 10), (2, 1, 8, 2, 96, 10),
                (2, 1, 8, 2, 128, -1), (2, 1, 0, 2, 128, 10)):
        assert gptq.gptq_kv8_attention_workspace_bytes(*bad) == 0


def _st(*v):
    return (ctypes.c_int64 * 3)(*v)


APP = dict(new_k=FAKE, ks=_st(1024, 256, 128), new_v=FAKE, vs=_st(1024, 256, 128), dtype=1, n_seq=2, n_new=4, n_kv=2,
           dim=128, k=FAKE, v=FAKE, ke=FAKE, ve=FAKE, n_blocks=8, table=FAKE, ld_table=4, max_blocks=4, start=FAKE,
           stream=None)
ATT = dict(q=FAKE, qs=_st(4096, 1024, 128), dtype=1, n_seq=2, n_new=4, n_heads=8, n_kv=2, dim=128, k=FAKE, v=FAKE,
           ke=FAKE, ve=FAKE, n_blocks=8, table=FAKE, ld_table=4, max_blocks=4, lengths=FAKE, causal=1, scale=0.1,
           out=FAKE, os=_st(4096, 1024, 128), ws=FAKE, ws_bytes=1 << 40, stream=None)
SHARED = [(dict(n_seq=-1), INV), (dict(n_new=-1), INV), (dict(n_kv=0), INV), (dict(dim=0), INV), (dict(dim=96), UNSUP),
          (dict(k=None), INV), (dict(v=None), INV), (dict(ke=None), INV), (dict(ve=None), INV), (dict(k=ODD), INV),
          (dict(v=ODD), INV), (dict(table=None), INV), (dict(ld_table=3), INV), (dict(n_blocks=-1), INV),
          (dict(max_blocks=-1), INV), (dict(n_seq=70000), UNSUP), (dict(n_blocks=1 << 31), UNSUP), (dict(dtype=5), INV)]


@pytest.mark.parametrize("kw,st", SHARED + [
    (dict(ks=_st(0, -1, 0)), INV), (dict(vs=None), INV), (dict(new_k=None), INV), (dict(new_v=None), INV),
    (dict(start=None), INV), (dict(new_k=P(256 * 1024 + 1)), INV)])
def test_append_refuses(kw, st):
    assert _call(gptq.gptq_kv8_append, APP, **kw) == st


@pytest.mark.parametrize("kw,st", SHARED + [
    (dict(dtype=2), INV), (dict(n_heads=7), INV), (dict(n_heads=0), INV), (dict(qs=_st(1, 1, -1)), INV),
    (dict(os=None), INV), (dict(scale=float("inf")), INV), (dict(scale=float("nan")), INV), (dict(q=None), INV),
    (dict(out=None), INV), (dict(lengths=None), INV), (dict(ws=None), WS), (dict(ws=ODD), WS), (dict(ws_bytes=0), WS)])
def test_attention_refuses(kw, st):
    assert _call(gptq.gptq_kv8_attention, ATT, **kw) == st


def test_append_of_nothing_is_ok():
    assert _call(gptq.gptq_kv8_append, APP, n_seq=0) == 0
    assert _call(gptq.gptq_kv8_append, APP, n_new=0) == 0
    assert _call(gptq.gptq_kv8_append, APP, n_blocks=0, k=None, v=None, ke=None, ve=None) == 0


def test_helpers_refuse_mismatched_tensors():
    torch = pytest.importorskip("torch")
    f8 = torch.float8_e4m3fn
    a, ae = torch.empty(4, 256, dtype=f8), torch.empty(4, 2, dtype=torch.uint8)
    w, we = torch.empty(130, 256, dtype=f8), torch.empty(2, 2, dtype=torch.uint8)
    with pytest.raises(ValueError):
        gptq.fp8_matmul(a, ae, w[:, :128], we)
    with pytest.raises(ValueError):
        gptq.fp8_matmul(a, ae[:3], w, we)
    with pytest.raises(ValueError):
        gptq.fp8_matmul(a, ae, w, we[:1])
    with pytest.raises(TypeError):
        gptq.fp8_matmul(a.view(torch.uint8), ae, w, we)
    with pytest.raises(ValueError):
        gptq.fp8_matmul(a, ae, w, we, a_scale=torch.empty(3))
    with pytest.raises(ValueError):
        gptq.rmsnorm_fp8(torch.empty(4, 8), torch.empty(7))
    with pytest.raises(TypeError):
        gptq.rmsnorm_fp8(torch.empty(4, 8), torch.empty(8), residual=torch.empty(4, 8, dtype=torch.float16))
    cache = gptq.kv8_cache(2, 2, 64, device="cpu")
    table, n = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        gptq.kv8_attention(torch.empty(1, 1, 4, 128), cache, table, n)
    with pytest.raises(TypeError):
        gptq.kv8_attention(torch.empty(1, 1, 4, 64), cache, table.long(), n)
    with pytest.raises(ValueError):
        gptq.kv8_append(cache, torch.empty(1, 1, 3, 64), torch.empty(1, 1, 3, 64), table, n)
    with pytest.raises(ValueError):
        gptq.kv8_attention(torch.empty(2, 1, 4, 64), cache, table, n)
