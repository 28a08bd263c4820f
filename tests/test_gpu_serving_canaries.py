"""Guard bytes around every buffer that the 8-bit serving entry points write, and between the
rows of pitched outputs: after calls through the C ABI on ragged shapes each of them must still
hold its pattern.  What lies between an input row's end and its pitch, or in cache slots that no
length covers, must not show in a result."""

import ctypes

import numpy as np
import pytest
import torch

from post_weight_quantization_03_gb300 import build_lib, gptq
from tests.test_gpu_canaries import PAT, Guarded

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    gptq.load()
    torch.cuda.init()


def _p(t):
    return ctypes.c_void_p(t.data_ptr())


def _randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


def _ok(st):
    assert st == 0, gptq.gptq_status_str(st)


def _matrix(rows, d, row_block=1, extra=0):
    """Guarded codes and exponents with their pitches (`extra` blocks of 16 and 4 more)."""
    ldc = -(-d // 16) * 16 + 16 * extra
    lde = -(-(-(-d // 128)) // 4) * 4 + 4 * extra
    erows = -(-rows // row_block)
    return Guarded(rows * ldc), ldc, Guarded(erows * lde), lde, erows


def _whole(codes, ldc, exps, lde, rows, erows, d):
    kb = -(-d // 128)
    assert codes.intact() and exps.intact()
    assert bool((codes.view(torch.uint8, (rows, ldc))[:, d:] == PAT).all())
    assert bool((exps.view(torch.uint8, (erows, lde))[:, kb:] == PAT).all())


@pytest.mark.parametrize("rows,d,extra", [(1, 1, 0), (3, 129, 1), (67, 1000, 0), (2, 4099, 1), (5, 8200, 0), (3, 17001, 1),
                                          (1300, 515, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_and_quantizers(rows, d, extra, dtype):
    x, r, w = _randn(1, rows, d, dtype=dtype), _randn(2, rows, d, dtype=dtype), _randn(3, d, dtype=dtype)
    es = x.element_size()
    codes, ldc, exps, lde, _ = _matrix(rows, d, 1, extra)
    h, rstd = Guarded(rows * (d + 3) * es), Guarded(rows * 4)
    _ok(gptq.gptq_rmsnorm_fp8(_p(x), DT[dtype], rows, d, d, _p(r), d, _p(w), DT[dtype], 1e-6, h.ptr, d + 3, codes.ptr, ldc,
                              exps.ptr, lde, rstd.ptr, gptq._stream(None)))
    _whole(codes, ldc, exps, lde, rows, rows, d)
    assert h.intact() and rstd.intact()
    assert bool((h.view(torch.uint8, (rows, (d + 3) * es))[:, d * es:] == PAT).all())
    for row_block in (1, 128):
        codes, ldc, exps, lde, erows = _matrix(rows, d, row_block, extra)
        _ok(gptq.gptq_fp8_quantize(_p(x), DT[dtype], rows, d, d, row_block, codes.ptr, ldc, exps.ptr, lde, gptq._stream(None)))
        _whole(codes, ldc, exps, lde, rows, erows, d)


@pytest.mark.parametrize("rows,d,bits", [(1, 5, 4), (130, 300, 3), (129, 1025, 2)])
def test_from_codes(rows, d, bits):
    g = torch.Generator().manual_seed(1)
    qp = torch.randint(0, 2 ** 31, (rows, gptq.packed_words(d, bits)), generator=g).to(torch.int32).to(DEV)
    zero = torch.randint(0, 2 ** bits, (rows,), generator=g).to(torch.int32).to(DEV)
    codes, ldc, exps, lde, erows = _matrix(rows, d, 128, 1)
    _ok(gptq.gptq_fp8_from_codes(_p(qp), bits, _p(zero), rows, d, codes.ptr, ldc, exps.ptr, lde, gptq._stream(None)))
    _whole(codes, ldc, exps, lde, rows, erows, d)


# tall and wide, K split and not, one and two tiles of tokens, more tiles than SMs
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 129, 4000), (15, 300, 131), (100, 130, 9000), (241, 1000, 500), (700, 4100, 300),
                                   (1500, 5000, 260)])
@pytest.mark.parametrize("extra", [0, 1])
def test_product(m, n, k, extra):
    kb = -(-k // 128)
    a, ldc, ae, lde, _ = _matrix(m, k, 1, extra)
    w, _, we, _, erows = _matrix(n, k, 128, extra)
    x, y = _randn(1, m, k), _randn(2, n, k)
    s = gptq._stream(None)
    _ok(gptq.gptq_fp8_quantize(_p(x), 2, m, k, k, 1, a.ptr, ldc, ae.ptr, lde, s))
    _ok(gptq.gptq_fp8_quantize(_p(y), 2, n, k, k, 128, w.ptr, ldc, we.ptr, lde, s))
    need = gptq.gptq_fp8_matmul_workspace_bytes(m, n, k)
    results = []
    for fill in (0x7F, 0):   # between the rows: NaN codes and the largest exponents, then zeros
        a.view(torch.uint8, (m, ldc))[:, k:] = fill
        w.view(torch.uint8, (n, ldc))[:, k:] = fill
        ae.view(torch.uint8, (m, lde))[:, kb:] = 2 * fill + 1
        we.view(torch.uint8, (erows, lde))[:, kb:] = 2 * fill + 1
        out, ws = Guarded(m * (n + 5) * 2), Guarded(need)
        _ok(gptq.gptq_fp8_matmul(a.ptr, ldc, ae.ptr, lde, None, w.ptr, ldc, we.ptr, lde, None, m, n, k, out.ptr, 1, n + 5,
                                 ws.ptr, need, s))
        assert out.intact() and ws.intact()
        got = out.view(torch.bfloat16, (m, n + 5))
        assert bool((out.view(torch.uint8, (m, 2 * (n + 5)))[:, 2 * n:] == PAT).all())
        results.append(got[:, :n].clone())
    assert bool(torch.isfinite(results[0]).all()) and torch.equal(results[0], results[1])
    assert a.intact() and ae.intact() and w.intact() and we.intact()


# decoding with whole items and with shares, prompts of one and of several pieces
@pytest.mark.parametrize("seqs,new,kv,group,d,longest", [(1, 1, 1, 1, 64, 70), (3, 1, 2, 8, 128, 900), (9, 3, 2, 4, 64, 4000),
                                                         (2, 33, 1, 8, 128, 300), (3, 130, 2, 4, 64, 2000)])
def test_append_and_attention(seqs, new, kv, group, d, longest):
    rng = np.random.default_rng(new)
    mb = -(-longest // 64)
    blocks = seqs * mb + 2
    lengths = rng.integers(new, longest + 1, seqs)
    lengths[0] = longest
    start = torch.from_numpy((lengths - new).astype(np.int32)).to(DEV)
    length = torch.from_numpy(lengths.astype(np.int32)).to(DEV)
    table = torch.from_numpy(rng.permutation(blocks)[:seqs * mb].astype(np.int32).reshape(seqs, mb)).to(DEV)
    s, heads = gptq._stream(None), kv * group
    strides = (ctypes.c_int64 * 3)(new * kv * d, kv * d, d)
    k, v = _randn(5, seqs, new, kv, d, dtype=torch.bfloat16), _randn(6, seqs, new, kv, d, dtype=torch.bfloat16)
    q = _randn(7, seqs, new, heads, d, dtype=torch.bfloat16)
    ostr = (new * (heads * d + 8) + 16, heads * d + 8, d)
    o_strides = (ctypes.c_int64 * 3)(*ostr)
    q_strides = (ctypes.c_int64 * 3)(new * heads * d, heads * d, d)
    elems = (seqs - 1) * ostr[0] + (new - 1) * ostr[1] + heads * d
    used = torch.zeros(elems, dtype=torch.bool, device=DEV)
    used.as_strided((seqs, new, heads, d), ostr + (1,))[:] = True
    need = gptq.gptq_kv8_attention_workspace_bytes(seqs, new, heads, kv, d, mb)
    g = torch.Generator().manual_seed(8)
    old_k = torch.randint(0, 120, (blocks, kv, 64, d), generator=g).to(torch.uint8).to(DEV)
    old_v = torch.randint(0, 120, (blocks, kv, d, 64), generator=g).to(torch.uint8).to(DEV)
    results = []
    for fill in (0x7F, 0):   # in the slots past each length
        ck, cv = Guarded(blocks * kv * 64 * d), Guarded(blocks * kv * 64 * d)
        ke, ve = Guarded(blocks * kv), Guarded(blocks * kv)
        K, V = ck.view(torch.uint8, (blocks, kv, 64, d)), cv.view(torch.uint8, (blocks, kv, d, 64))
        K[:], V[:] = old_k, old_v
        ke.view(torch.uint8, (blocks, kv))[:] = 120
        ve.view(torch.uint8, (blocks, kv))[:] = 121
        for i in range(seqs):
            last, at = divmod(int(lengths[i]), 64)
            for b in range(last, mb):
                K[table[i, b], :, at if b == last else 0:] = fill
                V[table[i, b], :, :, at if b == last else 0:] = fill
        _ok(gptq.gptq_kv8_append(_p(k), strides, _p(v), strides, 1, seqs, new, kv, d, ck.ptr, cv.ptr, ke.ptr, ve.ptr, blocks,
                                 _p(table), mb, mb, _p(start), s))
        out, ws = Guarded(elems * 2), Guarded(need)
        _ok(gptq.gptq_kv8_attention(_p(q), q_strides, 1, seqs, new, heads, kv, d, ck.ptr, cv.ptr, ke.ptr, ve.ptr, blocks,
                                    _p(table), mb, mb, _p(length), 1, d ** -0.5, out.ptr, o_strides, ws.ptr, need, s))
        for b in (ck, cv, ke, ve, out, ws):
            assert b.intact()
        got = out.view(torch.int16, (elems,))
        assert bool((got[~used] == np.array([PAT, PAT], np.uint8).view(np.int16)[0]).all())
        results.append(got[used].view(torch.bfloat16).clone())
    assert bool(torch.isfinite(results[0]).all()) and torch.equal(results[0], results[1])
