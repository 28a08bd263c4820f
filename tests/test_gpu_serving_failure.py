"""Bounded waits of the 8-bit serving kernels that run out, without a fault.

The library's test hooks run the product and the attention with one copy of every CTA left out, so
that the waits for it cannot complete; with a short budget each gives up, the kernel records
GPTQ_ERR_TIMEOUT and ends, and the next regular call on the same GPU gives what it gave before.
"""

import ctypes
import time

import numpy as np
import pytest
import torch

from post_weight_quantization_03_gb300 import gptq
from tests.test_gpu_serving import DEV, DT, _cache, _dev_cache, _i32, _lib, _randn, _table  # noqa: F401

pytestmark = pytest.mark.gpu

TIMEOUT, BUDGET = 4, 50_000_000


def _p(t):
    return ctypes.c_void_p(t.data_ptr())


def _strides(t):
    return (ctypes.c_int64 * 3)(*t.stride()[:3])


def _product(m, n, k):
    a, ae = gptq.fp8_quantize(_randn(1, m, k).to(DEV))
    w, we = gptq.fp8_quantize(_randn(2, n, k).to(DEV), 128)
    out = torch.zeros(m, n, dtype=torch.bfloat16, device=DEV)
    ws = gptq.workspace(gptq.gptq_fp8_matmul_workspace_bytes(m, n, k), DEV)

    def lost(copy):
        return gptq.gptq_debug_fp8_matmul_lost_copy(
            _p(a), a.stride(0), _p(ae), ae.stride(0), _p(w), w.stride(0), _p(we), we.stride(0), m, n, k, _p(out), 1, n, copy,
            BUDGET, _p(ws), ws.numel(), gptq._stream(None))

    return lambda: gptq.fp8_matmul(a, ae, w, we, ws=ws), lost, out, ws


def _attention(seqs, new, kv, group, d, length, dtype):
    mb = -(-length // 64)
    cache = _dev_cache(_cache(1, seqs * mb, kv, d))
    table = _i32(_table(np.random.default_rng(1), seqs, mb, seqs * mb))
    lengths = _i32([length] * seqs)
    heads = kv * group
    q = _randn(2, seqs, new, heads, d, dtype=dtype).to(DEV)
    out = torch.zeros_like(q)
    ws = gptq.workspace(gptq.gptq_kv8_attention_workspace_bytes(seqs, new, heads, kv, d, mb), DEV)

    def lost(copy):
        return gptq.gptq_debug_kv8_attention_lost_copy(
            _p(q), _strides(q), gptq._dtype_code(q), seqs, new, heads, kv, d, *(_p(t) for t in cache), seqs * mb, _p(table), mb,
            mb, _p(lengths), 1, d ** -0.5, _p(out), _strides(out), copy, BUDGET, _p(ws), ws.numel(), gptq._stream(None))

    return lambda: gptq.kv8_attention(q, cache, table, lengths, ws=ws), lost, out, ws


def _runs_out(call, lost, out, ws):
    want = call()
    seen = []
    for copy in (0, 1, 2, 6, 10 ** 6):                      # the last: no CTA has that many copies
        t0 = time.time()
        seen.append(lost(copy))
        assert time.time() - t0 < 2.0                       # a few budgets
        assert seen[-1] in (0, TIMEOUT), gptq.gptq_status_str(seen[-1])
        if seen[-1] == 0:
            assert torch.equal(out, want)
        again = call()
        assert gptq.gptq_workspace_status(_p(ws), gptq._stream(None)) == 0
        assert torch.equal(again, want)
    assert seen[0] == TIMEOUT and seen[-1] == 0 and seen == sorted(seen, reverse=True)


# one tile, K split over a cluster, a tile a CTA, several tiles a CTA
@pytest.mark.parametrize("m,n,k", [(1, 128, 512), (8, 512, 8192), (300, 2000, 2048), (1500, 8000, 1024)])
def test_product_with_a_lost_copy(m, n, k):
    _runs_out(*_product(m, n, k))


# decoding by shares, whole items to CTAs and to groups, one to four row tiles; prompts cut and uncut
@pytest.mark.parametrize("seqs,new,kv,group,d,length", [
    (4, 1, 2, 4, 128, 6000), (8, 2, 2, 8, 64, 3000), (8, 4, 1, 8, 64, 3000), (40, 1, 2, 4, 64, 3000), (3, 1, 2, 4, 64, 700),
    (200, 1, 2, 4, 64, 60), (2, 100, 2, 4, 128, 3000), (1, 2000, 4, 4, 64, 2000), (4, 64, 2, 4, 128, 200)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attention_with_a_lost_copy(seqs, new, kv, group, d, length, dtype):
    _runs_out(*_attention(seqs, new, kv, group, d, length, dtype))


def test_hooks_reject_bad_requests():
    call, lost, _, _ = _product(4, 128, 256)
    assert lost(-1) == 1
    call, lost, _, _ = _attention(1, 1, 1, 4, 64, 100, "bf16")
    assert lost(-1) == 1


def test_timeouts_of_calls_whose_status_is_gone():
    # the helpers' calls share a status block or drop their workspace: a wait that gave up is told all the same, once
    gptq.gptq_serving_status(gptq._stream(None))            # (of the tests before)
    regular, lost, _, _ = _product(8, 512, 8192)
    attend, lost_attend, _, _ = _attention(2, 100, 2, 4, 128, 3000, "bf16")
    other = torch.cuda.Stream()
    for hook in (lost, lost_attend, _attention(4, 1, 2, 4, 128, 6000, "bf16")[1]):
        assert hook(0) == TIMEOUT
        regular(), attend()                                 # later calls reset what they use
        with pytest.raises(gptq.GptqError) as e:
            gptq.serving_status(other)
        assert e.value.status == TIMEOUT
        regular(), attend()
        gptq.serving_status()
