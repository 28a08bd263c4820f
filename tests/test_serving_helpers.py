"""The serving helpers refuse what the kernels would read as something else: tensors on the host, and
integers of another width (no GPU is touched)."""

import pytest

torch = pytest.importorskip("torch")

from post_weight_quantization_03_gb300 import build_lib, gptq  # noqa: E402

F8, U8, I32 = torch.float8_e4m3fn, torch.uint8, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    gptq.load()


def _empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype)


def test_host_tensors_are_refused():
    cache = gptq.kv8_cache(2, 2, 64, device="cpu")
    table, n = torch.zeros(1, 2, dtype=I32), torch.zeros(1, dtype=I32)
    a, ae, w, we = _empty(4, 256, dtype=F8), _empty(4, 2, dtype=U8), _empty(130, 256, dtype=F8), _empty(2, 2, dtype=U8)
    for call in (lambda: gptq.rmsnorm_fp8(_empty(4, 64), _empty(64)), lambda: gptq.fp8_quantize(_empty(4, 64)),
                 lambda: gptq.fp8_from_codes(torch.zeros(4, 8, dtype=I32), torch.zeros(4, dtype=I32), 64),
                 lambda: gptq.fp8_matmul(a, ae, w, we),
                 lambda: gptq.kv8_append(cache, _empty(1, 1, 2, 64), _empty(1, 1, 2, 64), table, n),
                 lambda: gptq.kv8_attention(_empty(1, 1, 4, 64), cache, table, n)):
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.gpu
def test_one_host_tensor_among_others_is_refused():
    dev = "cuda:0"
    x, w = _empty(4, 64), _empty(64)
    with pytest.raises(ValueError, match="GPU"):
        gptq.rmsnorm_fp8(x.to(dev), w)
    with pytest.raises(ValueError, match="GPU"):
        gptq.rmsnorm_fp8(x.to(dev), w.to(dev), residual=x)
    a, ae = gptq.fp8_quantize(torch.ones(4, 256, device=dev))
    b, be = gptq.fp8_quantize(torch.ones(130, 256, device=dev), 128)
    for kw in (dict(a_scale=torch.ones(4)), dict(w_scale=torch.ones(130)), dict(out=_empty(4, 130)),
               dict(ws=torch.empty(256, dtype=U8))):
        with pytest.raises(ValueError, match="GPU"):
            gptq.fp8_matmul(a, ae, b, be, **kw)
    cache = gptq.kv8_cache(2, 2, 64, dev)
    table, n = torch.zeros(1, 2, dtype=I32, device=dev), torch.zeros(1, dtype=I32, device=dev)
    q, k = _empty(1, 1, 4, 64).to(dev), _empty(1, 1, 2, 64).to(dev)
    with pytest.raises(ValueError, match="GPU"):
        gptq.kv8_attention(q, cache, table.cpu(), n)
    with pytest.raises(ValueError, match="GPU"):
        gptq.kv8_append(cache, k, k, table, n.cpu())
    with pytest.raises(ValueError, match="GPU"):
        gptq.kv8_attention(q, (cache[0], cache[1], cache[2].cpu(), cache[3]), table, n)


@pytest.mark.parametrize("qdtype,zdtype", [(torch.uint8, I32), (torch.int64, I32), (I32, torch.int64), (I32, torch.uint8)])
def test_codes_of_another_width_are_refused(qdtype, zdtype):
    with pytest.raises(TypeError):
        gptq.fp8_from_codes(torch.zeros(4, 8, dtype=qdtype), torch.zeros(4, dtype=zdtype), 64)


def test_row_blocks():
    with pytest.raises(ValueError):
        gptq.fp8_quantize(_empty(4, 64), 0)
    with pytest.raises(ValueError):
        gptq.fp8_quantize(_empty(4, 64), 64)
