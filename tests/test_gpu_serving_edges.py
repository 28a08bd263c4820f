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
