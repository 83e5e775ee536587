"""The binding's checks of kv_attention and kv_evict that need no GPU."""
from __future__ import annotations

import pytest
import torch

fp8 = pytest.importorskip("fp8_precision_quantization_amd")


def _args():
    cache = torch.zeros((64, 2, 64), dtype=torch.uint8)
    scales = torch.ones((64, 2))
    return dict(k_cache=cache, v_cache=cache.clone(), k_scale_inv=scales, v_scale_inv=scales, page_size=16,
                page_table=torch.zeros((1, 4), dtype=torch.int32), lens=torch.ones(1, dtype=torch.int32))


WIDE = [1 << 31, (1 << 32) + 5, -(1 << 31) - 1]


@pytest.mark.parametrize("value", WIDE)
@pytest.mark.parametrize("name", ["window", "sinks", "page_size"])
def test_attention_numbers_past_32_bits(name, value):
    """Refused, before anything else: their low 32 bits would be another call."""
    with pytest.raises(ValueError, match="%s=%d does not fit" % (name, value)):
        fp8.kv_attention(torch.zeros((1, 2, 64), dtype=torch.bfloat16), **{**_args(), name: value})


@pytest.mark.parametrize("value", WIDE)
@pytest.mark.parametrize("name", ["budget", "sinks", "recent", "page_size"])
def test_evict_numbers_past_32_bits(name, value):
    with pytest.raises(ValueError, match="%s=%d does not fit" % (name, value)):
        fp8.kv_evict(weights=torch.zeros((1, 2, 64)), **{**_args(), "budget": 8, name: value})
