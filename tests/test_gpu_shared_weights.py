"""Accumulated weights of fp8_kv_attention_shared: the prefix's keys are those
of the first row's pages for them too."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import attention_ref as ref
from tests.test_gpu_shared import NEW, SharedCache, _heads, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(gpu):
    yield


@pytest.mark.parametrize("storage", [("e4m3", "e4m3", "token_head"), ("e5m2", "e4m3", "head"),
                                     ("bf16", "bf16", "token_head")], ids="-".join)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", NEW)
def test_other_rows_are_not_read(new, dim, storage):
    """The other rows' entries of the prefix name pages of NaN; sequences end inside it and behind it."""
    n = NEW[new]
    c = SharedCache([400, 350, max(130, n[2]), 500, 384], 320, 2, dim, 32, *storage, seed=dim)
    start = torch.rand(5, 2, c.max_len).cuda()
    w = start.clone()
    q, out, lse = _run(c, n, _heads(new, 4), weights=w)
    weights, delta, acc = ref.check_attention(c, q, n, out, lse)
    w, start = w.double().cpu().numpy(), start.double().cpu().numpy()
    at = 0
    for b in range(5):
        L = c.lens[b]
        d = delta[at:at + n[b]].max()
        at += n[b]
        got = w[b, :, :L] - start[b, :, :L]
        # the score's error in the weight and in the row's lse, an fp32 lse, sums of up to rows terms and the addition
        bound = weights[b] * (2 * d + 4 * acc + 2.0 ** -18) + (weights[b] + 1) * 64 * 2.0 ** -24
        assert (np.abs(got - weights[b]) <= bound).all()
        assert np.array_equal(w[b, :, L:], start[b, :, L:])
