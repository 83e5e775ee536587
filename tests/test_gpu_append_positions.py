"""fp8_kv_append's positions of several axes in one row of memory: what text
tokens have beside pictures, where every axis counts the same."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_append import Case

pytestmark = pytest.mark.gpu

fp8 = pytest.importorskip("fp8_precision_quantization_amd")


@pytest.fixture(autouse=True)
def _need_gpu(gpu):
    yield


def _caches(c):
    return [c.cache["k"].clone(), c.cache["v"].clone(), c.scale["k"].clone(), c.scale["v"].clone()]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n, sections", [(1, (16, 16)), (2, (8, 12, 12)), (65, (8, 12, 12)), (700, (3, 5, 7, 17))])
def test_expanded_axes(n, sections, interleaved):
    c = Case(n=n, sections=sections, interleaved=interleaved, padding=0, seed=n)
    row = c.pos[0].cuda()
    c.pos = c.pos[:1].repeat(len(sections), 1)
    want = c.call(positions=c.pos.cuda())
    c.check(want)
    caches = _caches(c)
    got = c.call(positions=row.expand(len(sections), n))
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(_caches(c), caches))


def test_axes_apart_and_overlapping():
    c = Case(n=65, sections=(16, 16), padding=0, seed=4)
    want = c.call()
    wide = torch.zeros(2, 80, dtype=torch.int64, device="cuda")
    wide[:, :65] = c.pos.cuda()
    assert torch.equal(c.call(positions=wide[:, :65]), want)
    line = torch.arange(200, device="cuda")
    for stride in (1, 64):
        with pytest.raises(ValueError, match="axes"):
            c.call(positions=line.as_strided((2, 65), (stride, 1)))
    with pytest.raises(ValueError, match="contiguous last dimension"):
        c.call(positions=line.as_strided((2, 65), (1, 2)))
    assert torch.equal(c.call(), want)
