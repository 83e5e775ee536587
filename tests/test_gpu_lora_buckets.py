"""fp8_lora_add where the rows of several adapters share a tile: ids that are
equal modulo the sort's 1024 buckets, beside rows without an adapter, over
several inner steps, parts and column steps."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_lora import DTYPES, Case

pytestmark = pytest.mark.gpu

ADAPTERS = 2050
USED = [0, 1024, 2048, 1023, 2047]       # buckets 1, 1, 1, 0, 0; rows without an adapter are in bucket 0


@pytest.fixture(autouse=True)
def _need_gpu(gpu):
    yield


class Shared(Case):
    def __init__(self, rows, inner, columns, rank, dtype, seed=0):
        super().__init__(rows, inner=inner, columns=columns, rank=rank, adapters=len(USED), dtype=dtype, none=0.15,
                         seed=seed, pad=8)
        self.small = {k: getattr(self, k) for k in ("a", "b", "gain", "ids")}
        at = torch.tensor(USED, device="cuda")
        live = (self.ids >= 0) & (self.ids < len(USED))
        ids = at[self.ids.long().clamp(0, len(USED) - 1)].int()
        # the values of ids without an adapter differ too: 2049 has none of its own here
        self.wide_ids = torch.where(live, ids, torch.where(self.ids == len(USED), ADAPTERS, self.ids))
        self.wide = []
        for t in (self.a, self.b, self.gain):
            w = torch.full((ADAPTERS,) + t.shape[1:], float("nan"), dtype=t.dtype, device="cuda")
            w[at] = t
            self.wide.append(w)

    def run_wide(self, **more):
        n, (a, b, gain), ids = self.adapters, self.wide, self.wide_ids
        self.a, self.b, self.gain, self.ids, self.adapters = a, b, gain, ids, ADAPTERS
        out = self.run(**more)
        self.a, self.b, self.gain, self.ids = (self.small[k] for k in ("a", "b", "gain", "ids"))
        self.adapters = n
        return out


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rank, inner, columns", [(16, 1000, (1000, 264)), (40, 2056, (1032, 248)), (64, 1400, (2056,)),
                                                  (128, 520, (264, 8, 520))])
@pytest.mark.parametrize("rows", [50, 400, 1500])
def test_shared_tiles(rows, rank, inner, columns, dtype):
    c = Shared(rows, inner, columns, rank, dtype, seed=rank)
    out = c.run_wide()
    c.check(out)
    assert torch.equal(c.run_wide(), out)
    # in place
    assert torch.equal(c.run_wide(out=c.y), out)
