"""fp8_lora_add where values are infinite or near the end of fp32: an infinite
A x or B gives the infinity that the formula gives, the largest finite values
stay finite, and nothing else changes by a bit."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_lora import DTYPES, Case

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(autouse=True)
def _need_gpu(gpu):
    yield


def positive(rows, rank, dtype, columns=(72, 56), exact=False):
    """A, B and the gains are positive, the rows of x of one sign each: every product of row m has the sign of x[m].
    exact: A x is a power of two, so that its second and third bf16 terms are 0."""
    c = Case(rows, columns=columns, rank=rank, dtype=dtype, none=0.0, adapters=3, seed=rank)
    sign = 1.0 - 2.0 * (torch.arange(rows, device="cuda") % 2)
    c.a, c.b = c.a.abs() + 0.125, c.b.abs() + 0.125
    c.x_all[:, :] = ((c.x_all.float().abs() + 0.125) * sign[:, None]).to(torch.bfloat16)
    if exact:
        c.a.fill_(2.0 ** -8)
        c.x_all[:, :] = sign[:, None].to(torch.bfloat16)
        c.gain.fill_(1.0)
    return c, sign


ROWS = [20, 64, 90, 700, 1100]        # one launch, two (a wave or a block sorts), three
RANKS = [8, 16, 32, 40, 64, 72, 96, 128]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rank", RANKS)
@pytest.mark.parametrize("rows", ROWS)
def test_infinite_x(rows, rank, dtype):
    c, sign = positive(rows, rank, dtype)
    good = c.run()
    assert good.isfinite().all()
    c.x_all[7, 3], c.x_all[12, 100] = -INF, INF
    got = c.run()
    others = torch.ones(rows, dtype=torch.bool)
    others[[7, 12]] = False
    assert torch.equal(got[others], good[others])
    assert (got[7] == -INF).all() and (got[12] == INF).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("exact", [False, True], ids=["any", "exact"])
@pytest.mark.parametrize("rank", RANKS)
@pytest.mark.parametrize("rows", ROWS)
def test_infinite_b(rows, rank, exact, dtype):
    """One infinite element makes its column of its adapter's rows infinite, and nothing else."""
    c, sign = positive(rows, rank, dtype, exact=exact)
    good = c.run()
    for l, column, r, value in ((0, 5, rank - 1, INF), (1, 100, 0, -INF), (2, 71, rank // 2, INF)):
        c.b[l, column, r] = value
    want = good.clone()
    for l, column, value in ((0, 5, INF), (1, 100, -INF), (2, 71, INF)):
        mine = c.ids == l
        want[mine, column] = (sign[mine] * value).to(dtype)
    got = c.run()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("value", [INF, -INF])
@pytest.mark.parametrize("rank", [8, 32, 40, 128])
@pytest.mark.parametrize("rows", ROWS)
def test_both_infinite(rows, rank, value, dtype):
    """Every element of A x is +inf, B's others are positive: with +inf in B the sum is +inf, with -inf it has both."""
    c, sign = positive(rows, rank, dtype)
    c.x_all[4, 9] = INF
    l = int(c.ids[4])
    c.b[l, 3, 1] = value
    got = c.run()
    assert got[4, 3] == INF if value > 0 else got[4, 3].isnan()
    rest = torch.cat([got[4, :3], got[4, 4:]])
    assert (rest == INF).all()


@pytest.mark.parametrize("rows", [20, 90, 1100])
def test_nan_stays_nan(rows):
    """What the formula does not define: opposite infinities, an infinity times zero, NaN itself."""
    c, sign = positive(rows, 16, torch.bfloat16)
    c.x_all[4, 9], c.x_all[4, 10], c.x_all[6, 2] = INF, -INF, float("nan")
    c.x_all[8] = 0
    c.b[:, 3, 1] = INF
    got = c.run()
    assert got[4].isnan().all() and got[6].isnan().all()
    assert got[8, 3].isnan() and got[8, :3].isfinite().all() and got[8, 4:].isfinite().all()


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rank", [8, 32, 40, 64, 128])
@pytest.mark.parametrize("rows", [20, 90, 1100])
def test_largest_values(rows, rank, dtype):
    """A x = +-(0x1.FEp127 + 1.5 * 2^119): finite, but its nearest bf16 is infinite.  With B near 2^-100 the product
    is an ordinary number."""
    c = Case(rows, columns=(72, 56), rank=rank, dtype=dtype, none=0.0, adapters=3, seed=rank)
    c.a.zero_()
    c.a[:, :, 0], c.a[:, :, 1] = 1.9921875, 1.5
    c.a[:, 1::2].neg_()
    c.x_all.zero_()
    c.x_all[:, 0], c.x_all[:, 1] = 2.0 ** 127, 2.0 ** 119
    c.x_all[1::2].neg_()
    c.b = (c.b.float() * 2.0 ** -100).to(torch.bfloat16)
    t = c.x[0].double() @ c.a[0, 0].double()
    assert 2.0 ** 128 * (1 - 2.0 ** -9) <= float(t) < 2.0 ** 128
    c.check(c.run(gain=None), gain=False)
