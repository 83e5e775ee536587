"""Edges of fp8_kv_attention and fp8_kv_evict on the GPU: infinite values and
scales of V that a row sees, rows that see a single token, sequences whose
neighbours change, weights and evictions in a cache whose offsets pass 32 bits,
and batches of thousands."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import attention_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

fp8 = pytest.importorskip("fp8_precision_quantization_amd")

INF = float("inf")


@pytest.fixture(autouse=True)
def _need_gpu(gpu):
    yield


def _run(cache, n, q_heads, window=0, sinks=0, ragged=False, q=None, **more):
    q = ref.queries(cache, n, q_heads) if q is None else q
    args = cache.device()
    if ragged:
        args["q_offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32).cuda()
    args.update(more)
    say("kv_attention", dict(lens=cache.lens[:6], n=list(n)[:6], heads=cache.heads, q_heads=q_heads, dim=cache.dim,
                             k=cache.k_storage, v=cache.v_storage, scaling=cache.scaling, window=window, sinks=sinks,
                             ragged=ragged))
    out, lse = fp8.kv_attention(q.cuda(), window=window, sinks=sinks, return_lse=True, **args)
    torch.cuda.synchronize()
    return q, out, lse


def _codes(cache):
    """V's stored values before their scale, [capacity, heads, dim] fp32."""
    return cache.v.float() if cache.v_storage == "bf16" else cache.v.view(ref.TORCH_FP8[cache.v_storage]).float()


@pytest.mark.parametrize("dim, q_heads", [(64, 8), (128, 8), (128, 40), (256, 8)])
@pytest.mark.parametrize("v_st", ["e5m2", "bf16"])
def test_one_token_sees_infinite_values(v_st, dim, q_heads):
    """A positive weight times an infinite value is that infinity, whatever
    the weight's low bits are; two of opposite signs are NaN; other channels
    and the log-sum-exp stay as they are."""
    lens = [1, 33, 90, 700, 2500]
    c = ref.Cache(lens, 2, dim, 16, "e4m3", v_st, seed=dim + q_heads)
    group = q_heads // 2
    plus, minus = (INF, -INF) if v_st == "bf16" else (0x7C, 0xFC)
    want_inf = np.zeros((len(lens), q_heads, dim))
    for b, n in enumerate(lens):
        for t, h, d, x in ((0, 0, 3, plus), (n // 2, 0, 4, minus), (n - 1, 1, dim - 1, plus), (n // 3, 1, 9, minus)):
            c.v[c.rows[b][t], h, d] = x
            want_inf[b, h * group:(h + 1) * group, d] = INF if x == plus else -INF
        if n > 1:
            c.v[c.rows[b][0], 1, 17] = plus
            c.v[c.rows[b][n - 1], 1, 17] = minus
            want_inf[b, group:, 17] = np.nan
    q, out, lse = _run(c, [1] * len(lens), q_heads)
    o = out.double().cpu().numpy()
    touched = want_inf != 0
    assert np.array_equal(o[touched], want_inf[touched], equal_nan=True)
    clean = torch.from_numpy(np.where(touched, ref.attention(c, q, [1] * len(lens))[0], o))
    ref.check_attention(c, q, [1] * len(lens), clean, lse, p_bits=15)


@pytest.mark.parametrize("v_st", ["e4m3", "e5m2"])
def test_one_token_sees_an_infinite_scale(v_st):
    """The token's values become infinite with their signs (zeros NaN)."""
    lens = [1, 33, 700, 2500]
    c = ref.Cache(lens, 2, 64, 16, "e4m3", v_st, seed=3)
    c.v[:, :, 5] = 0
    at = [c.rows[b][n // 2] for b, n in enumerate(lens)]
    c.vs[at, 1] = INF
    q, out, lse = _run(c, [1] * 4, 8)
    want = (_codes(c)[at, 1] * INF)[:, None].expand(4, 4, 64)
    assert torch.isnan(want[:, :, 5]).all() and torch.isinf(want[:, :, :5]).any()
    assert np.array_equal(out[:, 4:].float().cpu().numpy(), want.numpy(), equal_nan=True)
    assert torch.isfinite(out[:, :4]).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("n", [1, 2])
def test_infinite_scale_of_a_head(n):
    """Rows that see one token: its signs; a row that sees nothing: 0."""
    c = ref.Cache([1, 0], 2, 64, 16, "e4m3", "e5m2", "head", seed=4)
    c.v[:, :, 5] = 0
    c.vs[1] = INF
    q, out, lse = _run(c, [n, n], 4)
    want = (_codes(c)[c.rows[0][0], 1] * INF).expand(2, 64).numpy()
    assert np.array_equal(out[n - 1, 2:].float().cpu().numpy(), want, equal_nan=True)
    assert torch.isfinite(out[:n, :2]).all()
    assert (out[:n - 1] == 0).all() and (out[n:] == 0).all() and torch.isneginf(lse[n:]).all()


def _single(cache, b, j):
    """What a row returns that sees token j of sequence b alone: its values
    times its scale in fp32, rounded once to bf16; [heads, dim]."""
    row = cache.rows[b][j]
    v = _codes(cache)[row]
    if cache.v_storage != "bf16":
        v = v * (cache.vs[row] if cache.scaling == "token_head" else cache.vs)[:, None]
    return v.to(torch.bfloat16)


def _pow2_scales(cache):
    if cache.v_storage != "bf16" and cache.scaling == "token_head":
        cache.vs = torch.exp2(torch.floor(torch.log2(cache.vs)))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("v_st, scaling", [("bf16", "token_head"), ("e4m3", "token_head"),
                                           ("e5m2", "token_head"), ("e4m3", "head"), ("e5m2", "head")])
def test_rows_of_a_single_token_return_it(v_st, scaling, dim):
    """Several tokens at once: a row's only weight is 1 exactly, so a value
    (with scales per token: powers of two, any scale per head) comes back bit
    for bit."""
    lens = [40, 200]
    c = ref.Cache(lens, 2, dim, 16, "e4m3", v_st, scaling, seed=dim)
    _pow2_scales(c)
    for n, window, ragged in (([40, 40], 1, False), ([40, 133], 1, True), ([40, 200], 0, True)):
        q, out, lse = _run(c, n, 6, window, 0, ragged)
        at = 0
        for b in range(2):
            for i in range(n[b]):
                j = lens[b] - n[b] + i
                if window == 1 or j == 0:
                    want = _single(c, b, j).repeat_interleave(3, 0)
                    assert torch.equal(out[at + i].cpu(), want), (b, i)
            at += n[b]


@pytest.mark.parametrize("v_st, scaling", [("bf16", "token_head"), ("e4m3", "token_head"), ("e4m3", "head")])
def test_single_token_of_a_split_row(v_st, scaling):
    """The same where several blocks share a row's tokens, of which one is there."""
    n, length, there = 5, 2100, 1700
    c = ref.Cache([length], 2, 64, 1, "e4m3", v_st, scaling, seed=7,
                  absent=[(0, p) for p in range(length) if p != there])
    _pow2_scales(c)
    q, out, lse = _run(c, [n], 4)
    want = _single(c, 0, there).repeat_interleave(2, 0)
    for i in range(n):
        assert torch.equal(out[i].cpu(), want)


@pytest.mark.parametrize("n", [[1] * 4, [3, 2, 70, 1]])
@pytest.mark.parametrize("target", [0, 2])
def test_neighbours_contents_do_not_matter(n, target):
    """Other codes, scales and queries in the other sequences, of the same
    lengths: not a bit of this one's results changes."""
    lens = [700, 3, 2500, 41]
    c = ref.Cache(lens, 2, 128, 16, seed=6)
    ragged = len(set(n)) > 1
    q = ref.queries(c, n, 8)
    first = sum(n[:target])
    mine = slice(first, first + n[target])
    results = []
    for other in (False, True):
        if other:
            theirs = np.concatenate([c.rows[b] for b in range(4) if b != target])
            g = torch.Generator().manual_seed(11)
            for x in (c.k, c.v):
                x[theirs] = torch.randint(0, 0x7F, x[theirs].shape, generator=g, dtype=torch.uint8)
            for x in (c.ks, c.vs):
                x[theirs] *= 1 + torch.rand(x[theirs].shape, generator=g)
            keep = q[mine].clone()
            q = ref.queries(c, n, 8, seed=12)
            q[mine] = keep
        w = torch.zeros(4, 2, c.max_len, device="cuda")
        _, out, lse = _run(c, n, 8, ragged=ragged, q=q, weights=w)
        results.append((out[mine].clone(), lse[mine].clone(), w[target].clone(), out, w))
    for a, b in zip(results[0][:3], results[1][:3]):
        assert torch.equal(a, b)
    assert not torch.equal(results[0][3], results[1][3]) and not torch.equal(results[0][4], results[1][4])


class _Long:
    """A cache of more than 2^32 bytes with a small one's rows at its end."""

    def __init__(self, small):
        heads, dim, page = small.heads, small.dim, small.page
        capacity = (1 << 32) // (heads * dim) + 2 * small.capacity
        self.first = capacity - small.capacity
        self.first -= self.first % page
        end = slice(self.first, self.first + small.capacity)
        self.args = dict(page_size=page, lens=torch.tensor(small.lens, dtype=torch.int32).cuda(),
                         page_table=torch.from_numpy(small.table + self.first // page).cuda())
        for name, part in (("k_cache", small.k), ("v_cache", small.v)):
            t = torch.zeros((capacity, heads, dim), dtype=torch.uint8, device="cuda")
            t[end] = part.cuda()
            self.args[name] = t
        for name, part in (("k_scale_inv", small.ks), ("v_scale_inv", small.vs)):
            t = torch.ones((capacity, heads), device="cuda")
            t[end] = part.cuda()
            self.args[name] = t
        self.end = end


@pytest.mark.parametrize("n", [[1, 1], [9, 30]])
def test_weights_past_2_31_elements(n):
    """The keys that the weights are made from lie past 32-bit offsets."""
    small = ref.Cache([200, 90], 8, 128, 16, seed=9)
    long = _Long(small)
    q = ref.queries(small, n, 16)
    if n[0] > 1:
        long.args["q_offsets"] = torch.tensor([0, n[0], sum(n)], dtype=torch.int32).cuda()
    w = torch.zeros(2, 8, small.max_len, device="cuda")
    say("long cache, weights", n)
    out, lse = fp8.kv_attention(q.cuda(), weights=w, return_lse=True, **long.args)
    torch.cuda.synchronize()
    want, delta, acc = ref.check_attention(small, q, n, out, lse)
    for b, x in enumerate(want):
        got = w[b].double().cpu().numpy()
        bound = (2 * float(delta.max()) + acc + 2.0 ** -20) * (x + 1e-6 * n[b]) + 2.0 ** -23 * x
        assert (np.abs(got[:, :small.lens[b]] - x) <= bound).all()
        assert (got[:, small.lens[b]:] == 0).all()


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_past_2_31_elements(in_place):
    """The same rows move as in a small cache, and nothing below them changes."""
    small = ref.Cache([700, 333, 60], 8, 128, 16, seed=10, slack_pages=3 * 10)
    dst = np.setdiff1d(np.arange(small.capacity // 16), small.table.ravel())[:30].reshape(3, 10).astype(np.int32)
    w = torch.rand(3, 8, small.max_len, generator=torch.Generator().manual_seed(5)).cuda()
    long = _Long(small)
    results = []
    for args, at in ((small.device(), 0), (long.args, long.first)):
        args = {k: v for k, v in args.items() if k not in ("k_storage", "v_storage", "scaling")}
        table = None if in_place else torch.from_numpy(dst + at // 16).cuda()
        ww = w.clone()
        say("evict, first row", at, "in place", in_place)
        kept, lens = fp8.kv_evict(weights=ww, budget=160, sinks=4, recent=50, dst_page_table=table, **args)
        torch.cuda.synchronize()
        rows = slice(at, at + small.capacity)
        results.append([kept, lens, ww] + [args[x][rows] for x in ("k_cache", "v_cache", "k_scale_inv", "v_scale_inv")])
    for a, b in zip(*results):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    assert not long.args["k_cache"][:long.first].any() and not long.args["v_cache"][:long.first].any()
    assert (long.args["k_scale_inv"][:long.first] == 1).all()


@pytest.mark.parametrize("ragged", [False, True])
def test_thousands_of_sequences(ragged):
    """Shares and row tiles found among 3000 short sequences, empty ones among them."""
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(0, 40, 3000)]
    n = [int(x) for x in rng.integers(0, 4, 3000)] if ragged else [1] * 3000
    c = ref.Cache(lens, 1, 32, 8, seed=25)
    q, out, lse = _run(c, n, 2, ragged=ragged)
    ref.check_attention(c, q, n, out, lse, p_bits=8 if ragged else 15)


@pytest.mark.parametrize("same_cache", [True, False])
@pytest.mark.parametrize("in_place", [True, False])
def test_evict_where_k_and_v_share_arrays(same_cache, in_place):
    """One array for K and V, or for their scales alone, moves once."""
    lens, budget = [9500, 4097, 60], 4300
    c = ref.Cache(lens, 2, 32, 16, seed=12, slack_pages=3 * 270)
    dst = np.setdiff1d(np.arange(c.capacity // 16), c.table.ravel())[:3 * 270].reshape(3, 270).astype(np.int32)
    args = c.device()
    args["v_scale_inv"] = args["k_scale_inv"]
    if same_cache:
        args["v_cache"] = args["k_cache"]
    before = {x: args[x].clone() for x in ("k_cache", "v_cache", "k_scale_inv")}
    w = torch.rand(3, 2, c.max_len, generator=torch.Generator().manual_seed(6))
    say("evict, shared arrays", same_cache, in_place)
    kept, new_lens = fp8.kv_evict(weights=w.cuda(), budget=budget, sinks=4, recent=100,
                                  dst_page_table=None if in_place else torch.from_numpy(dst).cuda(), **args)
    torch.cuda.synchronize()
    want = {x: t.clone() for x, t in before.items()}
    to_table = c.table if in_place else dst
    for b, n in enumerate(lens):
        m = min(n, budget)
        r = np.arange(m)
        to = torch.from_numpy(to_table[b, r // 16].astype(np.int64) * 16 + r % 16).cuda()
        for h in range(2):
            keep = ref.evict(w[b, h].numpy(), n, budget, 4, 100)
            assert np.array_equal(kept[b, h, :m].cpu().numpy(), keep)
            src = torch.from_numpy(c.table[b, keep // 16].astype(np.int64) * 16 + keep % 16).cuda()
            for x in want:
                want[x][to, h] = before[x][src, h]
    for x in want:
        assert torch.equal(args[x].view(torch.uint8), want[x].view(torch.uint8)), x
