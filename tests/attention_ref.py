"""Plain float64 reference of attention over the paged KV cache and of the
eviction by accumulated weight, and the caches the GPU tests read: random
codes in shuffled pages, with everything that must not be read (rows of no
sequence, rows behind a sequence's end) holding NaN codes and NaN scales."""
from __future__ import annotations

import math

import numpy as np
import torch

TORCH_FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
NAN_CODE = {"e4m3": 0x7F, "e5m2": 0x7F}


class Cache:
    """Host copy of a layer's K and V for a batch: values k64, v64 [batch][len, heads, dim]."""

    def __init__(self, lens, heads, dim, page=16, k_storage="e4m3", v_storage="e4m3", scaling="token_head", seed=0,
                 slack_pages=3, absent=()):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.lens, self.heads, self.dim, self.page = list(lens), heads, dim, page
        self.k_storage, self.v_storage, self.scaling = k_storage, v_storage, scaling
        pages = max(1, -(-max(lens) // page)) if lens else 1
        total = len(lens) * pages + slack_pages
        perm = rng.permutation(total)
        self.table = perm[:len(lens) * pages].reshape(len(lens), pages).astype(np.int32)
        self.capacity = total * page
        self.max_len = pages * page
        self.rows = []
        for b, n in enumerate(lens):
            j = np.arange(n)
            self.rows.append(self.table[b, j // page].astype(np.int64) * page + j % page)
        for which, st in (("k", k_storage), ("v", v_storage)):
            x = torch.randn(self.capacity, heads, dim, generator=g, dtype=torch.float32)
            if which == "k":
                x[:, :, 1::13] *= 3.0
            x *= torch.exp2(torch.rand(self.capacity, heads, 1, generator=g) * 4 - 2)
            live = np.zeros(self.capacity, bool)
            for r in self.rows:
                live[r] = True
            dead = torch.from_numpy(~live)
            if st == "bf16":
                data = x.to(torch.bfloat16)
                val = data.double()
                data[dead] = float("nan")
                sinv = None
            else:
                amax = x.abs().amax(2) if scaling == "token_head" else x.abs().amax((0, 2)) * 0.9
                sinv = (amax.clamp(min=1e-20) / FMAX[st]).float()
                s = sinv[:, :, None] if scaling == "token_head" else sinv[None, :, None]
                data = (x / s).clamp(-FMAX[st], FMAX[st]).to(TORCH_FP8[st]).view(torch.uint8)
                val = data.view(TORCH_FP8[st]).double() * s.double()
                data[dead] = NAN_CODE[st]
                if scaling == "token_head":
                    sinv[dead] = float("nan")
            setattr(self, which, data)
            setattr(self, which + "s", sinv)
            setattr(self, which + "64", [val[torch.from_numpy(r)].numpy() for r in self.rows])
        # tokens of absent pages: (sequence, page) whose table entry names no page
        self.there = [np.ones(n, bool) for n in lens]
        for b, p in absent:
            self.there[b][p * page:(p + 1) * page] = False
            self.table[b, p] = -1 if (b + p) % 2 else total + 5

    def device(self):
        def put(t):
            return None if t is None else t.cuda()
        return dict(k_cache=put(self.k), v_cache=put(self.v),
                    page_table=torch.from_numpy(self.table).cuda(),
                    lens=torch.tensor(self.lens, dtype=torch.int32).cuda(), page_size=self.page,
                    k_scale_inv=put(self.ks), v_scale_inv=put(self.vs), k_storage=self.k_storage,
                    v_storage=self.v_storage, scaling=self.scaling)


def queries(cache, n, q_heads, seed=1, scale=0.5):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(sum(n), q_heads, cache.dim, generator=g)).to(torch.bfloat16)


def attention(cache, q, n, window=0, sinks=0, scale=None):
    """float64: out, lse, weights [batch][heads, len], and the bounds' parts
    (sum of p|v| per output, the score error delta per row)."""
    H, D = cache.heads, cache.dim
    q64 = q.double().numpy()
    G = q64.shape[1] // H
    scale = D ** -0.5 if scale is None else scale
    out = np.zeros(q64.shape)
    lse = np.full(q64.shape[:2], -np.inf)
    pv = np.zeros(q64.shape)
    delta = np.zeros(q64.shape[:2])
    weights = []
    at = 0
    for b, nb in enumerate(n):
        L = cache.lens[b]
        k, v = cache.k64[b], cache.v64[b]
        w = np.zeros((H, L))
        pos = L - nb + np.arange(nb)
        j = np.arange(L)
        see = (j[None] <= pos[:, None]) & cache.there[b][None]
        if window:
            see &= (j[None] > pos[:, None] - window) | (j[None] < sinks)
        some = see.any(1)
        for x in range(q64.shape[1]):
            qq = q64[at:at + nb, x]
            s = np.where(see, qq @ k[:, x // G].T * scale, -np.inf)
            m = np.where(some, s.max(1, initial=-np.inf), 0.0)
            e = np.exp(s - m[:, None])
            tot = e.sum(1)
            with np.errstate(divide="ignore", invalid="ignore"):
                p = np.where(some[:, None], e / tot[:, None], 0.0)
                lse[at:at + nb, x] = np.where(some, m + np.log(tot), -np.inf)
            vv = np.where(see.any(0)[:, None], v[:, x // G], 0.0)
            out[at:at + nb, x] = p @ vv
            pv[at:at + nb, x] = p @ np.abs(vv)
            w[x // G] += p.sum(0)
            sa = np.where(see, np.abs(qq) @ np.abs(k[:, x // G]).T * abs(scale), 0.0).max(1, initial=0.0)
            # the score: D products summed in fp32, three scalings and the
            # exponent's argument (a rounding each), and 2^x to 2 ulp
            delta[at:at + nb, x] = (D + 8) * 2.0 ** -24 * sa * math.log2(math.e) + 2.0 ** -22
        weights.append(w)
        at += nb
    return out, lse, weights, pv, delta


def check_attention(cache, q, n, got_out, got_lse, window=0, sinks=0, scale=None, p_bits=8):
    """out within: its bf16 rounding (2^-8), the weights' rounding to p_bits,
    the scores' error twice (weight and sum) and fp32 sums of len terms."""
    out, lse, weights, pv, delta = attention(cache, q, n, window, sinks, scale)
    o = got_out.double().cpu().numpy()
    longest = max(cache.lens) if cache.lens else 0
    acc = (longest + 64) * 2.0 ** -24
    bound = 2.0 ** -8 * np.abs(out) + (2.0 ** -p_bits + 2 * delta[..., None] + 2 * acc) * pv * 1.01
    err = np.abs(o - out)
    assert np.isfinite(o).all(), "out not finite at %s" % (np.argwhere(~np.isfinite(o))[:3],)
    assert (err <= bound + 1e-30).all(), (err.max(), np.argwhere(err > bound + 1e-30)[:3], float((err / (bound + 1e-30)).max()))
    if got_lse is not None:
        z = got_lse.double().cpu().numpy()
        empty = np.isneginf(lse)
        assert np.array_equal(empty, np.isneginf(z))
        zb = delta + acc + 2.0 ** -22 * (1 + np.abs(np.where(empty, 0, lse)))
        ze = np.abs(np.where(empty, 0, z) - np.where(empty, 0, lse))
        assert (ze <= zb).all(), (ze.max(), float((ze / zb).max()))
    return weights, delta, acc


def evict(weights, n, budget, sinks, recent):
    """Positions kept by one head of a sequence of n tokens (increasing)."""
    if n <= budget:
        return np.arange(n)
    lo, hi = sinks, n - recent
    mid = np.arange(lo, hi)
    w = weights[lo:hi].astype(np.float64)
    key = np.where(np.isnan(w), np.inf, w)
    nan = np.isnan(w)
    best = mid[np.lexsort((mid, -key, ~nan))][:budget - sinks - recent]
    return np.sort(np.concatenate([np.arange(lo), best, np.arange(hi, n)]))
