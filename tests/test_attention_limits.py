"""Sizes at the limits of fp8_kv_attention and fp8_kv_evict, checked without a
GPU through the workspace query and the calls' own refusals.  Pointers are
fake and never dereferenced."""
from __future__ import annotations

import ctypes

import pytest

from fp8_precision_quantization_amd import _lib as L
from tests.test_attention_boundary import U, attention, check, evict, pair


def size(p, total, q_heads, ragged=0, window=0, sinks=0, weighted=0):
    return L.lib().fp8_kv_attention_workspace(ctypes.byref(p), total, q_heads, ragged, window, sinks, weighted)


@pytest.mark.parametrize("group", [1, 3, 64, 1000])
@pytest.mark.parametrize("ragged", [0, 1])
def test_rows_stay_in_32_bits(group, ragged):
    """The kernels count (token, head) rows in 32 bits and round them up to
    tiles: one KV head's rows must leave room for that."""
    p = pair(batch=1, heads=1, head_dim=16)
    most = min(((1 << 31) - 256) // group, (1 << 30) - 1)
    assert size(p, most, group, ragged) >= 0
    for total in (most + 1, ((1 << 31) - 1) // group, ((1 << 31) - 64) // group):
        if total <= most:
            continue
        assert size(p, total, group, ragged) == -1 and "total_q" in L.lib().fp8_last_error().decode()
        check(attention(p, total_q=total, q_heads=group, ldq=16 * 1000, ldo=16 * 1000, q_offsets=0x10000 * ragged or None),
              U, "total_q")


@pytest.mark.parametrize("p, q, status", [
    # sequences of several tokens: a tile of 128 rows each, by every KV head
    (dict(batch=65535, heads=256), dict(total_q=65535, q_heads=256, ragged=1), U),
    (dict(batch=65000, heads=255), dict(total_q=65000, q_heads=255, ragged=1), 0),
    (dict(batch=65535, heads=512), dict(total_q=65535, q_heads=512, ragged=1), U),
    (dict(batch=32768, heads=512), dict(total_q=65536, q_heads=512), U),
    (dict(batch=32767, heads=512), dict(total_q=65534, q_heads=512), 0),
    (dict(batch=65535, heads=512), dict(total_q=65535, q_heads=512), 0),            # one token each
    # weights: a block for 128 tokens of a KV head, 256 of the last token's stored scores
    (dict(batch=1, heads=8, max_len=1 << 28), dict(total_q=2, q_heads=8, weighted=1), U),
    (dict(batch=1, heads=8, max_len=(1 << 28) - 128), dict(total_q=2, q_heads=8, weighted=1), 0),
    (dict(batch=1, heads=8, max_len=1 << 28), dict(total_q=2, q_heads=8), 0),
    (dict(batch=1, heads=8, max_len=1 << 28), dict(total_q=1, q_heads=8, weighted=1), 0),
    (dict(batch=1, heads=8, max_len=1 << 29), dict(total_q=1, q_heads=8, weighted=1), U),
    (dict(batch=1, heads=8, max_len=1 << 29), dict(total_q=1, q_heads=8, weighted=1, window=4096), 0),
    (dict(batch=1, heads=8, max_len=1 << 28), dict(total_q=1, q_heads=1024, weighted=1), U),
])
def test_launches_stay_below_2_32_threads(p, q, status):
    """A launch of more is refused by the runtime or wraps to fewer blocks."""
    c = pair(**{**dict(head_dim=16, page_size=1 << 20, page_ld=512), **p})
    got = size(c, q["total_q"], q["q_heads"], q.get("ragged", 0), q.get("window", 0), 0, q.get("weighted", 0))
    if status == 0:
        assert got >= 0, L.lib().fp8_last_error()
        return
    assert got == -1 and "2^24" in L.lib().fp8_last_error().decode()
    w = c.max_len if q.get("weighted") else 0
    check(attention(c, total_q=q["total_q"], q_heads=q["q_heads"], ldq=16 * q["q_heads"], ldo=16 * q["q_heads"],
                    q_offsets=0x10000 if q.get("ragged") else None, weights=0x10000 if w else None, ldw=w), status, "2^24")


@pytest.mark.parametrize("budget", [1 << 30, (1 << 31) - 1])
def test_budget_stays_below_2_30(budget):
    """No sequence is longer; loops over a larger budget would pass 2^31."""
    check(evict(budget=budget), U, "budget")
