"""Boundary checks of fp8_kv_attention and fp8_kv_evict that run without a
GPU: every invalid argument is rejected before any device call, with a
message that names it.  Pointers are fake and never dereferenced."""
from __future__ import annotations

import ctypes

import pytest

from fp8_precision_quantization_amd import _lib as L

FAKE = 0x10000
I, U, M = L.FP8_ERR_INVALID_ARG, L.FP8_ERR_UNSUPPORTED_SHAPE, L.FP8_ERR_MISALIGNED


def pair(**change):
    f = dict(k=FAKE, v=FAKE, k_scale_inv=FAKE, v_scale_inv=FAKE, capacity=4096, page_table=FAKE, page_ld=16, lens=FAKE,
             max_len=256, k_storage=L.FP8_KV_E4M3, v_storage=L.FP8_KV_BF16, scaling=L.FP8_KV_PER_TOKEN_HEAD, heads=8,
             head_dim=128, page_size=16, batch=2, reserved=0)
    f.update(change)
    return L.Fp8KvPair(**f)


def attention(p=None, **change):
    a = dict(q=FAKE, ldq=4096, total_q=2, q_heads=32, q_offsets=None, scale=0.1, window=0, sinks=0, out=FAKE, ldo=4096,
             lse=FAKE, weights=None, ldw=0, ws=FAKE, wsb=1 << 30)
    a.update(change)
    p = p or pair()
    return L.lib().fp8_kv_attention(ctypes.byref(p), a["q"], a["ldq"], a["total_q"], a["q_heads"], a["q_offsets"],
                                    a["scale"], a["window"], a["sinks"], a["out"], a["ldo"], a["lse"], a["weights"],
                                    a["ldw"], a["ws"], a["wsb"], None)


def evict(p=None, **change):
    a = dict(weights=FAKE, ldw=256, budget=64, sinks=4, recent=16, dst=None, dst_ld=0, wo=None, ldwo=0, kept=FAKE,
             lens=2 * FAKE)
    a.update(change)
    p = p or pair()
    return L.lib().fp8_kv_evict(ctypes.byref(p), a["weights"], a["ldw"], a["budget"], a["sinks"], a["recent"],
                                a["dst"], a["dst_ld"], a["wo"], a["ldwo"], a["kept"], a["lens"], None)


def check(got, status, word):
    assert got == status, (got, L.lib().fp8_last_error())
    assert word in L.lib().fp8_last_error().decode()


PAIRS = [
    (dict(k=None), I, "cache is NULL"), (dict(v=None), I, "cache is NULL"), (dict(k=FAKE + 8), M, "16-byte"),
    (dict(k_scale_inv=None), I, "scale_inv"), (dict(v_storage=0, v_scale_inv=None), I, "scale_inv"),
    (dict(v_storage=0, v_scale_inv=FAKE + 2), M, "scale_inv"),
    (dict(k_storage=3), I, "storage"), (dict(scaling=2), I, "scaling"), (dict(reserved=1), I, "reserved"),
    (dict(head_dim=8), U, "head_dim"), (dict(head_dim=120), U, "head_dim"), (dict(head_dim=272), U, "head_dim"),
    (dict(heads=0), I, "heads"), (dict(batch=-1), I, "batch"), (dict(batch=65536), U, "batch"),
    (dict(max_len=-1), I, "max_len"), (dict(max_len=1 << 30), U, "max_len"), (dict(capacity=1 << 31), U, "capacity"),
    (dict(capacity=-1), I, "capacity"),
    (dict(page_size=0), U, "page_size"), (dict(page_size=24), U, "page_size"), (dict(page_size=1 << 21), U, "page_size"),
    (dict(page_ld=15), I, "page_ld"), (dict(lens=None), I, "lens"), (dict(page_table=None), I, "page_table"),
    (dict(lens=FAKE + 2), M, "lens"), (dict(page_table=FAKE + 1), M, "page_table"),
]


@pytest.mark.parametrize("change, status, word", PAIRS, ids=lambda x: str(x) if isinstance(x, dict) else "")
def test_pair(change, status, word):
    check(attention(pair(**change)), status, word)
    check(evict(pair(**change)), status, word)


@pytest.mark.parametrize("change, status, word", [
    (dict(q=None), I, "q is NULL"), (dict(out=None), I, "out is NULL"), (dict(q=FAKE + 8), M, "16-byte"),
    (dict(out=FAKE + 2), M, "16-byte"), (dict(ldq=4088), I, "ldq"), (dict(ldo=4095), I, "ldo"),
    (dict(ldq=4100), M, "ldq"), (dict(ldo=4097), M, "ldo"), (dict(total_q=-1), I, "total_q"),
    (dict(total_q=3), I, "multiple of batch"), (dict(q_heads=0), I, "q_heads"), (dict(q_heads=12), I, "q_heads"),
    (dict(total_q=1 << 28), U, "total_q"), (dict(total_q=1 << 30, q_heads=8), U, "total_q"), (dict(window=-1), I, "window"), (dict(sinks=-2), I, "sinks"),
    (dict(scale=float("inf")), I, "scale"), (dict(scale=float("nan")), I, "scale"),
    (dict(q_offsets=FAKE + 2), M, "q_offsets"), (dict(lse=FAKE + 2), M, "lse"),
    (dict(weights=FAKE, ldw=256, lse=None), I, "lse"), (dict(weights=FAKE, ldw=255), I, "ldw"),
    (dict(weights=FAKE + 2, ldw=256), M, "weights"),
])
def test_attention(change, status, word):
    check(attention(**change), status, word)


def test_attention_workspace():
    lib = L.lib()

    def size(p, total=2, q_heads=32, ragged=0, window=0, sinks=0, weighted=0):
        return lib.fp8_kv_attention_workspace(ctypes.byref(p), total, q_heads, ragged, window, sinks, weighted)

    long = pair(max_len=65536, page_ld=4096)
    need = size(long)
    assert need > 0
    check(attention(long, wsb=need - 1), I, "workspace_bytes")
    check(attention(long, ws=None), I, "workspace is NULL")
    check(attention(long, ws=FAKE + 8), M, "workspace")
    assert size(pair(max_len=32, page_ld=2)) == 0        # one split
    assert size(long, window=16) < need
    weighted = size(long, weighted=1)                   # the scores too
    assert weighted >= need + 2 * 32 * 65536 * 4
    check(attention(long, wsb=weighted - 1, weights=FAKE, ldw=65536), I, "workspace_bytes")
    assert size(long, q_heads=1024, weighted=1) == size(long, q_heads=1024)       # keys read again instead
    assert size(pair(batch=0), total=0) == 0
    # sizes alone: no pointer is needed
    assert size(pair(k=None, v=None, k_scale_inv=None, v_scale_inv=None, lens=None, page_table=None, max_len=65536,
                     page_ld=4096)) == need
    assert size(long, total=3) == -1 and "multiple of batch" in lib.fp8_last_error().decode()
    assert size(pair(page_size=3)) == -1
    assert lib.fp8_kv_attention_workspace(None, 2, 32, 0, 0, 0, 0) == -1


@pytest.mark.parametrize("change, status, word", [
    (dict(weights=None), I, "weights is NULL"), (dict(ldw=255), I, "ldw"), (dict(budget=0), I, "budget"),
    (dict(sinks=-1), I, "sinks"), (dict(recent=-1), I, "recent"), (dict(sinks=60, recent=5), I, "together"),
    (dict(sinks=2147483647, recent=2147483647), I, "together"),
    (dict(wo=2 * FAKE, ldwo=63), I, "ldwo"), (dict(wo=FAKE, ldwo=200), I, "ldwo"),
    (dict(dst=2 * FAKE, dst_ld=3), I, "dst_page_ld"), (dict(dst=FAKE, dst_ld=4), I, "dst_page_table"),
    (dict(kept=None), I, "kept"), (dict(lens=None), I, "new_lens"), (dict(lens=FAKE), I, "new_lens"),
    (dict(weights=FAKE + 1), M, "weights"), (dict(kept=FAKE + 2), M, "kept"), (dict(wo=2 * FAKE + 2, ldwo=64), M, "4-byte"),
])
def test_evict(change, status, word):
    check(evict(**change), status, word)


def test_null_descriptor():
    assert L.lib().fp8_kv_evict(None, FAKE, 256, 64, 4, 16, None, 0, None, 0, FAKE, FAKE, None) == I
    assert "cache" in L.lib().fp8_last_error().decode()


def test_descriptor_size_matches_the_header():
    assert ctypes.sizeof(L.Fp8KvPair) == 104


def test_attention_limits_of_sizes():
    check(attention(pair(batch=65535, heads=32768, max_len=16), total_q=0, q_heads=32768, ldq=1 << 23, ldo=1 << 23), U,
          "batch * heads")
    check(attention(pair(batch=64, max_len=1 << 29, page_ld=1 << 25), total_q=64), U, "batch * max_len")
    check(attention(pair(batch=2, max_len=1 << 29, page_ld=1 << 25, heads=1024), total_q=2, q_heads=1024, ldq=1 << 18,
                    ldo=1 << 18), U, "max_len / 128")
