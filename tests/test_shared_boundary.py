"""Boundary checks of fp8_kv_attention_shared that run without a GPU: every
invalid argument is rejected before any device call, with a message that names
it, and its workspace follows the sizes.  Pointers are fake and never
dereferenced."""
from __future__ import annotations

import ctypes

import pytest
import torch

from fp8_precision_quantization_amd import _lib as L
from tests.test_attention_boundary import FAKE, I, M, PAIRS, U, check, pair
from tests.test_attention_binding import WIDE, _args

fp8 = pytest.importorskip("fp8_precision_quantization_amd")


def shared(p=None, **change):
    a = dict(q=FAKE, ldq=4096, total_q=2, q_heads=32, q_offsets=None, scale=0.1, window=0, sinks=0, shared=128, out=FAKE,
             ldo=4096, lse=FAKE, weights=None, ldw=0, ws=FAKE, wsb=1 << 30)
    a.update(change)
    p = p or pair()
    return L.lib().fp8_kv_attention_shared(
        ctypes.byref(p), a["q"], a["ldq"], a["total_q"], a["q_heads"], a["q_offsets"], a["scale"], a["window"], a["sinks"],
        a["shared"], a["out"], a["ldo"], a["lse"], a["weights"], a["ldw"], a["ws"], a["wsb"], None)


def size(p, total=2, q_heads=32, ragged=0, window=0, sinks=0, weighted=0, shared=128):
    return L.lib().fp8_kv_attention_shared_workspace(ctypes.byref(p), total, q_heads, ragged, window, sinks, weighted, shared)


@pytest.mark.parametrize("change, status, word", PAIRS, ids=lambda x: str(x) if isinstance(x, dict) else "")
def test_pair(change, status, word):
    check(shared(pair(**change)), status, word)


@pytest.mark.parametrize("change, status, word", [
    (dict(shared=-1), I, "shared=-1"), (dict(shared=257), I, "shared=257"), (dict(shared=1 << 40), I, "shared"),
    (dict(q=None), I, "q is NULL"), (dict(out=FAKE + 8), M, "16-byte"), (dict(ldq=4088), I, "ldq"),
    (dict(total_q=3), I, "multiple of batch"), (dict(window=-1), I, "window"), (dict(scale=float("nan")), I, "scale"),
    (dict(weights=FAKE, ldw=256, lse=None), I, "lse"), (dict(weights=FAKE, ldw=255), I, "ldw"),
    (dict(ws=None), I, "workspace is NULL"), (dict(ws=FAKE + 8), M, "workspace"), (dict(wsb=64), I, "workspace_bytes"),
    (dict(total_q=1 << 28), U, "total_q"),
])
def test_arguments(change, status, word):
    check(shared(**change), status, word)


def test_workspace():
    p = pair(max_len=65536, page_ld=4096)
    plain = L.lib().fp8_kv_attention_workspace(ctypes.byref(p), 2, 32, 0, 0, 0, 0)
    assert size(p, shared=0) == size(p, shared=63) == plain             # no whole step: the ordinary call
    assert size(p, shared=4096, window=16) == L.lib().fp8_kv_attention_workspace(ctypes.byref(p), 2, 32, 0, 16, 0, 0)
    one = pair(batch=1, max_len=65536, page_ld=4096)
    assert size(one, total=1, shared=4096) == L.lib().fp8_kv_attention_workspace(ctypes.byref(one), 1, 32, 0, 0, 0, 0)
    for total, ragged in ((2, 0), (6, 0), (7, 1), (400, 1)):
        need = size(p, total=total, ragged=ragged, shared=60000)
        assert need > 0 and need % 16 == 0
        check(shared(p, total_q=total, q_offsets=FAKE if ragged else None, shared=60000, wsb=need - 1), I, "workspace_bytes")
    assert size(p, total=0) == 0
    assert size(p, shared=65537) == -1 and "shared" in L.lib().fp8_last_error().decode()
    # sizes alone: no pointer is needed
    assert size(pair(k=None, v=None, k_scale_inv=None, v_scale_inv=None, lens=None, page_table=None)) == size(pair())


@pytest.mark.parametrize("p, q, status", [
    (dict(batch=65535, heads=512), dict(total_q=65535, q_heads=512), 0),
    (dict(batch=65535, heads=256), dict(total_q=65535, q_heads=256, ragged=1), U),
    (dict(batch=32768, heads=512), dict(total_q=65536, q_heads=512), U),
    (dict(batch=2, heads=8, max_len=1 << 28), dict(total_q=2, q_heads=8, weighted=1), U),
    (dict(batch=2, heads=8, max_len=1 << 28), dict(total_q=2, q_heads=8), 0),
])
def test_launches_stay_below_2_32_threads(p, q, status):
    c = pair(**{**dict(head_dim=16, page_size=1 << 20, page_ld=512), **p})
    got = size(c, q["total_q"], q["q_heads"], q.get("ragged", 0), weighted=q.get("weighted", 0), shared=64)
    if status == 0:
        assert got >= 0, L.lib().fp8_last_error()
    else:
        assert got == -1 and "2^24" in L.lib().fp8_last_error().decode()


@pytest.mark.parametrize("value", WIDE)
def test_numbers_past_32_bits(value):
    with pytest.raises(ValueError, match="shared=%d does not fit" % value):
        fp8.kv_attention(torch.zeros((1, 2, 64), dtype=torch.bfloat16), **{**_args(), "shared": value})
