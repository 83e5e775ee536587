"""Boundary checks of fp8_kv_append and its binding that run without a GPU:
every invalid argument is rejected before any device call, with a message that
names it.  Pointers are fake and never dereferenced."""
from __future__ import annotations

import ctypes

import pytest
import torch

from fp8_precision_quantization_amd import _lib as L
from tests.test_attention_boundary import FAKE, I, M, U, check, pair

fp8 = pytest.importorskip("fp8_precision_quantization_amd")


def append(p=None, **change):
    a = dict(k=FAKE, ldk=1024, v=FAKE, ldv=1024, q=FAKE, ldq=4096, q_heads=32, q_out=2 * FAKE, ldqo=4096,
             dt=L.FP8_IN_BF16, n=5, slots=FAKE, positions=FAKE, pos_ld=5, sections=None, axes=1, inv_freq=FAKE,
             rotary=128, flags=0, diag=None)
    a.update(change)
    if a["sections"] is not None:
        a["sections"] = (ctypes.c_int32 * len(a["sections"]))(*a["sections"])
    p = p or pair(v=2 * FAKE)
    return L.lib().fp8_kv_append(ctypes.byref(p), a["k"], a["ldk"], a["v"], a["ldv"], a["q"], a["ldq"], a["q_heads"],
                                 a["q_out"], a["ldqo"], a["dt"], a["n"], a["slots"], a["positions"], a["pos_ld"],
                                 a["sections"], a["axes"], a["inv_freq"], a["rotary"], a["flags"], a["diag"], None)


@pytest.mark.parametrize("change, status, word", [
    (dict(k=None), I, "cache is NULL"), (dict(k=FAKE + 8), M, "16-byte"), (dict(k_scale_inv=None), I, "scale_inv"),
    (dict(k_storage=3), I, "storage"), (dict(scaling=2), I, "scaling"), (dict(head_dim=24), U, "head_dim"),
    (dict(head_dim=272), U, "head_dim"), (dict(heads=0), I, "heads"), (dict(capacity=-1), I, "capacity"),
    (dict(capacity=1 << 31), U, "capacity"), (dict(v=FAKE), I, "one array"),
])
def test_caches(change, status, word):
    check(append(pair(**{**dict(v=2 * FAKE), **change})), status, word)


def test_pages_are_not_read():
    """What only sequences need may hold anything: the call gets as far as its own arguments."""
    p = pair(v=2 * FAKE, page_table=None, page_ld=-1, lens=None, max_len=-7, page_size=3, batch=-2, reserved=9)
    check(append(p, rotary=24), U, "rotary_dim")


@pytest.mark.parametrize("change, status, word", [
    (dict(k=None), I, "k or v is NULL"), (dict(v=None), I, "k or v is NULL"), (dict(k=FAKE + 8), M, "16-byte"),
    (dict(v=FAKE + 2), M, "16-byte"), (dict(q=FAKE + 8), M, "16-byte"), (dict(q_out=FAKE + 8), M, "16-byte"),
    (dict(ldk=1016), I, "ldk"), (dict(ldv=1000), I, "ldv"), (dict(ldq=4095), I, "ldq"), (dict(ldqo=8), I, "ldqo"),
    (dict(ldk=1028), M, "ldk"), (dict(ldqo=4100), M, "ldqo"), (dict(dt=2), I, "in_dtype"), (dict(n=-1), I, "n_tokens"),
    (dict(n=1 << 22), U, "n_tokens"), (dict(q_heads=-1), I, "q_heads"), (dict(q_heads=65536, ldq=1 << 23, ldqo=1 << 23), U, "q_heads"),
    (dict(q=None), I, "q_out is NULL"), (dict(q_out=None), I, "q_out is NULL"), (dict(q_heads=0), I, "q_heads=0"),
    (dict(q_out=FAKE, ldqo=4104), I, "q_out is q"), (dict(q_out=FAKE, dt=L.FP8_IN_F32), I, "q_out is q"),
    (dict(slots=FAKE + 4), M, "slots"), (dict(positions=FAKE + 4), M, "positions"), (dict(inv_freq=FAKE + 2), M, "inv_freq"),
    (dict(diag=FAKE + 2), M, "diag"), (dict(flags=2), I, "flag"), (dict(flags=16), I, "flag"),
    (dict(rotary=144), U, "rotary_dim"), (dict(rotary=8), U, "rotary_dim"), (dict(rotary=-16), U, "rotary_dim"),
    (dict(axes=0), U, "axes"), (dict(axes=5, sections=[32, 8, 8, 8, 8]), U, "axes"), (dict(inv_freq=None), I, "inv_freq"),
    (dict(positions=None), I, "positions"), (dict(axes=2), I, "sections is NULL"),
    (dict(axes=2, sections=[32, 31]), I, "sections hold 63"), (dict(axes=2, sections=[65, -1]), I, "sections[1]"),
    (dict(axes=3, sections=[1 << 30, 1 << 30, 1 << 30]), I, "sections hold"), (dict(axes=1, sections=[32]), I, "sections hold"),
    (dict(axes=2, sections=[32, 32], pos_ld=4), I, "pos_ld"),
])
def test_arguments(change, status, word):
    check(append(**change), status, word)


def test_null_descriptor():
    assert L.lib().fp8_kv_append(None, FAKE, 8, FAKE, 8, None, 0, 0, None, 0, 1, 1, None, None, 0, None, 1, None, 0, 0,
                                 None, None) == I
    assert "cache" in L.lib().fp8_last_error().decode()


def _host(**change):
    t = torch.zeros
    a = dict(k=t(3, 2, 64), v=t(3, 2, 64), k_cache=t(8, 2, 64, dtype=torch.uint8), v_cache=t(8, 2, 64, dtype=torch.uint8))
    a.update(change)
    return a


def test_binding_wants_device_tensors():
    with pytest.raises(ValueError, match="device tensor"):
        fp8.kv_append(**_host())
    with pytest.raises(ValueError, match="device tensor"):
        fp8.kv_append(**_host(k_cache=torch.zeros(8, 128, dtype=torch.uint8)))
