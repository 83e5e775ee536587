"""fp8_kv_append's pitch of the positions' axes, checked without a GPU: 0 is
one row for all of them.  Pointers are fake and never dereferenced."""
from __future__ import annotations

import pytest

from tests.test_append_boundary import append
from tests.test_attention_boundary import I, check


@pytest.mark.parametrize("pos_ld, word", [(0, "sections hold 63"), (5, "sections hold 63"), (1, "pos_ld"), (4, "pos_ld"),
                                          (-1, "pos_ld"), (-5, "pos_ld")])
def test_pitch_of_the_axes(pos_ld, word):
    """(The sections are looked at behind the pitch.)"""
    check(append(axes=2, sections=[32, 31], pos_ld=pos_ld), I, word)
