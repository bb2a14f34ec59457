"""Row counts at the ends of the token operators' ranges: what the library says on the host."""

from __future__ import annotations

import pytest

from test_tokens_abi import HEADS, INVALID, PTR, attention, lib  # noqa: F401

MOST = (1 << 31) - 4096
TOO_LARGE = -8


@pytest.mark.parametrize("off,status", [((0, MOST), INVALID), ((0, MOST + 1), TOO_LARGE), ((0, 5, (1 << 31) - 1), TOO_LARGE),
                                        ((0, 1 << 31), INVALID)])
def test_attention_rows(lib, off, status):  # noqa: F811
    # (Within the range what is wrong with the call is its host pointers.)
    few = tuple(min(x, 4) for x in off)
    for q, k in ((off, few), (few, off)):
        p, alive = attention(q, k)
        assert lib.pv_attention(p, HEADS, HEADS, HEADS, HEADS, None, None) == status
        assert lib.pv_attention_backward(p, HEADS, HEADS, HEADS, HEADS, HEADS, PTR, HEADS, HEADS, HEADS, None) == status
        del alive
