"""Pins of oracle/rows.py: the grouping by its defining properties and a case
by hand, the sum and norm by closed forms, the quantisers by those they are."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import boundary, moe, rows
from oracle.codecs import e4m3_decode, f32


def test_grouping_by_hand():
    ids = np.array([[2, 0], [1, 2], [2, 1]])
    offsets, tokens, pos = rows.group_routes(ids, 0, 4)
    assert offsets.tolist() == [0, 1, 3, 6, 6]
    assert tokens.tolist() == [0, 1, 2, 0, 1, 2]
    assert pos.tolist() == [[3, 0], [1, 4], [5, 2]]
    offsets, tokens, pos = rows.group_routes(ids, 1, 1)
    assert offsets.tolist() == [0, 2] and tokens.tolist() == [1, 2]
    assert pos.tolist() == [[-1, -1], [0, -1], [-1, 1]]


@pytest.mark.parametrize("lb,lc", [(0, 12), (3, 5)])
def test_grouping_properties(lb, lc):
    rng = np.random.default_rng(1)
    ids = np.stack([rng.permutation(12)[:4] for _ in range(50)])
    offsets, tokens, pos = rows.group_routes(ids, lb, lc)
    local = (ids >= lb) & (ids < lb + lc)
    assert (pos >= 0).tolist() == local.tolist()
    assert sorted(pos[local]) == list(range(local.sum())) and offsets[-1] == local.sum()
    for e in range(lc):
        mine = tokens[offsets[e]:offsets[e + 1]]
        assert mine.tolist() == sorted(np.nonzero((ids == lb + e).any(axis=1))[0])
    t, j = np.nonzero(local)
    assert (tokens[pos[t, j]] == t).all()


def test_sum_rounds_once():
    """1 + 2^-24 + 2^-24 is 1 when each sum is rounded, 1 + 2^-23 when once."""
    one, tiny = np.ones((1, 8)), np.full((1, 8), 2.0**-24)
    y = np.stack([tiny[0], 100 * tiny[0]])
    h = rows.sum_rows(one, tiny, y, np.array([[0, -1, 2]]), np.array([[1.0, 5.0, 7.0]]))
    assert (h == 1 + 2.0**-23).all()


def test_norm_closed_form():
    v = rows.norm_rows(np.full((2, 16), -3.0), np.full(16, 0.5), 0.0)
    assert np.abs(v + 0.5).max() <= 2.0**-24
    assert not rows.norm_rows(np.zeros((1, 16)), np.ones(16), 1e-5).any()


def test_quantisers():
    v = f32(np.random.default_rng(2).standard_normal((3, 256)))
    for quant, want in (("fp8", moe.quantize_blocks(v, False, True)), ("fp8_p2", moe.quantize_blocks(v, True, True)),
                        ("mxfp8", boundary.mxfp8_quantize(v))):
        q, s = rows.quantize_rows(v, quant)
        assert np.array_equal(q, want[0]) and np.array_equal(s, want[1])
    q, s = rows.quantize_rows(v, "fp8")
    back = e4m3_decode(q).reshape(3, 2, 128) * s[..., None]
    assert np.abs(back - v.reshape(3, 2, 128)).max() <= np.abs(v).max() * 2.0**-4
