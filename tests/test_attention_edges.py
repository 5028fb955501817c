"""What the tests of tree_attention on the GPU would notice, on the CPU: mistakes planted in the reference."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from attention_helpers import BLOCK, LONG, attention_bound, long_case


@pytest.mark.parametrize("heads,kv,d,rows,lengths", LONG)
def test_a_block_left_out_or_taken_twice_is_noticed(heads, kv, d, rows, lengths):
    """In the last row of the longest request, for every head and each of its blocks."""
    c = long_case(heads, kv, d, rows, lengths)
    i = int(np.argmax(lengths))
    one = dict(q=c["q"][int(c["row_start"][i + 1]) - 1:][:1], k_cache=c["k_cache"], v_cache=c["v_cache"], table=c["table"][i: i + 1],
               lengths=c["lengths"][i: i + 1] + rows - 1, row_start=np.array([0, 1]))
    total = np.zeros((1, heads))
    ref, size, far = oracle.tree_attention(**one, totals=total)
    bound = attention_bound(one["q"], c["lengths"], c["row_start"], ref, size, far, total, 1.0, d ** -0.5)
    n = lengths[i] + rows
    assert n // BLOCK >= 200
    for e in range(heads):
        k, _ = oracle.cached_tokens(c["k_cache"], c["table"][i], n, e // (heads // kv))
        w = np.exp(k.astype(np.float64) @ one["q"][0, e].astype(np.float64) * d ** -0.5)
        w /= w.sum()
        block = np.add.reduceat(w, np.arange(0, n, BLOCK))
        column = np.arange(len(block)) % d
        assert np.allclose(np.bincount(column, block, minlength=d), ref[0, e])
        for sign in (-1, 1):
            wrong = (ref[0, e, column] + sign * block) / (1 + sign * block)
            full = np.arange(len(block)) < n // BLOCK
            assert (np.abs(wrong - ref[0, e, column]) > 4 * bound[0, e, column])[full].all()
