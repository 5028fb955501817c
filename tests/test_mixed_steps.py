"""What one step can hold: masks reach over 64 rows of a request, so that longer prompts stand in a call without a tree."""
from __future__ import annotations

import numpy as np

import oracle


def test_rows_of_a_tree_step_from_the_64th_on_have_no_place():
    """A chain of 100 rows beside a tree of 3: 36 rows of it have no slot and no position, though their pages are opened. Planned without
    parents every row has both."""
    parents = np.concatenate([np.arange(100) - 1, [-1, 0, 0]]).astype(np.int32)
    table, free = np.full((2, 9), -1, np.int32), np.arange(20, dtype=np.int32)
    start, _, position, slot, anc, left, _ = oracle.cache_plan(np.zeros(2), np.array([100, 3]), table, free, 20, 16, 20, 103, parents)
    assert (slot[:64] >= 0).all() and (slot[64:100] == -1).all() and (position[64:100] == -1).all() and (anc[64:100] == 0).all()
    assert (slot[100:] >= 0).all() and position[100:].tolist() == [0, 1, 1] and left == 20 - 8
    _, _, position, slot, _, _, _ = oracle.cache_plan(np.zeros(1), np.array([100]), table[:1], free, 20, 16, 20, 100)
    assert (slot >= 0).all() and np.array_equal(position, np.arange(100))


def test_masks_reach_over_64_rows():
    """The same chain through its masks misses tokens that it sees without them."""
    rng = np.random.default_rng(1)
    k, v = (rng.standard_normal((7, 1, 16, 8)).astype(np.float16) for _ in range(2))
    q = rng.standard_normal((100, 1, 8)).astype(np.float16)
    c = dict(q=q, k_cache=k, v_cache=v, table=np.arange(7, dtype=np.int32)[None], lengths=np.zeros(1, np.int32), row_start=np.array([0, 100]))
    masks = np.array([(1 << min(a + 1, 64)) - 1 for a in range(100)], np.uint64)
    plain, with_masks = oracle.tree_attention(**c)[0], oracle.tree_attention(**c, ancestors=masks)[0]
    assert np.array_equal(plain[:64], with_masks[:64]) and (plain[64:] != with_masks[64:]).all()
