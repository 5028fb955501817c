"""Trees, single tokens and prompts of one step on the GPU: what may stand in one call, and both kinds in two calls over one cache."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from attention_helpers import attention_bound
from helpers import assert_within
from test_step_gpu import dev, host, pbg, say  # noqa: F401 (pbg is a fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("heads,kv,d", [(8, 2, 64), (4, 1, 128), (2, 1, 256)])
def test_a_step_of_trees_tokens_and_prompts(pbg, heads, kv, d):  # noqa: F811
    """Requests 0 to 3 are a tree, a token, a prompt of 64 rows and an idle one, in a call with parents; requests 4 to 6 a prompt of 150
    rows, a token and a prompt of 65, in a call without, on the same stack. One rotary call for all rows."""
    say(f"mixed step {heads}/{kv} x {d}")
    rng = np.random.default_rng(d)
    page, pages, width = 16, 80, 24
    lengths = np.array([40, 33, 15, 7, 0, 64, 100], np.int32)
    added = np.array([30, 1, 64, 0, 150, 1, 65], np.int32)
    kinds = [slice(0, 4), slice(4, 7)]
    tree = np.arange(30) - rng.integers(1, 5, 30)
    parents = np.concatenate([tree, [-1], np.arange(64) - 1]).astype(np.int32)
    table = np.full((7, width), -1, np.int32)
    ids, at = rng.permutation(pages).astype(np.int32), 0
    for i, n in enumerate(-(-lengths // page)):
        table[i, :n] = ids[at: at + n]
        at += n
    free, left = dev(ids[at:]), dev(np.array([pages - at], np.int32))
    k, v = (dev(rng.standard_normal((pages, kv, page, d)).astype(np.float16)) for _ in range(2))
    table_d, plans, was = dev(table), [], pages - at
    for kind, par in zip(kinds, (parents, None)):
        m = int(added[kind].sum())
        plan = pbg.cache_plan(dev(lengths[kind]), dev(added[kind]), table_d[kind], free, left, page, pages, rows=m,
                              parents=None if par is None else dev(par))
        want = oracle.cache_plan(lengths[kind], added[kind], table[kind], host(free), was, page, pages, m, par)
        for got, w in zip((*plan[:4], table_d[kind]), (*want[:4], want[6])):
            assert np.array_equal(host(got), w)
        left, was = plan[5], want[5]
        assert int(left) == was and (host(plan[3]) >= 0).all() and (host(plan[2]) >= 0).all()
        plans.append(plan)
    rows = int(added.sum())
    qkv = rng.standard_normal((rows, (heads + 2 * kv) * d)).astype(np.float32)
    freq, _ = pbg.rotary_frequencies(d, device="cuda:0")
    q = pbg.rotary_qkv(dev(qkv), torch.cat([p[2] for p in plans]), torch.cat([p[3] for p in plans]), freq, k, v)
    outs = [pbg.tree_attention(q[a: b], k, v, table_d[kind], dev(lengths[kind]), p[0], p[4])
            for kind, p, (a, b) in zip(kinds, plans, ((0, 95), (95, rows)))]
    # each request on its own, seen by the oracle as what it is
    got, first = host(torch.cat(outs)), 0
    for i in range(7):
        end = first + int(added[i])
        if end == first:
            continue
        masks = None
        if i == 0:
            masks = np.array([sum(1 << p for p in oracle.tree_path(tree, c)) for c in range(30)], np.uint64)
        c = dict(q=host(q)[first: end], k_cache=host(k), v_cache=host(v), table=host(table_d)[i: i + 1], lengths=lengths[i: i + 1],
                 row_start=np.array([0, end - first], np.int32), ancestors=masks)
        total = np.zeros((end - first, heads))
        ref, size, far = oracle.tree_attention(**c, totals=total)
        high = float(np.abs(host(v)).max())
        assert_within(got[first: end], ref, attention_bound(c["q"], lengths, np.array([0, 150]), ref, size, far, total, high, d ** -0.5), f"request {i}")
        first = end
    assert first == rows
