"""A serving loop on the GPU over many steps: trees whose pages are opened and given back, accepted rows moved together, requests that end.
Every page keeps one place, and the cache holds each request's tokens."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from page_helpers import give_back, pages_in_use, steps
from test_step_gpu import dev, host, pbg, say  # noqa: F401 (pbg is a fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("page", [1, 8, 16])
def test_a_loop_of_steps(pbg, page):  # noqa: F811
    requests, heads, kv, d, count = 6, 2, 1, 8, 40
    width = (5 * page + 60 + max(34, 3 * page)) // page + 1
    pages = requests * width
    table = torch.full((requests, width), -1, dtype=torch.int32, device="cuda:0")
    free = dev(np.random.default_rng(3).permutation(pages).astype(np.int32))
    left, lengths = dev(np.array([pages], np.int32)), torch.zeros(requests, dtype=torch.int32, device="cuda:0")
    k, v = (torch.zeros((pages, kv, page, d), dtype=torch.float16, device="cuda:0") for _ in range(2))
    said = [[] for _ in range(requests)]  # what each request's tokens are, told by their keys and values
    rng = np.random.default_rng(4)
    for n, (added, parents, keep) in enumerate(steps(page, requests, page, count)):
        say(f"pages page={page} step {n}")
        keep[host(lengths) > 5 * page + 60] = -1
        m = max(int(added.sum()), 1)
        if parents is not None and not len(parents):
            parents = np.zeros(1, np.int32)
        before = host(lengths)
        plan = oracle.cache_plan(before, added, host(table), host(free), int(left), page, pages, m, parents)
        start, request, position, slot, anc, left = pbg.cache_plan(lengths, dev(added), table, free, left, page, pages, rows=m,
                                                                   parents=None if parents is None else dev(parents))
        for got, want in zip((start, request, position, slot, table), (*plan[:4], plan[6])):
            assert np.array_equal(host(got), want)
        assert int(left) == plan[5] and (host(slot)[: int(added.sum())] >= 0).all()
        name = rng.integers(-1000, 1000, m)
        qkv = np.repeat(name[:, None], (heads + 2 * kv) * d, 1).astype(np.float32)
        qkv[:, (heads + kv) * d:] += 1
        pbg.rotary_qkv(dev(qkv), position, slot, None, k, v)
        # the accepted rows: all of a prompt, a path of a tree as long as `keep` says where there is one
        kept = np.zeros(requests, np.int32)
        for i in range(requests):
            first = int(plan[0][i])
            rows = list(range(int(added[i])))
            if parents is not None and len(rows):
                rows = max((oracle.tree_path(parents[first: first + c + 1], c)[::-1] for c in rows), key=len)[: max(int(keep[i]), 0)]
            if keep[i] < 0:
                said[i] = []
                continue
            src = slot[[first + r for r in rows]]
            dst = slot[first: first + len(rows)]
            for cache in (k, v):
                cache[dst // page, :, dst % page] = cache[src // page, :, src % page]
            said[i] += [int(name[first + r]) for r in rows]
            kept[i] = before[i] + len(rows)
            assert kept[i] == len(said[i])
        left, lengths = give_back(table=table, lengths=lengths, start=start, kept=dev(kept), page_size=page, free=free, left=left)
        assert sorted(pages_in_use(host(table), kept, page) + host(free)[: int(left)].tolist()) == list(range(pages))
        for i in range(requests):
            for cache, more in ((host(k), 0), (host(v), 1)):
                tokens, held = oracle.cached_tokens(cache, host(table)[i], len(said[i]), 0)
                assert held.all() and np.array_equal(tokens[:, 0], np.array(said[i]) + more)
