"""Pages of a serving loop on the CPU, with the oracle's cache_plan and README's way of giving pages back: every page stays in one
request's table or on the stack."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from page_helpers import give_back, pages_in_use, steps

torch = pytest.importorskip("torch")


def loop(page, back, requests=8, count=60):
    # as many as the longest request of steps() and of what is below can hold
    width = (5 * page + 60 + max(34, 3 * page)) // page + 1
    pages = requests * width
    table = torch.full((requests, width), -1, dtype=torch.int32)
    free = torch.from_numpy(np.random.default_rng(3).permutation(pages).astype(np.int32))
    left, lengths = torch.tensor([pages], dtype=torch.int32), torch.zeros(requests, dtype=torch.int32)
    missing = 0
    for added, parents, keep in steps(page, requests, page, count):
        keep[lengths.numpy() > 5 * page + 60] = -1
        m = max(int(added.sum()), 1)
        if parents is not None and not len(parents):
            parents = np.zeros(1, np.int32)
        start, request, position, slot, anc, after, new = oracle.cache_plan(lengths.numpy(), added, table.numpy(), free.numpy(), int(left), page,
                                                                            pages, m, parents)
        missing += int((slot[: int(added.sum())] < 0).sum())
        table.copy_(torch.from_numpy(new))
        start, left = torch.from_numpy(start), torch.tensor([after], dtype=torch.int32)
        kept = torch.from_numpy(np.where(keep < 0, 0, lengths.numpy() + keep).astype(np.int32))
        if back:
            left, lengths = give_back(table=table, lengths=lengths, start=start, kept=kept, page_size=page, free=free, left=left)
            every = sorted(pages_in_use(table, lengths, page) + free[: int(left)].tolist())
            assert every == list(range(pages)), "every page has one place"
        else:
            lengths = kept
    return missing, int(left)


@pytest.mark.parametrize("page", [1, 4, 8, 16, 64])
def test_no_page_is_lost(page):
    missing, _ = loop(page, True)
    assert missing == 0


def test_without_giving_back_the_stack_runs_dry():
    missing, left = loop(16, False)
    assert missing > 0 and left == 0


def test_pages_that_were_missing_are_not_given_back():
    """A stack that runs out leaves -1 in the table, which is no page."""
    page, pages = 4, 5
    table, free = torch.full((2, 6), -1, dtype=torch.int32), torch.arange(pages, dtype=torch.int32)
    start, _, _, slot, _, left, new = oracle.cache_plan(np.zeros(2), np.array([18, 9]), table.numpy(), free.numpy(), pages, page, pages, 27)
    assert (slot >= 0).sum() == 18 and left == 0
    left, lengths = give_back(table=torch.from_numpy(new), lengths=torch.zeros(2, dtype=torch.int32), start=torch.from_numpy(start),
                              kept=torch.tensor([6, 0], dtype=torch.int32), page_size=page, free=free, left=torch.tensor([left]))
    assert int(left) == 3 and sorted(free[:3].tolist() + pages_in_use(new, [6, 0], page)) == list(range(pages))
