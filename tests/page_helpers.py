"""A serving loop's pages: steps of trees, tokens and prompts of which a part is kept, with README's way of giving pages back."""
from __future__ import annotations

import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def readme_block(first_line: str):
    """Code of the README's python block that begins with this line."""
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), flags=re.S)
    found = [b for b in blocks if b.startswith(first_line)]
    assert len(found) == 1, first_line
    return compile(found[0], "README.md", "exec")


def give_back(**names):
    """What README does after a step: (free_count, lengths) for the next one; free is changed in place."""
    import torch

    exec(readme_block("# give back:"), {"torch": torch}, names)
    return names["count"], names["lengths"]


def pages_in_use(table, lengths, page_size):
    return [int(table[i, p]) for i in range(len(lengths)) for p in range(-(-int(lengths[i]) // page_size))]


def steps(seed, requests, page_size, count):
    """(added, parents or None, kept rows of each request as a function of its rows) of each step: prompts, trees, single tokens; the kept
    count -1 ends the request."""
    rng = np.random.default_rng(seed)
    for n in range(count):
        kind = ("prompt", "tree", "tree", "token")[n % 4] if n else "prompt"
        if kind == "prompt":
            added = rng.integers(0, 3 * page_size, requests)
        elif kind == "tree":
            added = rng.integers(0, 34, requests)
        else:
            added = np.ones(requests, int)
        keep = added.copy() if kind != "tree" else np.minimum(added, rng.integers(0, 5, requests))
        keep[rng.random(requests) < 0.1] = -1
        parents = None
        if kind == "tree":
            row = np.concatenate([np.arange(a) for a in added]) if added.sum() else np.zeros(0, int)
            parents = (row - rng.integers(1, 4, len(row))).astype(np.int32)
        yield added.astype(np.int32), parents, keep
