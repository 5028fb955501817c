"""tree_attention on the GPU where its softmax is at its ends: scores of any size, tokens of next to no weight beside one of nearly
all of it, and requests that many workgroups share, every piece of which has to count once. References in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from attention_helpers import LONG, attention_bound, long_case
from helpers import assert_within
from test_step_gpu import attention_case, dev, host, pbg, say  # noqa: F401 (pbg is a fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# heads, kv heads, head_dim, rows of a request: both tile sizes of the kernel for few query rows, the wide one, that for wide heads
KERNELS = [(4, 1, 128, 1), (8, 2, 64, 1), (2, 1, 256, 3), (6, 1, 128, 4), (8, 8, 128, 40), (4, 2, 64, 130), (2, 1, 256, 40), (3, 1, 200, 70)]


def run(pbg, c, scale=None):  # noqa: F811
    return host(pbg.tree_attention(**{k: dev(v) for k, v in c.items()}, scale=scale))


def set_token(c, i, t, key=None, value=None):
    """Key and value of token t of request i, for every head."""
    page = c["k_cache"].shape[2]
    for name, x in (("k_cache", key), ("v_cache", value)):
        if x is not None:
            c[name][c["table"][i, t // page], :, t % page] = x


@pytest.mark.parametrize("heads,kv,d,rows", KERNELS)
@pytest.mark.parametrize("scale", [1.0, 9.0, 130.0, 3e4, 1.7e9, 2.3e17, 1e30])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(pbg, heads, kv, d, rows, scale, sign):  # noqa: F811
    """Scores that are far apart leave one token's value, scores that are equal the mean of two, however large they are.

    Queries and keys are small integers, so that products are exact, and scores differ by at least 100 in powers of two or not at all:
    one or two equal weights, each off by its own rounding to fp16 (2^-11) above and not below, and the output's rounding. What a score
    is off by is off in the largest as well.
    """
    say(f"attention scores {heads}/{kv} x {d} rows={rows} scale={scale} sign={sign}")
    lengths = [700, 65, 3]
    c = attention_case(d + rows, lengths, [rows] * 3, heads, kv, d, 16)
    rng = np.random.default_rng(1)
    c["q"][:], c["k_cache"][:] = 0, 0
    c["q"][..., 0] = 100
    c["v_cache"][:] = rng.integers(-32, 33, c["v_cache"].shape)
    most = max(lengths) + rows
    for i in range(3):
        # the tokens before the step in any order, the step's own below all of them, those of the step among them by their row
        order = rng.permutation(lengths[i])
        for t in range(lengths[i] + rows):
            key = order[t] + rows if t < lengths[i] else t - lengths[i]
            set_token(c, i, t, key + 1 if sign > 0 else key - most)
        # a tie of the two largest
        a, b = int(np.flatnonzero(order == lengths[i] - 1)[0]), int(np.flatnonzero(order == lengths[i] - 2)[0])
        if i < 2:
            set_token(c, i, b, lengths[i] - 1 + rows + 1 if sign > 0 else lengths[i] - 1 + rows - most)
            assert np.array_equal(c["k_cache"][c["table"][i, a // 16], :, a % 16], c["k_cache"][c["table"][i, b // 16], :, b % 16])
    ref, size, _ = oracle.tree_attention(**c, scale=scale)
    bound = 2.0 ** -11 * (size + np.abs(ref)) * 1.01 + 2.0 ** -25
    assert_within(run(pbg, c, scale), ref, bound)


# heads, kv heads, head_dim, requests, tokens, rows: several units of a request in a workgroup, so that many tokens share a maximum
LIGHT = [(8, 8, 64, 16, 3000, 1), (8, 8, 128, 16, 3000, 1), (8, 4, 128, 16, 3000, 12), (8, 8, 256, 8, 3000, 2), (8, 8, 64, 4, 3000, 70),
         (8, 8, 128, 4, 3000, 40), (4, 4, 256, 8, 3000, 33)]


@pytest.mark.parametrize("heads,kv,d,requests,tokens,rows", LIGHT)
@pytest.mark.parametrize("light,where", [(12.3, "last"), (21.45, "first"), (25.2, "first")])
def test_light_tokens_beside_a_heavy_one(pbg, heads, kv, d, requests, tokens, rows, light, where):  # noqa: F811
    """One token has nearly all the weight and no value, all others 2^-light of it each: they alone are the output."""
    say(f"attention light {heads}/{kv} x {d} requests={requests} rows={rows} light={light} heavy={where}")
    c = attention_case(d + rows, [tokens] * requests, [rows] * requests, heads, kv, d, 16)
    rng = np.random.default_rng(2)
    c["q"][:], c["k_cache"][:] = 0, 0
    c["q"][..., 0] = 1
    c["k_cache"][..., 0] = -light * np.log(2.0)
    c["v_cache"][:] = rng.uniform(0.5, 1.5, c["v_cache"].shape)
    for i in range(requests):
        set_token(c, i, 0 if where == "first" else tokens - 1, 0, 0)
    total = np.zeros(c["q"].shape[:2])
    ref, size, far = oracle.tree_attention(**c, scale=1.0, totals=total)
    bound = attention_bound(c["q"], c["lengths"], c["row_start"], ref, size, far, total, 1.5, 1.0)
    # what is tested is well above what is allowed
    assert (bound < 0.02 * ref).all()
    assert_within(run(pbg, c, 1.0), ref, bound)


@pytest.mark.parametrize("heads,kv,d,rows,lengths", LONG)
def test_every_block_of_a_long_request_counts_once(pbg, heads, kv, d, rows, lengths):  # noqa: F811
    """Requests that every workgroup has a piece of. (A block of tokens left out or taken twice is 4 bounds off: test_attention_edges.)"""
    say(f"attention long {heads}/{kv} x {d} rows={rows} {lengths}")
    c = long_case(heads, kv, d, rows, lengths)
    total = np.zeros(c["q"].shape[:2])
    ref, size, far = oracle.tree_attention(**c, totals=total)
    assert_within(run(pbg, c), ref, attention_bound(c["q"], c["lengths"], c["row_start"], ref, size, far, total, 1.0, d ** -0.5))


@pytest.mark.parametrize("heads,kv,d,rows", [(4, 1, 128, 4), (2, 1, 256, 6), (8, 1, 64, 4), (32, 32, 128, 12), (32, 32, 64, 60),
                                              (32, 32, 128, 60), (32, 32, 256, 60)])
@pytest.mark.parametrize("tree", [True, False])
def test_scores_that_a_row_does_not_see_do_not_change_it(pbg, heads, kv, d, rows, tree):  # noqa: F811
    """A row's token with scores far above all others, finite: rows that do not see it keep their bits. (The first lengths: several units in a
    workgroup, whose maxima are raised between them.)"""
    say(f"attention unseen scores {heads}/{kv} x {d} rows={rows} tree={tree}")
    for lengths in ([700, 650], [0, 9], [61, 63]):
        c = attention_case(d + rows + lengths[0], lengths, [rows, rows], heads, kv, d, 16, tree=tree, spread=1.0)
        # tokens before the step score lower than its own
        for t in range(lengths[0]):
            page, off = c["table"][0, t // 16], t % 16
            c["k_cache"][page, :, off] *= np.float16(0.1)
        for times, scale, row in [(x, None, y) for x in (3, 30, 300) for y in (0, rows // 2, rows - 1)] + [(60000, 1.0, rows // 2)]:
            base = run(pbg, c, scale)
            bad = {k: None if v is None else v.copy() for k, v in c.items()}
            q = bad["q"][row, 0].astype(np.float32)
            set_token(bad, 0, lengths[0] + row, np.clip(q * times, -60000, 60000))
            got = run(pbg, bad, scale)
            sees = np.array([(int(c["ancestors"][a]) >> row & 1) if tree else a >= row for a in range(rows)] + [False] * rows, bool)
            assert sees.any() and np.isfinite(got).all()
            assert np.array_equal(got[~sees].view(np.uint16), base[~sees].view(np.uint16)), (lengths, times, row)
