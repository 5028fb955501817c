"""GPU parity of the attention half of a step (cache_plan, rotary_qkv,
tree_attention) and of penalize_logits against the CPU oracle in 64 bits.

Tables, tokens and penalized logits must match bit for bit (every step that
leads to a logit is one IEEE fp32 operation). Tolerances, with u = 2^-24:
* rotary_qkv: the norm's factor is within (d / 2 + 8) u (an fp32 sum of d
  squares in any order, halved by the root); the weight's two products add
  2 u; cosine and sine come from an angle reduced in 64 bits and rounded once
  (pi 2^-24 = 4 u absolute at most), then 2 u of the functions and one product with the
  amplitude; a turn is two products and a sum, 3 u; then one fp16 rounding
  (2^-11 relative, 2^-25 below the normals).
* tree_attention: a score is an fp32 sum of d products: off by at most
  (d + 4) u scale sum_j |q_j k_j|, d_s, times log2(e) in the exponent and back;
  the exponential adds 4 u and its argument's rounding u |s - top|, below
  24 u where the weight is not 0 in fp16. A weight is then rounded to fp16 (2^-11
  relative; 2^-25 of the row's largest below the normals). With e the sum of
  these, a weighted mean moves by at most e (sum w |v| + |out|) / (1 - e); the
  sums of n terms add (n / 32 + 64) u each (a matrix instruction's chains are
  added in blocks of 32 tokens, and states of at most 64 pieces are joined), and
  the result is rounded to fp16.
"""
from __future__ import annotations

import sys

import numpy as np
import pytest

import oracle
from helpers import assert_within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
NAN = float("nan")


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def pbg(gpu):
    import packed_bit_gemv_amd as m

    m.lib()
    return m


def dev(a):
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int64) if a.dtype == np.uint64 else a.view(np.int32) if a.dtype == np.uint32 else a).to("cuda:0")


def host(t):
    return t.cpu().numpy()


# ---- cache_plan -------------------------------------------------------------


def plan_case(seed, r, page, most, longest, tree, spare=9, extra_width=2, pad=0):
    rng = np.random.default_rng(seed)
    lengths = rng.integers(0, longest + 1, r).astype(np.int32)
    lengths[rng.random(r) < 0.2] //= page
    lengths[rng.random(r) < 0.2] //= page * page
    lengths = np.where(rng.random(r) < 0.3, lengths // page * page, lengths).astype(np.int32)
    added = rng.integers(0, most + 1, r).astype(np.int32)
    width = int((-(-(lengths + added) // page)).max(initial=1)) + extra_width
    have = -(-lengths // page)
    need = int((-(-(lengths + added) // page) - have).sum())
    pages = int(have.sum()) + need + spare
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((r, width), -7, np.int32)
    at = 0
    for i in range(r):
        table[i, : have[i]] = ids[at: at + have[i]]
        at += have[i]
    m = max(int(added.sum()) + pad, 1)
    parents = rng.integers(-2, most + 2, m).astype(np.int32) if tree else None
    if tree:
        # mostly rows that follow one of the rows before them
        first = np.concatenate([np.arange(n) for n in added] + [np.zeros(m - int(added.sum()))]).astype(np.int64)
        back = rng.integers(1, 4, m)
        parents = np.where(rng.random(m) < 0.85, first - back, parents).astype(np.int32)
    return dict(lengths=lengths, added=added, table=table, free_pages=ids[at:], free_count=np.array([pages - at], np.int32),
                page_size=page, pages=pages, parents=parents, m=m)


def run_plan(pbg, c, chain=True):
    m, r = c["m"], len(c["lengths"])
    table = dev(c["table"])
    anc = torch.full((m,), 5, dtype=torch.int64, device="cuda:0") if chain or c["parents"] is not None else None
    out = pbg.cache_plan(dev(c["lengths"]), dev(c["added"]), table, dev(c["free_pages"]), dev(c["free_count"]), c["page_size"],
                         c["pages"], parents=dev(c["parents"]), ancestors=anc, rows=m)
    assert out[0].numel() == r + 1
    return out, table


def check_plan(pbg, c):
    got, table = run_plan(pbg, c)
    ref = oracle.cache_plan(c["lengths"], c["added"], c["table"], c["free_pages"], c["free_count"][0], c["page_size"], c["pages"],
                            c["m"], c["parents"])
    for name, g, w in zip(("row_start", "request", "position", "slot"), got, ref):
        assert np.array_equal(host(g), w), name
    assert np.array_equal(host(got[4]).view(np.uint64), ref[4]), "ancestors"
    assert int(got[5]) == ref[5]
    assert np.array_equal(host(table), ref[6]), "table"


PLANS = [(1, 16, 1, 100, False), (1, 1, 5, 3, False), (3, 2, 0, 9, False), (64, 16, 1, 8192, False), (64, 16, 8, 500, True),
         (5, 64, 700, 300, False), (7, 4, 64, 40, True), (257, 64, 100, 1000, False), (1000, 8, 20, 100, True), (4096, 16, 3, 60, False),
         (4096, 32, 2, 9000, True), (2, 4096, 5000, 9000, False), (33, 16, 63, 0, True), (1, 128, 20000, 0, False)]


@pytest.mark.parametrize("r,page,most,longest,tree", PLANS)
def test_cache_plan(pbg, r, page, most, longest, tree):
    say(f"plan r={r} page={page} most={most} longest={longest} tree={tree}")
    check_plan(pbg, plan_case(r + page, r, page, most, longest, tree))
    check_plan(pbg, plan_case(r + page + 1, r, page, most, longest, tree, pad=300))


@pytest.mark.parametrize("tree", [False, True])
def test_cache_plan_what_does_not_fit(pbg, tree):
    """Rows past the m-th, pages past the stack, the table's end and the cache, negative counts, trees of over 64 rows."""
    for seed in range(6):
        say(f"plan limits seed={seed} tree={tree}")
        c = plan_case(seed, 40, 8, 90, 200, tree)
        check_plan(pbg, {**c, "m": c["m"] // 2, "parents": None if c["parents"] is None else c["parents"][: c["m"] // 2]})
        check_plan(pbg, {**c, "free_count": np.array([seed * 17], np.int32)})
        check_plan(pbg, {**c, "free_count": np.array([-3], np.int32)})
        check_plan(pbg, {**c, "free_count": np.array([2 ** 31 - 1], np.int32)})
        check_plan(pbg, {**c, "table": np.ascontiguousarray(c["table"][:, : c["table"].shape[1] // 2])})
        check_plan(pbg, {**c, "pages": c["pages"] // 2})
        bad = c["lengths"].copy()
        bad[::5], bad[1::7] = -4, 2 ** 31 - 1
        more = c["added"].copy()
        more[::3] = -100
        check_plan(pbg, {**c, "lengths": bad, "added": more} if not tree else {**c, "added": more})
    c = plan_case(1, 4096, 16, 1, 10, False)
    check_plan(pbg, {**c, "added": np.full(4096, 2 ** 31 - 1, np.int32)})


def test_cache_plan_again_and_in_a_graph(pbg):
    """A second call writes the same tables; a captured one follows its inputs."""
    c = plan_case(3, 20, 16, 9, 300, True)
    ref, table = run_plan(pbg, c)
    args = [dev(c[x]) for x in ("lengths", "added", "table", "free_pages", "free_count")]
    m = c["m"]
    outs = dict(row_start=torch.empty_like(ref[0]), request=torch.empty_like(ref[1]), position=torch.empty_like(ref[2]),
                slot=torch.empty_like(ref[3]), free_left=torch.empty_like(ref[5]), parents=dev(c["parents"]),
                ancestors=torch.empty_like(ref[4]))
    call = lambda: pbg.cache_plan(*args, c["page_size"], c["pages"], **outs)  # noqa: E731
    call()
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        for o in outs.values():
            if o is not outs["parents"]:
                o.fill_(-9)
        args[0].copy_(dev(np.maximum(c["lengths"] - k, 0)))
        args[2].copy_(dev(c["table"]))
        graph.replay()
        torch.cuda.synchronize()
        want, t = run_plan(pbg, {**c, "lengths": np.maximum(c["lengths"] - k, 0)})
        got = [outs[x] for x in ("row_start", "request", "position", "slot", "ancestors", "free_left")]
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(args[2], t)


# ---- rotary_qkv -------------------------------------------------------------


def rotary_case(seed, m, heads, kv, d, rot, norm, page=16, positions=5000):
    rng = np.random.default_rng(seed)
    pages = -(-m // page) + 2
    slot = rng.permutation(pages * page)[:m].astype(np.int64)
    return dict(qkv=(rng.standard_normal((m, (heads + 2 * kv) * d)) * 2).astype(np.float32),
                position=rng.integers(0, positions, m).astype(np.int32), slot=slot,
                inv_freq=1e6 ** (-2.0 * np.arange(rot // 2) / rot) if rot else None,
                q_weight=rng.uniform(0.5, 1.5, d).astype(np.float32) if norm & 1 else None,
                k_weight=rng.uniform(0.5, 1.5, d).astype(np.float32) if norm & 2 else None), pages, page


def check_rotary(pbg, c, pages, page, heads, kv, d, inter=False, amplitude=1.0, eps=1e-6):
    m = len(c["position"])
    mark = np.float16(777)
    kc = torch.full((pages, kv, page, d), 777.0, dtype=torch.float16, device="cuda:0")
    vc = torch.full((pages, kv, page, d), 777.0, dtype=torch.float16, device="cuda:0")
    q = torch.full((m, heads, d), 777.0, dtype=torch.float16, device="cuda:0")
    pbg.rotary_qkv(dev(c["qkv"]), dev(c["position"]), dev(c["slot"]), dev(c["inv_freq"]), kc, vc, dev(c["q_weight"]), dev(c["k_weight"]),
                   eps, amplitude, inter, q=q)
    ref = oracle.rotary_qkv(c["qkv"], c["position"], c["inv_freq"], heads, kv, d, c["q_weight"], c["k_weight"], eps, amplitude, inter)
    plain = oracle.rotary_qkv(c["qkv"], c["position"], None, heads, kv, d, c["q_weight"], c["k_weight"], eps)
    half = 0 if c["inv_freq"] is None else len(c["inv_freq"])
    live = c["position"] >= 0
    kept = live & (c["slot"] >= 0) & (c["slot"] < pages * page)
    gk = host(kc).transpose(0, 2, 1, 3).reshape(pages * page, kv, d)
    gv = host(vc).transpose(0, 2, 1, 3).reshape(pages * page, kv, d)
    got = [host(q)[live], gk[c["slot"][kept]], gv[c["slot"][kept]]]
    for name, g, w, y, rows in zip("qkv", got, ref, plain, (live, kept, kept)):
        w, y = w[rows], np.abs(y[rows])
        pair = y.copy()  # |a| + |b| of the element's pair
        if name != "v" and half:
            a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if inter else (slice(0, half), slice(half, 2 * half))
            pair[..., a] = pair[..., b] = y[..., a] + y[..., b]
        rel = 0.0 if name == "v" else (d / 2 + 10 + 12) * U
        amp = max(abs(amplitude), 1.0)
        assert_within(g.astype(np.float64), w, (np.abs(w) * 2.0 ** -11 + amp * pair * rel) * 1.001 + 2.0 ** -25, name)
    assert (host(q)[~live] == mark).all()
    free = np.ones(pages * page, bool)
    free[c["slot"][kept]] = False
    assert (gk[free] == mark).all() and (gv[free] == mark).all()


ROTARY = [(1, 32, 8, 128, 128, False, 3), (7, 32, 8, 128, 128, True, 3), (333, 14, 2, 80, 32, True, 0), (300, 8, 8, 64, 64, False, 3),
          (5, 1, 1, 8, 8, False, 1), (5, 1, 1, 8, 8, True, 2), (3, 4, 2, 8, 0, False, 3), (40, 12, 4, 96, 72, False, 0),
          (260, 3, 3, 256, 256, False, 3), (260, 16, 1, 256, 64, True, 3), (9, 71, 1, 64, 16, False, 2), (256, 5, 5, 136, 128, False, 1),
          (255, 9, 3, 72, 40, True, 3), (2000, 32, 8, 128, 64, False, 3), (1, 1, 1, 248, 248, True, 3)]


@pytest.mark.parametrize("m,heads,kv,d,rot,inter,norm", ROTARY)
def test_rotary_qkv(pbg, m, heads, kv, d, rot, inter, norm):
    say(f"rotary m={m} heads={heads}/{kv} d={d} rot={rot} inter={inter} norm={norm}")
    c, pages, page = rotary_case(m + d, m, heads, kv, d, rot, norm)
    check_rotary(pbg, c, pages, page, heads, kv, d, inter)
    check_rotary(pbg, c, pages, page, heads, kv, d, inter, amplitude=1.31, eps=0.5)
    # rows behind the last request, rows without a slot, slots outside the cache
    c["position"][::3] = -1
    c["slot"][1::4] = -1
    c["slot"][2::7] = pages * page
    check_rotary(pbg, c, pages, page, heads, kv, d, inter)


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_far_positions(pbg, inter):
    """Angles of positions up to 2^24 keep their 64-bit reduction, with every kind of scaling."""
    c, pages, page = rotary_case(5, 300, 4, 2, 128, 128, 3, page=1, positions=2 ** 24)
    check_rotary(pbg, c, pages, page, 4, 2, 128, inter)
    for scaling in ("linear", "ntk", "yarn"):
        freq, amplitude = pbg.rotary_frequencies(128, 1e6, scaling, 4.0, 32768, "cuda:0")
        check_rotary(pbg, {**c, "inv_freq": host(freq)}, pages, page, 4, 2, 128, inter, amplitude)


def test_rotary_rows_do_not_mix(pbg):
    """NaN, infinities and overflow stay in their own head and row; values past fp16's range become infinities."""
    c, pages, page = rotary_case(6, 30, 6, 2, 64, 64, 3)
    base = [torch.zeros((pages, 2, page, 64), dtype=torch.float16, device="cuda:0") for _ in range(4)]
    args = lambda x, k, v: pbg.rotary_qkv(dev(x), dev(c["position"]), dev(c["slot"]), dev(c["inv_freq"]), k, v, dev(c["q_weight"]), dev(c["k_weight"]))  # noqa: E731
    q0 = args(c["qkv"], base[0], base[1])
    x = c["qkv"].copy().reshape(30, 10, 64)
    x[4, 2, 5], x[7, 6, 1], x[9, 9, 3], x[9, 8, 0] = np.nan, np.inf, 1e6, -np.inf
    q1 = args(x.reshape(30, -1), base[2], base[3])
    same = torch.ones((30, 6), dtype=torch.bool, device="cuda:0")
    same[4, 2] = False
    assert torch.equal(q0[same], q1[same]) and torch.isnan(q1[4, 2]).all()
    flat = [b.transpose(1, 2).reshape(pages * page, 2, 64) for b in base]
    s = c["slot"]
    assert torch.isnan(flat[2][s[7], 0]).any()
    assert float(flat[3][s[9], 1, 3]) == np.inf and float(flat[3][s[9], 0, 0]) == -np.inf
    keep = torch.ones((pages * page, 2), dtype=torch.bool, device="cuda:0")
    keep[s[7], 0] = False
    assert torch.equal(flat[0][keep], flat[2][keep])


# ---- tree_attention ---------------------------------------------------------


def attention_case(seed, lengths, added, heads, kv, d, page, tree=False, pad=0, width=0, spread=2.0):
    rng = np.random.default_rng(seed)
    lengths, added = np.array(lengths, np.int32), np.array(added, np.int32)
    used = -(-(lengths + added) // page)
    pages = int(used.sum()) + 2
    width = max(width, int(used.max(initial=1)) + 1, 1)
    table = np.full((len(lengths), width), -1, np.int32)
    ids, at = rng.permutation(pages), 0
    for i, n in enumerate(used):
        table[i, :n] = ids[at: at + n]
        at += n
    m = max(int(added.sum()) + pad, 1)
    row_start = np.concatenate([[0], np.cumsum(added)]).astype(np.int32)
    ancestors = None
    if tree:
        ancestors = np.zeros(m, np.uint64)
        for i in range(len(lengths)):
            parents = np.arange(added[i]) - rng.integers(1, 5, added[i])
            for c in range(min(int(added[i]), 64)):
                ancestors[row_start[i] + c] = sum(1 << p for p in oracle.tree_path(parents, c))
    return dict(q=(rng.standard_normal((m, heads, d)) * spread).astype(np.float16),
                k_cache=rng.standard_normal((pages, kv, page, d)).astype(np.float16),
                v_cache=rng.standard_normal((pages, kv, page, d)).astype(np.float16), table=table, lengths=lengths,
                row_start=row_start, ancestors=ancestors)


def attention_bound(c, ref, size, far, scale=None):
    d = c["q"].shape[2]
    scale = d ** -0.5 if scale is None else scale
    n = int(c["lengths"].max(initial=0)) + int(np.diff(c["row_start"]).max(initial=0))
    e = 2 * (d + 4) * U * scale * far + 30 * U + 2.0 ** -11  # d_s twice: in the weight and in the largest
    v = np.abs(c["v_cache"].astype(np.float64))
    high = np.nanmax(np.where(np.isfinite(v), v, 0.0))
    # rows without a weight are zero, whatever their scores
    some = np.where(size + np.abs(ref) > 0, e[:, :, None] + (n / 32 + 64) * U, 0.0)
    off = some * (size + np.abs(ref)) * 1.01 + n * 2.0 ** -25 * 2 * high
    return off + (np.abs(ref) + off) * 2.0 ** -11 + 2.0 ** -25


def check_attention(pbg, c, scale=None):
    mark = 333.0
    d = {k: dev(v) for k, v in c.items()}
    out = torch.full_like(d["q"], mark)
    pbg.tree_attention(**d, scale=scale, out=out)
    ref, size, far = oracle.tree_attention(**c, scale=scale)
    got = host(out).astype(np.float64)
    end = int(min(c["row_start"][-1], len(got)))
    assert (got[end:] == mark).all(), "rows behind the last request"
    assert_within(got[:end], ref[:end], attention_bound(c, ref, size, far, scale)[:end], "out")
    return out


HEADS = [(32, 8, 128), (4, 4, 64), (14, 2, 64), (12, 4, 80), (6, 2, 96), (3, 1, 256), (5, 5, 8), (9, 3, 136), (24, 1, 72), (71, 1, 64),
         (16, 1, 128), (130, 2, 32)]


@pytest.mark.parametrize("heads,kv,d", HEADS)
def test_attention_single_tokens(pbg, heads, kv, d):
    say(f"attention tokens {heads}/{kv} x {d}")
    lengths = [0, 1, 15, 16, 31, 32, 33, 127, 128, 129, 300, 5]
    check_attention(pbg, attention_case(d, lengths, [1] * 12, heads, kv, d, 16, pad=3))
    check_attention(pbg, attention_case(d, [700], [1], heads, kv, d, 64))


@pytest.mark.parametrize("page", [8, 16, 32, 64, 256, 4096])
def test_attention_pages(pbg, page):
    say(f"attention page={page}")
    check_attention(pbg, attention_case(page, [0, 7, 64, 130, 500], [3, 1, 8, 2, 5], 8, 2, 64, page))
    check_attention(pbg, attention_case(page, [9, 257], [30, 64], 8, 2, 128, page, tree=True, width=300))


@pytest.mark.parametrize("heads,kv,d,lengths,added,page,tree", [
    (24, 2, 256, [3000], [96], 16, False),                # several units of a tile in one workgroup
    (16, 1, 256, [3000, 0, 1500], [96, 200, 33], 64, False),
    (16, 1, 256, [2000, 0, 700, 64, 1], [40, 1, 64, 3, 64], 8, True),
    (8, 8, 200, [130, 63, 64, 65, 0], [129, 1, 1, 1, 257], 128, False),  # single tokens beside prompts
    (40, 2, 136, [900, 5], [17, 70], 8, False),           # 20 query heads a key head: a row and its pair's tail empty
    (130, 1, 256, [200, 31], [5, 2], 32, True)])          # more heads than a tile has rows
def test_attention_wide_heads(pbg, heads, kv, d, lengths, added, page, tree):
    """Two waves a query row: its tokens' halves and the halves of its columns meet."""
    say(f"attention wide heads {heads}/{kv} x {d} {lengths} {added}")
    c = attention_case(d + heads, lengths, added, heads, kv, d, page, tree=tree, pad=2)
    check_attention(pbg, c)
    # a page in the middle that no request has, and what no row sees is not finite
    c["table"][0, c["lengths"][0] // page // 2] = -1
    for cache in (c["k_cache"], c["v_cache"]):
        free = np.setdiff1d(np.arange(len(cache)), c["table"])
        cache[free] = np.nan
        for i in range(len(lengths)):
            end = int(c["lengths"][i] + added[i])
            if end % page and c["table"][i, end // page] >= 0:
                cache[c["table"][i, end // page], :, end % page:] = np.inf
    # one score far above the others, in either half of a unit, early and late
    for t in (3, 40, int(c["lengths"][0]) - 1):
        number = c["table"][0, t // page]
        if number >= 0:
            c["k_cache"][number, :, t % page] = c["q"][0, :kv] * 4
    check_attention(pbg, c)


@pytest.mark.parametrize("heads,kv,d", HEADS)
def test_attention_trees(pbg, heads, kv, d):
    say(f"attention trees {heads}/{kv} x {d}")
    check_attention(pbg, attention_case(d + 1, [0, 40, 129], [64, 7, 33], heads, kv, d, 16, tree=True, pad=2))
    check_attention(pbg, attention_case(d + 2, [200, 3], [5, 2], heads, kv, d, 32, tree=True))


@pytest.mark.parametrize("heads,kv,d", HEADS)
def test_attention_prompts(pbg, heads, kv, d):
    say(f"attention prompts {heads}/{kv} x {d}")
    check_attention(pbg, attention_case(d + 3, [0, 100, 0], [150, 75, 1], heads, kv, d, 16, pad=1))


def test_attention_prompt_lengths(pbg):
    """Prompts that end around the sizes of tiles, alone and after cached tokens."""
    for n in (15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257):
        for have in (0, 1, 63, 128):
            say(f"attention prompt n={n} have={have}")
            check_attention(pbg, attention_case(n + have, [have], [n], 2, 1, 64, 16))


def test_attention_mixed_batch(pbg):
    """Prompts, trees' worth of rows, single tokens and idle requests side by side."""
    check_attention(pbg, attention_case(1, [0, 600, 33, 0, 0, 90, 1000], [300, 1, 0, 0, 1, 20, 1], 8, 2, 128, 16, pad=5))
    check_attention(pbg, attention_case(2, [5] * 200, [1] * 200, 4, 1, 64, 8))
    check_attention(pbg, attention_case(3, [0] * 50 + [900] + [0] * 50, [0] * 50 + [9] + [2] * 50, 4, 2, 64, 8))


@pytest.mark.parametrize("heads,kv,d,rows", [(4, 1, 128, 1), (4, 2, 64, 6), (2, 1, 256, 3), (4, 1, 128, 40)])
def test_attention_long_context_in_pieces(pbg, heads, kv, d, rows):
    """More tokens than one workgroup takes: every workgroup has a piece, and they are joined."""
    say(f"attention long {heads}/{kv} x {d} rows={rows}")
    check_attention(pbg, attention_case(d, [30001], [rows], heads, kv, d, 16, tree=True))
    check_attention(pbg, attention_case(d, [9000, 12, 14001], [rows, 2, 1], heads, kv, d, 64))


def test_attention_pieces_of_both_kernels(pbg):
    """Single tokens of long requests beside prompts, each in several pieces, with up to and with more than 64 requests."""
    check_attention(pbg, attention_case(4, [9000, 700, 0, 12001], [1, 250, 130, 2], 4, 1, 64, 16, pad=4))
    check_attention(pbg, attention_case(5, [6000, 300], [1, 140], 6, 1, 128, 32))
    check_attention(pbg, attention_case(6, [6000, 300], [1, 140], 8, 1, 256, 32))
    many = [int(x) for x in np.random.default_rng(7).integers(0, 300, 90)]
    check_attention(pbg, attention_case(7, many, [700 if i == 50 else 40 if i % 30 == 0 else i % 3 for i in range(90)], 8, 1, 64, 16))


def test_attention_trees_with_more_rows_than_a_tree_has(pbg):
    """Of a request's rows from the 64th on none is seen; those rows themselves see what their masks say."""
    c = attention_case(8, [20, 7], [100, 3], 4, 2, 64, 16, tree=True)
    c["ancestors"][64:100] = np.random.default_rng(1).integers(0, 2 ** 63, 36).astype(np.uint64)
    check_attention(pbg, c)
    c["ancestors"][:] = np.uint64(2 ** 64 - 1)
    check_attention(pbg, c)


def test_attention_refusals_of_the_binding(pbg):
    c = {k: dev(v) for k, v in attention_case(9, [20, 7], [2, 3], 4, 2, 64, 16).items()}
    for bad in (dict(q=c["q"][:, :, :32]), dict(q=c["q"].transpose(0, 1)), dict(lengths=c["lengths"][:1]), dict(lengths=c["lengths"].long()),
                dict(row_start=c["row_start"][:2]), dict(table=c["table"].cpu()), dict(v_cache=c["v_cache"][:1]), dict(ancestors=c["lengths"]),
                dict(out=torch.empty_like(c["q"]).float()), dict(workspace=torch.empty(4))):
        with pytest.raises(ValueError):
            pbg.tree_attention(**{**c, **bad})
    for bad in (dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda:0")), dict(scale=0.0), dict(scale=NAN)):
        with pytest.raises(pbg.PbgError):
            pbg.tree_attention(**{**c, **bad})


def test_attention_sharp_scores(pbg):
    """A few tokens hold all the weight, the largest score comes late or early, and weights fall below fp16's range."""
    for scale in (0.01, 1.0, 30.0):
        for where in (3, 200, 399):
            c = attention_case(7, [400, 130], [1, 3], 4, 2, 64, 16)
            k = oracle.cached_tokens(c["k_cache"], c["table"][0], 400, 0)[0]
            page, off = c["table"][0][where // 16], where % 16
            c["k_cache"][page, 0, off] = np.sign(c["q"][0, 0]) * 3
            assert k.shape == (400, 64)
            check_attention(pbg, c, scale=scale)


@pytest.mark.parametrize("rows", [1, 20])
def test_attention_rows_that_see_nothing(pbg, rows):
    """No cached tokens and an empty mask; a mask of tokens that are not there; tokens without a page; scores of -infinity only."""
    c = attention_case(8, [0, 50, 0], [rows, rows, rows], 4, 2, 64, 16, tree=True)
    c["ancestors"][: rows] = 0
    c["ancestors"][2 * rows:] = np.uint64(1 << 63)
    out = host(check_attention(pbg, c))
    assert (out[:rows] == 0).all() and (out[2 * rows: 3 * rows] == 0).all()
    c = attention_case(9, [40, 70], [rows, rows], 4, 2, 64, 16)
    c["table"][0, :] = 10 ** 6
    c["table"][1, 1] = -5
    out = host(check_attention(pbg, c))
    assert (out[:rows] == 0).all()
    c = attention_case(10, [40, 20], [rows, rows], 4, 2, 64, 16)
    c["q"][:] = np.abs(c["q"]) + np.float16(1)
    c["k_cache"][:] = -np.inf
    out = check_attention(pbg, c)
    assert (host(out)[: 2 * rows] == 0).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("heads,kv,d", [(8, 2, 128), (4, 4, 64), (3, 1, 256)])
def test_attention_what_is_not_seen_does_not_matter(pbg, bad, heads, kv, d):
    """NaN and infinities behind the last token, in sibling branches, in later rows of a prompt and in other requests' pages."""
    say(f"attention unseen {bad} {heads}/{kv} x {d}")
    for tree, added in ((True, [30, 5, 64]), (False, [30, 1, 150]), (False, [1, 1, 1])):
        c = attention_case(d, [33, 200, 64], added, heads, kv, d, 16, tree=tree)
        clean = {k: v.copy() if v is not None else None for k, v in c.items()}
        base = host(pbg.tree_attention(**{k: dev(v) for k, v in clean.items()}))
        # everything that no request uses
        used = np.zeros(c["k_cache"].shape[:1] + (16,), bool)
        for i in range(3):
            for t in range(c["lengths"][i] + added[i]):
                used[c["table"][i, t // 16], t % 16] = True
        for cache in (c["k_cache"], c["v_cache"]):
            cache.transpose(0, 2, 1, 3)[~used] = bad
        got = host(pbg.tree_attention(**{k: dev(v) for k, v in c.items()}))
        assert np.array_equal(got.view(np.uint16), base.view(np.uint16))
        # one row of the step: those that do not see it keep their bits, those that do follow the formula
        if added[2] == 1:
            continue
        row, t = 20, 64 + 20
        page, off = c["table"][2, t // 16], t % 16
        c["v_cache"][page, :, off, 3] = bad
        got = host(pbg.tree_attention(**{k: dev(v) for k, v in c.items()}))
        first = int(c["row_start"][2])
        sees = np.array([(int(c["ancestors"][first + a]) >> row & 1) if tree else a >= row for a in range(added[2])], bool)
        assert sees.any() and not sees.all()
        assert np.array_equal(got[first: first + added[2]][~sees].view(np.uint16), base[first: first + added[2]][~sees].view(np.uint16))
        mine = got[first: first + added[2]][sees]
        assert np.array_equal(mine[..., 3], np.full(mine.shape[:2], bad, np.float16), equal_nan=True)
        keep = np.arange(d) != 3
        assert np.array_equal(mine[..., keep].view(np.uint16), base[first: first + added[2]][sees][..., keep].view(np.uint16))
        c["k_cache"][page, :, off, 5] = np.nan
        got = host(pbg.tree_attention(**{k: dev(v) for k, v in c.items()}))
        assert np.isnan(got[first: first + added[2]][sees]).all()
        assert np.array_equal(got[first: first + added[2]][~sees].view(np.uint16), base[first: first + added[2]][~sees].view(np.uint16))


@pytest.mark.parametrize("rows", [1, 9, 200])
def test_attention_nan_rows_stay_alone(pbg, rows):
    """A NaN query or a NaN cached token reaches its own rows and requests only."""
    c = attention_case(11, [300, 40, 128], [rows, rows, rows], 8, 2, 64, 16)
    base = host(pbg.tree_attention(**{k: dev(v) for k, v in c.items()}))
    c["q"][rows // 2, 3, 7] = np.nan
    c["v_cache"][c["table"][1, 0], 1, 5, 9] = np.inf
    got = host(pbg.tree_attention(**{k: dev(v) for k, v in c.items()}))
    assert np.isnan(got[rows // 2, 3]).all()
    assert np.isinf(got[rows: 2 * rows, 4:, 9]).all()
    same = np.ones(base.shape, bool)
    same[rows // 2, 3] = False
    same[rows: 2 * rows, 4:, 9] = False
    assert np.array_equal(got[same].view(np.uint16), base[same].view(np.uint16))


def test_attention_hostile_tables(pbg):
    """Lengths beyond the table, negative ones, row starts that run backwards or past the rows: bounded, and sound elsewhere."""
    c = attention_case(12, [40, 10, 20, 30], [2, 2, 2, 2], 4, 2, 64, 16)
    good = host(pbg.tree_attention(**{k: dev(v) for k, v in c.items()}))
    bad = {**c, "lengths": np.array([40, 2 ** 31 - 1, -3, 30], np.int32)}
    got = host(pbg.tree_attention(**{k: dev(v) for k, v in bad.items()}))
    assert np.array_equal(got[[0, 1, 6, 7]], good[[0, 1, 6, 7]])
    check_attention(pbg, {**c, "lengths": np.array([40, 200, 0, 30], np.int32)})
    for rows in (2, 30):
        c2 = attention_case(12, [40, 10, 20], [rows, rows, rows], 4, 2, 64, 16)
        check_attention(pbg, {**c2, "lengths": np.array([40, 2 ** 31 - 1, 2 ** 31 - 1 - rows], np.int32)})
    bad = {**c, "row_start": np.array([0, 2, -5, 6, 100], np.int32)}
    pbg.tree_attention(**{k: dev(v) for k, v in bad.items()})
    bad = {**c, "row_start": np.array([-9, 2, 4, 2, 8], np.int32)}
    pbg.tree_attention(**{k: dev(v) for k, v in bad.items()})
    torch.cuda.synchronize()


def test_attention_far_pages(pbg):
    """Pages whose elements lie past 2^32 bytes and past 2^31 elements of the cache."""
    pages, kv, page, d = 17000, 8, 128, 128
    k = torch.zeros((pages, kv, page, d), dtype=torch.float16, device="cuda:0")
    v = torch.zeros((pages, kv, page, d), dtype=torch.float16, device="cuda:0")
    c = attention_case(13, [700, 100], [2, 3], 16, kv, d, page)
    n = c["k_cache"].shape[0]
    where = torch.from_numpy(np.linspace(pages // 2 - 3, pages - 1, n).astype(np.int64))
    k[where], v[where] = dev(c["k_cache"]), dev(c["v_cache"])
    base = pbg.tree_attention(**{x: dev(y) for x, y in c.items()})
    table = np.where(c["table"] >= 0, where.numpy()[np.maximum(c["table"], 0)], -1).astype(np.int32)
    far = pbg.tree_attention(dev(c["q"]), k, v, dev(table), dev(c["lengths"]), dev(c["row_start"]))
    assert torch.equal(far, base)
    del k, v
    torch.cuda.empty_cache()


@pytest.mark.parametrize("lengths,added,tree", [([300, 5000], [1, 1], False), ([3000], [7], True), ([50, 900], [130, 64], False)])
def test_attention_same_bits_graph_streams_workspace(pbg, lengths, added, tree):
    """The same call gives the same bits; a graph follows its inputs; two graphs share a workspace in turn; two streams with their own
    run side by side; nothing is written past the workspace that was asked for."""
    c = attention_case(14, lengths, added, 8, 2, 128, 16, tree=tree)
    d = {k: dev(v) for k, v in c.items()}
    size = pbg.attention_workspace(8, 2, 128, "cuda:0").numel()
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda:0")
    base = pbg.tree_attention(**d, workspace=ws[:size])
    assert (ws[size:] == 255).all()
    for _ in range(3):
        assert torch.equal(pbg.tree_attention(**d, workspace=ws[:size]), base)
    c2 = attention_case(15, lengths[::-1], added[::-1], 8, 2, 128, 16, tree=tree)
    d2 = {k: dev(v) for k, v in c2.items()}
    base2 = pbg.tree_attention(**d2)
    outs, graphs = [torch.zeros_like(base), torch.zeros_like(base2)], []
    for x, o in zip((d, d2), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pbg.tree_attention(**x, out=o, workspace=ws[:size])
        graphs.append(g)
    for _ in range(3):
        for g, o, b in zip(graphs, outs, (base, base2)):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, b)
    # shorter requests through the same graph
    short = np.maximum(c["lengths"] // 2, 0).astype(np.int32)
    d["lengths"].copy_(dev(short))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], pbg.tree_attention(**{**d, "lengths": dev(short)}))
    d["lengths"].copy_(dev(c["lengths"]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [pbg.attention_workspace(8, 2, 128, "cuda:0") for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for n, (st, x, w) in enumerate(zip(streams, (d, d2), spaces)):
            with torch.cuda.stream(st):
                got[n].append(pbg.tree_attention(**x, workspace=w))
    torch.cuda.synchronize()
    assert all(torch.equal(g, base) for g in got[0]) and all(torch.equal(g, base2) for g in got[1])


# ---- penalize_logits --------------------------------------------------------


def logits_case(seed, r, rows, n, hist, drafts=False, bias=0, grammar=0, outside=True):
    rng = np.random.default_rng(seed)
    m = r * rows
    lo, hi = (-3, n + 5) if outside else (0, n)
    c = dict(logits=(rng.standard_normal((m, n)) * 3).astype(np.float32), request=np.repeat(np.arange(r), rows).astype(np.int32),
             tokens=rng.integers(lo, hi, (r, max(hist, 1))).astype(np.int32),
             length=rng.integers(0, hist + 1, r).astype(np.int32), prompt_length=rng.integers(0, hist + 1, r).astype(np.int32),
             repetition=rng.uniform(0.8, 1.5, r).astype(np.float32), frequency=rng.uniform(-0.2, 0.5, r).astype(np.float32),
             presence=rng.uniform(-0.2, 0.5, r).astype(np.float32))
    c["logits"][:, :: max(1, n // 7)] = 1.5  # ties
    c["logits"][:, 1:: max(2, n // 5)] = np.float32(-0.0)
    if drafts:
        c["drafts"] = rng.integers(lo, hi, m).astype(np.int32)
        c["row_start"] = (np.arange(r + 1) * rows).astype(np.int32)
        c["ancestors"] = rng.integers(0, 2 ** min(rows, 63), m).astype(np.uint64)
    if bias:
        counts = rng.integers(0, bias + 1, r)
        c["bias_start"] = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        c["bias_token"] = rng.integers(lo, min(hi, lo + 50), max(int(counts.sum()), 1)).astype(np.int32)
        c["bias_value"] = (rng.standard_normal(len(c["bias_token"])) * 5).astype(np.float32)
    if grammar:
        c["grammar"] = rng.integers(0, 2 ** 32, (grammar, (n + 31) // 32), dtype=np.uint64).astype(np.uint32)
        c["grammar_row"] = rng.integers(-1, grammar + 1, m).astype(np.int32)
    return c


def check_logits(pbg, c, in_place=False):
    d = {k: dev(v) for k, v in c.items()}
    mark = torch.full_like(d["logits"], 123.0)
    out = d["logits"] if in_place else mark
    token = torch.full((len(c["request"]),), -77, dtype=torch.int32, device="cuda:0")
    top = torch.full((len(c["request"]),), 77.0, device="cuda:0")
    pbg.penalize_logits(**d, out=out, token=token, top=top)
    ref, tok, best = oracle.penalize_logits(**c)
    live = tok != -2
    got = host(out)
    assert np.array_equal(got[live].view(np.uint32) & 0xFFFFFFFF, ref[live].view(np.uint32)) or np.array_equal(got[live], ref[live], equal_nan=True)
    assert np.array_equal(got[~live], c["logits"][~live] if in_place else host(mark)[~live])
    assert np.array_equal(host(token)[live], tok[live]) and (host(token)[~live] == -77).all()
    assert np.array_equal(host(top)[live], best[live]) and (host(top)[~live] == 77.0).all()
    return out


LOGITS = [(1, 1, 1, 0, 0, 0), (1, 1, 3, 5, 2, 1), (2, 3, 31, 9, 0, 2), (3, 2, 1023, 100, 5, 0), (1, 1, 8192, 300, 0, 1), (2, 1, 8193, 50, 9, 3),
          (1, 8, 20000, 5000, 60, 2), (5, 4, 4099, 1, 1, 1), (1, 2, 151936, 40000, 100, 1), (64, 1, 1000, 10, 3, 4), (1, 1, 70000, 20000, 0, 0)]


@pytest.mark.parametrize("r,rows,n,hist,bias,grammar", LOGITS)
def test_penalize_logits(pbg, r, rows, n, hist, bias, grammar):
    say(f"logits r={r} rows={rows} n={n} history={hist} bias={bias} grammar={grammar}")
    c = logits_case(n + r, r, rows, n, hist, rows > 1, bias, grammar)
    check_logits(pbg, c)
    check_logits(pbg, c, in_place=True)
    c["request"][::2] = -1
    c["request"][1::5] = r
    check_logits(pbg, c)


def test_penalize_logits_ends(pbg):
    """Everything forbidden, NaN and infinities among the logits, lengths and lists outside their arrays, whole histories as prompt."""
    c = logits_case(1, 3, 2, 5000, 200, True, 20, 2)
    c["grammar"][0] = 0
    c["grammar_row"][:] = [0, 1, -1, 0, 5, 1]
    out = check_logits(pbg, c)
    assert torch.isinf(out[0]).all()
    c["logits"][1, :50], c["logits"][2, 7], c["logits"][2, 9], c["logits"][3] = np.nan, np.inf, -np.inf, np.nan
    check_logits(pbg, c)
    c["length"][:], c["prompt_length"][:] = [-4, 10 ** 6, 200], [5, 10 ** 6, -1]
    check_logits(pbg, c)
    c["bias_start"][:] = [-3, 5, 2, 10 ** 6]
    check_logits(pbg, c)
    c["row_start"][:] = [-2, 5, 100, 0]
    check_logits(pbg, c)
    c["repetition"][:], c["frequency"][:], c["presence"][:] = [np.inf, 1e-30, -1.0], [0.0, 1e30, -0.0], [np.inf, 0.0, 1e-40]
    check_logits(pbg, c)


def test_penalize_logits_one_token_many_times(pbg):
    """Every token of a long history is the same: one counter takes them all."""
    c = logits_case(2, 2, 1, 9000, 30000, outside=False)
    c["tokens"][:], c["length"][:], c["prompt_length"][:] = 8500, 30000, [0, 100]
    check_logits(pbg, c)


def test_penalize_logits_in_a_graph(pbg):
    c = logits_case(3, 4, 3, 30001, 700, True, 30, 2)
    d = {k: dev(v) for k, v in c.items()}
    base = pbg.penalize_logits(**d, greedy=True)
    outs = [torch.zeros_like(b) for b in base]
    ws = pbg.logits_workspace(12, 30001, "cuda:0")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pbg.penalize_logits(**d, out=outs[0], token=outs[1], top=outs[2], workspace=ws)
    for k in range(3):
        for o in outs:
            o.zero_()
        ws.fill_(-1)
        d["length"].copy_(dev(np.maximum(c["length"] - 50 * k, 0)))
        graph.replay()
        torch.cuda.synchronize()
        want = pbg.penalize_logits(**d, greedy=True)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


# ---- together ---------------------------------------------------------------


def test_a_prompt_a_verify_step_and_tokens_together(pbg):
    """Two requests through the whole half layer: prompts, a tree of drafted tokens of which a path is kept, single tokens; each step's
    attention is the oracle's over the keys and values that the steps before it left in the cache."""
    rng = np.random.default_rng(5)
    heads, kv, d, page, pages, width, n = 8, 2, 64, 16, 24, 9, 1000
    k_cache = torch.full((pages, kv, page, d), NAN, dtype=torch.float16, device="cuda:0")
    v_cache = torch.full((pages, kv, page, d), NAN, dtype=torch.float16, device="cuda:0")
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda:0")
    free, left = dev(rng.permutation(pages).astype(np.int32)), dev(np.array([pages], np.int32))
    freq, amp = pbg.rotary_frequencies(d, 1e4, "yarn", 2.0, 64, "cuda:0")
    w = [dev(rng.uniform(0.5, 1.5, d).astype(np.float32)) for _ in range(2)]
    ws = pbg.attention_workspace(heads, kv, d, "cuda:0")
    lengths = np.zeros(2, np.int32)
    steps = [([37, 50], None), ([6, 4], [-1, 0, 0, 1, 2, 4, -1, 0, 1, 1]), ([1, 1], None), ([0, 1], None)]
    for n_step, (added, parents) in enumerate(steps):
        say(f"together step {n_step}")
        rows = sum(added) + 2
        par = None if parents is None else dev(np.array(parents + [0, 0], np.int32))
        start, request, position, slot, anc, left = pbg.cache_plan(dev(lengths), dev(np.array(added, np.int32)), table, free, left, page,
                                                                   pages, parents=par, rows=rows)
        qkv = rng.standard_normal((rows, (heads + 2 * kv) * d)).astype(np.float32)
        q = pbg.rotary_qkv(dev(qkv), position, slot, freq, k_cache, v_cache, *w, amplitude=amp)
        out = pbg.tree_attention(q, k_cache, v_cache, table, dev(lengths), start, anc, workspace=ws)
        c = dict(q=host(q), k_cache=host(k_cache), v_cache=host(v_cache), table=host(table), lengths=lengths, row_start=host(start),
                 ancestors=None if anc is None else host(anc).view(np.uint64))
        ref, size, far = oracle.tree_attention(**c)
        end = sum(added)
        assert np.isfinite(ref[:end]).all()
        assert_within(host(out)[:end].astype(np.float64), ref[:end], attention_bound(c, ref, size, far)[:end], f"step {n_step}")
        # the o linear's 8-bit rows
        q8, s8 = pbg.quantize_rows(out[:end].reshape(end, heads * d))
        assert torch.isfinite(s8).all()
        if parents is None:
            lengths = lengths + np.array(added, np.int32)
            continue
        # rows 0, 2, 4, 5 of the first request's tree were accepted, rows 0, 1, 2 of the second's: their keys and values move together
        for i, path in enumerate(([0, 2, 4, 5], [0, 1])):
            rows_at = [int(host(start)[i]) + p for p in path]
            assert host(position)[rows_at].tolist() == [lengths[i] + j for j in range(len(path))]
            src = slot[torch.tensor(rows_at, device="cuda:0")]
            dst = slot[int(host(start)[i]): int(host(start)[i]) + len(path)]
            for cache in (k_cache, v_cache):
                cache[dst // page, :, dst % page] = cache[src // page, :, src % page]
            lengths[i] += len(path)
    # the tree's penalties: a row's own branch counts
    m = 10
    logits = rng.standard_normal((m, n)).astype(np.float32)
    plan = oracle.cache_plan(np.array([5, 6]), np.array([6, 4]), np.zeros((2, 4), np.int32), np.arange(8), 8, page, 8, m,
                             np.array(steps[1][1], np.int32))
    c = dict(logits=logits, request=plan[1], tokens=rng.integers(0, n, (2, 60)).astype(np.int32), length=np.array([50, 60], np.int32),
             prompt_length=np.array([20, 0], np.int32), repetition=np.array([1.2, 1.0], np.float32),
             frequency=np.array([0.1, 0.3], np.float32), presence=np.array([0.2, 0.0], np.float32),
             drafts=rng.integers(0, n, m).astype(np.int32), row_start=plan[0], ancestors=plan[4])
    check_logits(pbg, c)


def test_tokens_one_by_one_equal_the_prompt(pbg):
    """A prompt in one step, and the same tokens one step each: the same queries, keys and values, bit for bit, and attention within
    twice the tolerance."""
    rng = np.random.default_rng(6)
    heads, kv, d, page, n = 4, 2, 128, 8, 45
    qkv = dev(rng.standard_normal((n, (heads + 2 * kv) * d)).astype(np.float32))
    freq, _ = pbg.rotary_frequencies(d, device="cuda:0")
    free = dev(np.arange(8, dtype=np.int32))
    results = []
    for pieces in ([n], [1] * n, [20, 1, 24]):
        k, v = (torch.zeros((8, kv, page, d), dtype=torch.float16, device="cuda:0") for _ in range(2))
        table = torch.full((1, 8), -1, dtype=torch.int32, device="cuda:0")
        left, have, outs = dev(np.array([8], np.int32)), 0, []
        for p in pieces:
            lengths = dev(np.array([have], np.int32))
            start, _, position, slot, _, left = pbg.cache_plan(lengths, dev(np.array([p], np.int32)), table, free, left, page, 8, rows=p)
            q = pbg.rotary_qkv(qkv[have: have + p], position, slot, freq, k, v)
            outs.append(pbg.tree_attention(q, k, v, table, lengths, start))
            have += p
        results.append((torch.cat(outs), k, v, table))
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r[1:], results[0][1:]))
        diff = (r[0].float() - results[0][0].float()).abs().max()
        assert float(diff) < 2 * 2.0 ** -10 * float(v.float().abs().max())
