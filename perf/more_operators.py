"""The cases on which the attention half of a step and the logits' penalties of packed_bit_gemv_amd are measured.

Four operators: cache_plan (block tables, slots and positions of a step's rows from the requests' lengths, and the ancestors
of drafted tokens), rotary_qkv (per-head norms and rotary positions of a q|k|v linear's output, keys and values written into
the cache's pages), tree_attention (attention over the paged cache for single tokens, trees of drafted tokens and prompts)
and penalize_logits (penalties for repeated tokens, biases and grammar masks on logits, with the greedy token).

The head shapes are those of the decoder layer this library serves (32 query heads over 8 key and value heads of 128) and
generic ones; the longest context is that model's 40,960 tokens, the widest logits its 151,936.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TREE = 64  # rows of one request that a tree can have
CONTEXT = 40960
VOCABULARY = 151936


def listed():
    return [
        # the tables of a decode step: one token of each of 64 requests
        {"name": "plan-decode", "op": "plan", "r": 64, "ctx": 8192, "new": 1, "ragged": 0.9, "page": 16, "tree": False, "pad": 0},
        # the tables of a step with many prompts and an odd number of requests, some rows unused
        {"name": "plan-prompts", "op": "plan", "r": 257, "ctx": 1000, "new": 100, "ragged": 0.9, "page": 64, "tree": False, "pad": 77},
        # one decoded token: its latency is what counts
        {"name": "rotary-token", "op": "rotary", "m": 1, "heads": 32, "kv": 8, "d": 128, "rot": 128, "inter": False, "norm": True, "ctx": 4096, "page": 16, "pad": 0},
        # a prompt, heads of which a part is rotated, pairs side by side, positions past the trained context
        {"name": "rotary-part", "op": "rotary", "m": 333, "heads": 14, "kv": 2, "d": 80, "rot": 32, "inter": True, "norm": False, "ctx": 40000, "page": 32, "pad": 5},
        # a long prompt
        {"name": "rotary-prompt", "op": "rotary", "m": 4096, "heads": 32, "kv": 8, "d": 128, "rot": 128, "inter": False, "norm": True, "ctx": 0, "page": 64, "pad": 0},
        # one decoded token of one request: its latency is what counts
        {"name": "attention-token", "op": "attention", "r": 1, "ctx": 1000, "new": 1, "ragged": 0.0, "tree": False, "heads": 32, "kv": 8, "d": 128, "page": 16, "pad": 0},
        # a verify step of seven rows at the end of the longest context
        {"name": "attention-verify", "op": "attention", "r": 1, "ctx": CONTEXT - 7, "new": 7, "ragged": 0.0, "tree": True, "heads": 32, "kv": 8, "d": 128, "page": 64, "pad": 1},
        # one decoded token of each of 64 requests of very different lengths
        {"name": "attention-batch", "op": "attention", "r": 64, "ctx": 8192, "new": 1, "ragged": 0.9, "tree": False, "heads": 32, "kv": 8, "d": 128, "page": 16, "pad": 0},
        # trees of up to 61 drafted tokens of 16 requests
        {"name": "attention-trees", "op": "attention", "r": 16, "ctx": 4100, "new": 61, "ragged": 0.5, "tree": True, "heads": 32, "kv": 8, "d": 128, "page": 32, "pad": 3},
        # a chunk of a long prompt over what came before it
        {"name": "attention-chunk", "op": "attention", "r": 1, "ctx": 8192, "new": 4096, "ragged": 0.0, "tree": False, "heads": 32, "kv": 8, "d": 128, "page": 64, "pad": 0},
        # one request's logits, a long history
        {"name": "logits-token", "op": "logits", "r": 1, "new": 1, "n": VOCABULARY, "history": 8000, "bias": 0, "grammar": False},
        # a verify step of eight requests, with biases and grammars
        {"name": "logits-verify", "op": "logits", "r": 8, "new": 8, "n": VOCABULARY, "history": 2000, "bias": 40, "grammar": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


HEADS = [(32, 8, 128), (32, 8, 128), (16, 8, 128), (8, 8, 64), (14, 2, 64), (12, 4, 80), (24, 3, 96), (16, 1, 256)]


def draw(rng):
    op = rng.choice(["plan", "rotary", "attention", "attention", "logits"])
    page, pad = rng.choice([8, 16, 32, 64, 128]), rng.choice([0, 0, rng.randint(1, 40)])
    if op == "plan":
        tree, r = rng.random() < 0.4, _log(rng, 1, 512)
        new = rng.randint(1, min(TREE, 32768 // r)) if tree else _log(rng, 1, 32768 // r)
        return {"op": op, "r": r, "ctx": rng.choice([0, _log(rng, 1, CONTEXT)]), "new": new, "ragged": rng.random(), "page": page,
                "tree": tree, "pad": pad}
    if op == "rotary":
        heads, kv, d = rng.choice(HEADS)
        return {"op": op, "m": _log(rng, 1, 4096 * 48 * 128 // ((heads + 2 * kv) * d)), "heads": heads, "kv": kv, "d": d,
                "rot": rng.choice([d, d, 8 * rng.randint(1, d // 8)]), "inter": rng.random() < 0.4, "norm": rng.random() < 0.6,
                "ctx": rng.choice([0, _log(rng, 1, CONTEXT)]), "page": page, "pad": pad}
    if op == "attention":
        heads, kv, d = rng.choice(HEADS)
        kind = rng.choice(["token", "tree", "prompt"])
        # what the cache holds, and the scores of every request at once
        new = {"token": 1, "tree": rng.randint(2, TREE), "prompt": _log(rng, 2, 4096)}[kind]
        ctx = _log(rng, 1, CONTEXT if kind != "prompt" else 8192)
        r = _log(rng, 1, max(1, min(64, 64 * 8192 * 1024 // ((ctx + new) * kv * d), (3 << 29) // ((ctx + new) * new * heads))))
        return {"op": op, "r": r, "ctx": ctx, "new": new, "ragged": rng.random(), "tree": kind == "tree", "heads": heads, "kv": kv, "d": d,
                "page": page, "pad": pad}
    new = rng.choice([1, 1, rng.randint(2, 16)])
    return {"op": op, "r": _log(rng, 1, 64 // new), "new": new, "n": rng.choice([VOCABULARY, _log(rng, 100, VOCABULARY)]),
            "history": rng.choice([0, _log(rng, 1, 20000)]), "bias": rng.choice([0, _log(rng, 1, 300)]), "grammar": rng.random() < 0.5}


# ---- inputs ----------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _spread(case, key, least):
    """A value for each request: the case's for the first, less by up to its share `ragged` for the others."""
    return [max(least, round(case[key] * (1.0 - case["ragged"] * (i * 0.6180339887 % 1.0)))) for i in range(case["r"])]


def _lengths(case):
    """Tokens that each request has in the cache, and rows that it adds."""
    return _spread(case, "ctx", 0), _spread(case, "new", 1)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def _parents(g, added, rows):
    """A drafted tree for each request: the parent of row c is one of the four rows before it, or the cached context."""
    row = torch.cat([torch.arange(c, device=DEV) for c in added] + [torch.zeros(rows - sum(added), dtype=torch.int64, device=DEV)])
    back = torch.randint(1, 5, (rows,), generator=g, device=DEV)
    return (row - back).clamp(min=-1).to(torch.int32)


def _reach(parents, start, r):
    """[r, TREE, TREE]: whether row c of a request is c' or descends from it."""
    c = torch.arange(TREE, device=DEV)
    rows = start[1:] - start[:-1]
    at = (start[:-1, None] + c).clamp(max=parents.numel() - 1)
    parent = parents.long()[at]
    fine = (c < rows[:, None]) & (parent >= 0) & (parent < c)
    step = torch.eye(TREE, device=DEV) + (fine[:, :, None] & (parent[:, :, None] == c)).float()
    # paths of up to TREE - 1 steps; the counts stay far below the end of fp32
    return (torch.linalg.matrix_power(step, TREE - 1) > 0) & (c < rows[:, None])[:, :, None]


def _bits(reach):
    return (reach.long() << torch.arange(TREE, device=DEV)).sum(-1)


def _plan_inputs(case, seed):
    g, page = _gen(seed), case["page"]
    lengths, added = _lengths(case)
    rows = sum(added) + case["pad"]
    have, want = [-(-a // page) for a in lengths], [-(-(a + b) // page) for a, b in zip(lengths, added)]
    pages = sum(want) + 19
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    width = max(want) + 3
    table = torch.full((case["r"], width), -1, dtype=torch.int32, device=DEV)
    held = torch.arange(width, device=DEV) < _i32(have)[:, None]
    table[held] = ids[: sum(have)]
    return {"lengths": _i32(lengths), "added": _i32(added), "table": table, "free_pages": ids[sum(have):].clone(),
            "free_count": _i32([pages - sum(have)]), "pages": pages, "rows": rows,
            "parents": _parents(g, added, rows) if case["tree"] else None}


def _rotary_inputs(case, seed):
    g, m, h, kv, d, page = _gen(seed), case["m"], case["heads"], case["kv"], case["d"], case["page"]
    rows = m + case["pad"]
    pages = -(-m // page) + 3
    # tokens of consecutive positions in pages of any order; rows behind the last sequence have neither
    order = torch.randperm(pages, generator=g, device=DEV)
    t = torch.arange(m, device=DEV)
    slot, position = torch.full((rows,), -1, dtype=torch.int64, device=DEV), torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    slot[:m] = order[t // page] * page + t % page
    position[:m] = (t + case["ctx"]).to(torch.int32)
    i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=DEV)
    return {"qkv": torch.randn((rows, (h + 2 * kv) * d), generator=g, device=DEV) * 2.0, "slot": slot, "position": position,
            "inv_freq": 1e6 ** (-2.0 * i / case["rot"]),
            "q_weight": torch.rand((d,), generator=g, device=DEV) + 0.5 if case["norm"] else None,
            "k_weight": torch.rand((d,), generator=g, device=DEV) + 0.5 if case["norm"] else None,
            "k_cache": torch.zeros((pages, kv, page, d), dtype=torch.float16, device=DEV),
            "v_cache": torch.zeros((pages, kv, page, d), dtype=torch.float16, device=DEV)}


def _attention_inputs(case, seed):
    g, r, h, kv, d, page = _gen(seed), case["r"], case["heads"], case["kv"], case["d"], case["page"]
    lengths, added = _lengths(case)
    rows = sum(added) + case["pad"]
    used = [-(-(a + b) // page) for a, b in zip(lengths, added)]
    pages, width = sum(used) + 1, max(used) + 1
    table = torch.full((r, width), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(width, device=DEV) < _i32(used)[:, None]] = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)[: sum(used)]
    start = _i32(_starts(added))
    ancestors = None
    if case["tree"]:
        ancestors = torch.zeros((rows,), dtype=torch.int64, device=DEV)
        bits = _bits(_reach(_parents(g, added, rows), start.long(), r))
        ancestors[: sum(added)] = bits[torch.arange(TREE, device=DEV) < _i32(added)[:, None]]
    # normed heads; queries wide enough for scores with a few tokens that matter
    return {"q": (torch.randn((rows, h, d), generator=g, device=DEV) * 2.0).to(torch.float16),
            "k_cache": torch.randn((pages, kv, page, d), generator=g, device=DEV, dtype=torch.float16),
            "v_cache": torch.randn((pages, kv, page, d), generator=g, device=DEV, dtype=torch.float16),
            "table": table, "lengths": _i32(lengths), "row_start": start, "ancestors": ancestors}


def _logits_inputs(case, seed):
    g, r, n, new, hist = _gen(seed), case["r"], case["n"], case["new"], case["history"]
    m = r * new
    start = torch.arange(r + 1, device=DEV) * new
    # tokens repeat as words do: the square of a uniform number prefers low ids
    def words(*shape):
        return (torch.rand(shape, generator=g, device=DEV).pow(4) * n).to(torch.int32).clamp_(max=n - 1)

    parents = _parents(g, [new] * r, m)
    bits = _bits(_reach(parents, start, r))[:, :new].reshape(-1)
    length = torch.randint(hist // 2, hist + 1, (r,), generator=g, device=DEV, dtype=torch.int32)
    nb = case["bias"]
    bias_start = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.randint(0, nb + 1, (r,), generator=g, device=DEV).cumsum(0)]) if nb else None
    out = {"logits": torch.randn((m, n), generator=g, device=DEV) * 3.0,
           "request": torch.arange(m, device=DEV, dtype=torch.int32) // new, "tokens": words(r, max(1, hist)),
           "prompt_length": length // 3, "length": length,
           "repetition": 1.0 + torch.rand((r,), generator=g, device=DEV) * 0.3, "frequency": torch.rand((r,), generator=g, device=DEV) * 0.5,
           "presence": torch.rand((r,), generator=g, device=DEV) * 0.5,
           "drafts": words(m) if new > 1 else None, "row_start": start.to(torch.int32) if new > 1 else None,
           "ancestors": bits if new > 1 else None,
           "bias_start": None if bias_start is None else bias_start.to(torch.int32), "bias_token": None, "bias_value": None,
           "grammar": None, "grammar_row": None}
    if nb:
        # as long as every request's list could be; the starts say what is used
        out["bias_token"] = words(r * nb)
        out["bias_value"] = torch.randn((r * nb,), generator=g, device=DEV) * 4.0
    if case["grammar"]:
        # two grammar states: one that allows a few tokens, one that forbids a few; every third row has none
        words32 = (n + 31) // 32
        few = torch.randint(-2 ** 31, 2 ** 31, (3, words32), generator=g, device=DEV).to(torch.int32)
        out["grammar"] = torch.stack([few[0] & few[1] & few[2], few[0] | few[1] | few[2]])
        out["grammar_row"] = (torch.arange(m, device=DEV) % 3 - 1).to(torch.int32)
    return out


def _inputs(case, seed):
    return {"plan": _plan_inputs, "rotary": _rotary_inputs, "attention": _attention_inputs, "logits": _logits_inputs}[case["op"]](case, seed)


def prepare(case, seed):
    s, op = _inputs(case, seed), case["op"]
    # output buffers and workspaces that a serving loop keeps from step to step
    if op == "plan":
        m, r = s["rows"], case["r"]
        s["row_start"] = torch.empty((r + 1,), dtype=torch.int32, device=DEV)
        s["request"], s["position"] = (torch.empty((m,), dtype=torch.int32, device=DEV) for _ in range(2))
        s["slot"] = torch.empty((m,), dtype=torch.int64, device=DEV)
        s["ancestors"] = torch.empty((m,), dtype=torch.int64, device=DEV) if case["tree"] else None
        s["free_left"] = torch.empty((1,), dtype=torch.int32, device=DEV)
        s["page"] = case["page"]
    elif op == "rotary":
        s["q"] = torch.zeros((s["qkv"].shape[0], case["heads"], case["d"]), dtype=torch.float16, device=DEV)
        s["inter"] = case["inter"]
    elif op == "attention":
        s["out"] = torch.zeros_like(s["q"])
        s["workspace"] = torch.empty((256 << 20,), dtype=torch.uint8, device=DEV)
        s["added"] = s["row_start"][1:] - s["row_start"][:-1]
        s["most"] = case["new"]
        s["longest"] = case["ctx"] + case["new"]
    else:
        m = s["logits"].shape[0]
        s["out"] = torch.empty_like(s["logits"])
        s["token"], s["top"] = torch.empty((m,), dtype=torch.int32, device=DEV), torch.empty((m,), device=DEV)
        # room for a candidate of every 1,024 tokens of every row
        s["workspace"] = torch.empty((m * ((s["logits"].shape[1] + 1023) // 1024),), dtype=torch.int64, device=DEV)
    s["op"] = op
    return s


# ---- one pass --------------------------------------------------------------


def run(s):
    if own:
        return _own(s)
    return {"plan": _plan, "rotary": _rotary, "attention": _attention, "logits": _logits}[s["op"]](s)


def _own(s):
    import packed_bit_gemv_amd as pbg

    if s["op"] == "plan":
        pbg.cache_plan(s["lengths"], s["added"], s["table"], s["free_pages"], s["free_count"], s["page"], s["pages"],
                       s["row_start"], s["request"], s["position"], s["slot"], s["free_left"], s["parents"], s["ancestors"])
        return {x: s[x] for x in ("row_start", "request", "position", "slot", "ancestors", "free_left", "table")}
    if s["op"] == "rotary":
        pbg.rotary_qkv(s["qkv"], s["position"], s["slot"], s["inv_freq"], s["k_cache"], s["v_cache"], s["q_weight"], s["k_weight"], EPS,
                       interleaved=s["inter"], q=s["q"])
        return {x: s[x] for x in ("q", "k_cache", "v_cache")}
    if s["op"] == "attention":
        return pbg.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["row_start"], s["ancestors"],
                                  out=s["out"], workspace=s["workspace"])
    pbg.penalize_logits(s["logits"], s["request"], s["tokens"], s["prompt_length"], s["length"], s["repetition"], s["frequency"],
                        s["presence"], drafts=s["drafts"], row_start=s["row_start"], ancestors=s["ancestors"],
                        bias_start=s["bias_start"], bias_token=s["bias_token"], bias_value=s["bias_value"], grammar=s["grammar"],
                        grammar_row=s["grammar_row"], out=s["out"], token=s["token"], top=s["top"], workspace=s["workspace"])
    return {x: s[x] for x in ("out", "token", "top")}


def _plan(s):
    page, m, table = s["page"], s["rows"], s["table"]
    r, width = table.shape
    length, added = s["lengths"].long().clamp(min=0), s["added"].long().clamp(min=0)
    start = torch.nn.functional.pad(added.cumsum(0), (1, 0)).clamp(max=m)
    n = start[1:] - start[:-1]
    have = (length + page - 1) // page
    need = (((length + n + page - 1) // page).clamp(max=width) - have).clamp(min=0)
    first = need.cumsum(0) - need
    row = torch.arange(m, device=DEV)
    live = row < start[-1]
    q = torch.searchsorted(start[1:].contiguous(), row, right=True).clamp(max=r - 1)
    c = row - start[q]
    t = length[q] + c
    p = t // page
    count = s["free_count"].long().clamp(0, s["free_pages"].numel())
    at = count - 1 - (first[q] + p - have[q])
    taken = torch.where(at >= 0, s["free_pages"].long()[at.clamp(0, s["free_pages"].numel() - 1)], -1)
    taken = torch.where((taken >= 0) & (taken < s["pages"]), taken, -1)
    held = table.long()[q, p.clamp(max=width - 1)]
    number = torch.where(p < have[q], held, taken)
    fine = live & (p < width) & (number >= 0) & (number < s["pages"])
    opens = live & (t % page == 0) & (p < width)
    # every page of the step is opened by one row, the others write to a place behind the table
    flat = torch.nn.functional.pad(table.view(-1), (0, 1))
    flat = flat.scatter(0, torch.where(opens, q * width + p, r * width), number.to(torch.int32))
    depth, ancestors = c, None
    if s["parents"] is not None:
        reach = _reach(s["parents"], start, r)
        tree = live & (c < TREE)
        mine = reach[q, c.clamp(max=TREE - 1)]
        depth = mine.sum(-1) - 1
        fine, live_position = fine & tree, tree
        ancestors = torch.where(tree, _bits(mine), 0)
    else:
        live_position = live
    return {"row_start": start.to(torch.int32), "request": torch.where(live, q, -1).to(torch.int32),
            "position": torch.where(live_position, length[q] + depth, -1).to(torch.int32),
            "slot": torch.where(fine, number * page + t % page, -1), "ancestors": ancestors,
            "free_left": (count - need.sum()).clamp(min=0).to(torch.int32), "table": flat[:-1].view(r, width)}


def _normed(x, weight):
    return x if weight is None else x * weight / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)


def _turned(x, cos, sin, inter):
    half = cos.shape[-1]
    if inter:
        a, b = x[..., 0: 2 * half: 2], x[..., 1: 2 * half: 2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half: 2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _rotary(s):
    pages, kv, page, d = s["k_cache"].shape
    rows, heads = s["q"].shape[:2]
    angle = s["position"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = s["qkv"].view(rows, heads + 2 * kv, d)
    q = _turned(_normed(x[:, :heads], s["q_weight"]), cos, sin, s["inter"]).to(torch.float16)
    k = _turned(_normed(x[:, heads: heads + kv], s["k_weight"]), cos, sin, s["inter"]).to(torch.float16)
    live = s["position"] >= 0
    # rows without a slot write to a page behind the cache
    slot = torch.where(live & (s["slot"] >= 0), s["slot"], pages * page)
    out = {"q": torch.where(live[:, None, None], q, s["q"])}
    for name, y in (("k_cache", k), ("v_cache", x[:, heads + kv:].to(torch.float16))):
        longer = torch.nn.functional.pad(s[name], (0, 0, 0, 0, 0, 0, 0, 1))
        longer[slot // page, :, slot % page] = y
        out[name] = longer[:-1]
    return out


def _attention(s):
    rows, heads, d = s["q"].shape
    kv, page = s["k_cache"].shape[1:3]
    r, most, longest = s["lengths"].numel(), s["most"], s["longest"]
    start, length, added = s["row_start"].long(), s["lengths"].long(), s["added"].long()
    wide = -(-longest // page)
    table = s["table"][:, :wide].long().clamp(min=0)
    keys, values = (s[x][table].transpose(1, 2).reshape(r, kv, wide * page, d).float() for x in ("k_cache", "v_cache"))
    c = torch.arange(most, device=DEV)
    mine = c < added[:, None]
    row = (start[:-1, None] + c).clamp(max=rows - 1)
    q = s["q"][row].float().view(r, most, kv, heads // kv, d).permute(0, 2, 3, 1, 4).reshape(r, kv, -1, d)
    score = torch.matmul(q, keys.transpose(2, 3).contiguous()).view(r, kv, heads // kv, most, -1) * (1.0 / math.sqrt(d))
    t = torch.arange(wide * page, device=DEV)
    new = t - length[:, None]
    if s["ancestors"] is None:
        sees = new[:, None] <= c[:, None]
    else:
        bit = (s["ancestors"][row][:, :, None] >> new.clamp(0, 63)[:, None]) & 1
        sees = (new < 0)[:, None] | ((new < TREE)[:, None] & (bit > 0))
    sees = (sees & (t < (length + added)[:, None])[:, None])[:, None, None]
    score = score.masked_fill_(~sees, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score.sub_(torch.where(top > -math.inf, top, 0.0)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(r, kv, -1, wide * page), values).view(r, kv, heads // kv, most, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(r, most, heads, d).to(torch.float16)
    s["out"][row[mine]] = o[mine]
    return s["out"]


def _counted(tokens, used, n):
    """[m, n]: how often a row's tokens hold each token, of those that are used."""
    fine = used & (tokens >= 0) & (tokens < n)
    count = torch.zeros((tokens.shape[0], n), device=DEV)
    return count.scatter_add_(1, tokens.long().clamp(0, n - 1), fine.float())


def _logits(s):
    x, q = s["logits"], s["request"].long()
    m, n = x.shape
    at = torch.arange(s["tokens"].shape[1], device=DEV)
    length, prompt = s["length"][q][:, None], s["prompt_length"][q][:, None]
    tokens = s["tokens"][q]
    given = _counted(tokens, (at < prompt) & (at < length), n)
    count = _counted(tokens, (at >= prompt) & (at < length), n)
    if s["drafts"] is not None:
        c = torch.arange(TREE, device=DEV)
        row = (s["row_start"].long()[q][:, None] + c).clamp(max=m - 1)
        count += _counted(s["drafts"][row], (s["ancestors"][:, None] >> c) & 1 > 0, n)
    repetition, frequency, presence = (s[p][q][:, None] for p in ("repetition", "frequency", "presence"))
    x = torch.where(given + count > 0, torch.where(x > 0, x / repetition, x * repetition), x)
    x = torch.where(count > 0, x - frequency * count - presence, x)
    if s["bias_start"] is not None:
        # where a list names a token twice its last value counts
        r, entries = s["tokens"].shape[0], torch.arange(s["bias_token"].numel(), device=DEV)
        whose = torch.searchsorted(s["bias_start"][1:].long().contiguous(), entries, right=True)
        last = torch.full(((r + 1) * n,), -1, dtype=torch.int64, device=DEV)
        last = last.scatter_reduce_(0, whose * n + s["bias_token"].long(), entries, "amax").view(r + 1, n)[q]
        x = torch.where(last >= 0, x + s["bias_value"][last.clamp(min=0)], x)
    if s["grammar"] is not None:
        v = torch.arange(n, device=DEV)
        state = s["grammar_row"].long()[:, None]
        allowed = (s["grammar"][state.clamp(min=0), v // 32] >> (v % 32)) & 1 > 0
        x = torch.where(allowed | (state < 0), x, -math.inf)
    top, token = x.amax(1), x.argmax(1)
    return {"out": x, "token": torch.where(top > -math.inf, token, -1).to(torch.int32), "top": top}


# ---- what a pass cannot do without -----------------------------------------


def work(case):
    op = case["op"]
    if op in ("plan", "attention"):
        lengths, added = _lengths(case)
        r, m = case["r"], sum(added)
    if op == "plan":
        page, rows = case["page"], m + case["pad"]
        pages = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(lengths, added))
        each = 4 + 4 + 8 + (12 if case["tree"] else 0)
        return {"bytes": 8 * r + 4 * (r + 1) + rows * each + 8 * pages + 4 * r + 8, "flops": 4 * rows}
    if op == "rotary":
        n = (case["heads"] + 2 * case["kv"]) * case["d"]
        turned = (case["heads"] + case["kv"]) * (3 * case["rot"] + (4 * case["d"] if case["norm"] else 0))
        return {"bytes": case["m"] * (6 * n + 12) + 4 * case["rot"], "flops": case["m"] * turned}
    if op == "attention":
        h, kv, d = case["heads"], case["kv"], case["d"]
        held = sum(a + b for a, b in zip(lengths, added))
        # of a tree a row sees its ancestors: about the logarithm of its size, counted as one token
        pairs = sum(a * b + (b if case["tree"] else b * (b + 1) // 2) for a, b in zip(lengths, added))
        return {"bytes": 4 * m * h * d + 4 * held * kv * d + (8 * m if case["tree"] else 0) + 4 * held // case["page"] + 8 * r,
                "flops": 4 * pairs * h * d}
    m, n = case["r"] * case["new"], case["n"]
    return {"bytes": 8 * m * n + 4 * case["r"] * (case["history"] * 3 // 4 + case["bias"]) + (n // 4 if case["grammar"] else 0) + 20 * m,
            "flops": 2 * m * n}


# ---- the same from the definitions in 64 bits -------------------------------


def exact(case, seed):
    i, op = _inputs(case, seed), case["op"]
    if op == "plan":
        return None
    if op == "rotary":
        rows, h, kv, d, rot, m, page = i["qkv"].shape[0], case["heads"], case["kv"], case["d"], case["rot"], case["m"], case["page"]
        x = i["qkv"].double().view(rows, h + 2 * kv, d)[:m]
        heads = x[:, : h + kv].clone()
        if case["norm"]:
            heads /= (heads.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
            heads[:, :h] *= i["q_weight"].double()
            heads[:, h:] *= i["k_weight"].double()
        turn = torch.polar(torch.ones((m, rot // 2), dtype=torch.float64, device=DEV), i["position"][:m].double()[:, None] * i["inv_freq"])
        even, odd = (slice(0, rot, 2), slice(1, rot, 2)) if case["inter"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(heads[..., even].contiguous(), heads[..., odd].contiguous()) * turn[:, None]
        heads[..., even], heads[..., odd] = z.real, z.imag
        out = {"q": torch.zeros((rows, h, d), dtype=torch.float64, device=DEV)}
        out["q"][:m] = heads[:, :h]
        for name, y in (("k_cache", heads[:, h:]), ("v_cache", x[:, h + kv:])):
            cache = torch.zeros(i[name].shape, dtype=torch.float64, device=DEV)
            cache[i["slot"][:m] // page, :, i["slot"][:m] % page] = y
            out[name] = cache
        return out
    if op == "attention":
        lengths, added = _lengths(case)
        h, kv, d, page = case["heads"], case["kv"], case["d"], case["page"]
        out, first = torch.zeros(i["q"].shape, dtype=torch.float64, device=DEV), 0
        for j, (a, b) in enumerate(zip(lengths, added)):
            t = torch.arange(a + b, device=DEV)
            at = i["table"][j].long()[t // page]
            late = t[a:] - a
            if i["ancestors"] is None:
                sees = late <= torch.arange(b, device=DEV)[:, None]
            else:
                sees = (i["ancestors"][first: first + b, None] >> late) & 1 == 1
            sees = torch.cat([torch.ones((b, a), dtype=torch.bool, device=DEV), sees], 1)
            for g in range(kv):
                k, v = i["k_cache"][at, g, t % page].double(), i["v_cache"][at, g, t % page].double()
                k = k.t().contiguous()
                for e in range(g * (h // kv), (g + 1) * (h // kv)):
                    score = torch.mm(i["q"][first: first + b, e].double(), k) / math.sqrt(d)
                    w = torch.softmax(score.masked_fill(~sees, -math.inf), 1)
                    out[first: first + b, e] = torch.mm(w, v)
            first += b
        return out
    x = i["logits"].double()
    m, n = x.shape
    for j in range(m):
        q = j // case["new"]
        said = i["tokens"][q, : int(i["length"][q])].long()
        before = int(i["prompt_length"][q])
        drafted = said[:0]
        if i["drafts"] is not None:
            mine = i["drafts"][q * case["new"]: (q + 1) * case["new"]].long()
            drafted = mine[(i["ancestors"][j] >> torch.arange(case["new"], device=DEV)) & 1 == 1]
        output = torch.cat([said[before:], drafted])
        every = torch.cat([said, drafted]).unique()
        x[j, every] *= torch.where(x[j, every] > 0, 1.0 / i["repetition"][q].double(), i["repetition"][q].double())
        x[j] -= i["frequency"][q].double() * torch.bincount(output, minlength=n)
        x[j, output.unique()] -= i["presence"][q].double()
        if i["bias_start"] is not None:
            a, b = int(i["bias_start"][q]), int(i["bias_start"][q + 1])
            for token, value in dict(zip(i["bias_token"][a:b].tolist(), i["bias_value"][a:b].tolist())).items():
                x[j, token] += value
        if i["grammar"] is not None and int(i["grammar_row"][j]) >= 0:
            word = i["grammar"][int(i["grammar_row"][j])].long()
            bit = (word[:, None] >> torch.arange(32, device=DEV)).flatten()[:n] & 1
            x[j, bit == 0] = -math.inf
    return {"out": x, "token": None, "top": x.max(1).values}
