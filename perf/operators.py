"""The cases on which the 8-bit activation path and the adapters of packed_bit_gemv_amd are measured.

Five operators: add_rmsnorm (residual addition, root-mean-square norm, fp16 and 8-bit outputs), quantize_rows (fp16 rows to
8 bits with a scale per row), ternary_gemm_i8 (8-bit rows times a packed ternary matrix, any number of rows),
ternary_swiglu_gate_up_i8 (the gated half of a feed-forward block on 8-bit rows) and lora_add (adapters of many requests beside
a shared projection). Weight shapes are those of the decoder layer this library serves.

The 8-bit codes come back as whole numbers beside their scales: every step that leads to a code is one IEEE fp32 operation on
one element (the norm's factor cancels in it), so two implementations have equal codes.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TINY = 2.0 ** -100  # rows whose largest magnitude is below this have the codes 0 and the scale 0


def listed():
    return [
        # the norm in front of a linear, one decoded token: its latency is what counts
        {"name": "norm-token", "op": "norm", "m": 1, "k": 4096, "residual": True, "h": True, "q": False},
        # the same over a prompt, fp16 rows for the adapters and 8-bit rows for the shared linears
        {"name": "norm-prompt", "op": "norm", "m": 4096, "k": 4096, "residual": True, "h": True, "q": True},
        # attention outputs of a batch of sequences, a width that is no multiple of 64
        {"name": "quant-batch", "op": "quant", "m": 33, "k": 4100},
        # a prompt's gated feed-forward activations on their way into the down linear
        {"name": "quant-prompt", "op": "quant", "m": 2048, "k": 12288},
        # the q|k|v pack for one decoded token
        {"name": "linear-token", "op": "linear", "m": 1, "n": 6144, "k": 4096},
        # the down linear for the rows of a speculative verify step
        {"name": "linear-verify", "op": "linear", "m": 7, "n": 4096, "k": 12288},
        # a k or v projection for a batch of sequences
        {"name": "linear-batch", "op": "linear", "m": 100, "n": 1024, "k": 4096},
        # the down linear over a long prompt
        {"name": "linear-prompt", "op": "linear", "m": 4096, "n": 4096, "k": 12288},
        # gate and up for a verify step
        {"name": "gateup-verify", "op": "gateup", "m": 8, "n": 12288, "k": 4096},
        # gate and up over a prompt
        {"name": "gateup-prompt", "op": "gateup", "m": 2048, "n": 12288, "k": 4096},
        # one decoded token of each of 64 requests, 24 adapters loaded, some requests without one
        {"name": "lora-batch", "op": "lora", "m": 64, "n": 4096, "k": 4096, "rank": 16, "adapters": 24, "runs": False},
        # the prompts of a few requests back to back on the gate linear, an odd number of rows
        {"name": "lora-prompt", "op": "lora", "m": 1531, "n": 12288, "k": 4096, "rank": 64, "adapters": 3, "runs": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _rows(rng, hi, cost, most):
    """A number of rows up to hi whose work (rows times cost) stays within most."""
    return _log(rng, 1, max(1, min(hi, most // cost)))


def draw(rng):
    op = rng.choice(["norm", "quant", "linear", "gateup", "lora"])
    if op == "norm":
        k = _log(rng, 64, 8192)
        out = rng.choice([(True, False), (False, True), (True, True)])
        return {"op": op, "m": _rows(rng, 4096, k, 4096 * 4096), "k": k, "residual": rng.random() < 0.8, "h": out[0], "q": out[1]}
    if op == "quant":
        k = _log(rng, 64, 16384)
        return {"op": op, "m": _rows(rng, 4096, k, 2048 * 12288), "k": k}
    k, n = _log(rng, 64, 12288), _log(rng, 64, 12288)
    if op == "linear":
        return {"op": op, "m": _rows(rng, 4096, n * k, 4096 * 4096 * 12288), "n": n, "k": k}
    if op == "gateup":
        k = _log(rng, 64, 4096)
        return {"op": op, "m": _rows(rng, 2048, n * k, 2048 * 12288 * 4096), "n": n, "k": k}
    rank, adapters = rng.choice([4, 8, 12, 16, 32, 64]), _log(rng, 1, 64)
    m = _rows(rng, 1531, rank * (n + k) + 8 * n, 1531 * 64 * (12288 + 4096))
    return {"op": op, "m": m, "n": n, "k": k, "rank": rank, "adapters": adapters, "runs": rng.random() < 0.5}


# ---- inputs ----------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _codes(g, n, k):
    """Ternary codes with the published shares of zero, plus and minus."""
    u = torch.rand((n, k), generator=g, device=DEV)
    return (u < 0.1868).to(torch.int8) - (u >= 1.0 - 0.1869).to(torch.int8)


def _scales(g, n):
    return torch.rand((n,), generator=g, device=DEV) * 0.04 + 0.01


def _q8(g, m, k):
    """8-bit rows as a quantizer leaves them (about four standard deviations across the range) and their scales."""
    q = (torch.randn((m, k), generator=g, device=DEV) * 32.0).round_().clamp_(-127, 127).to(torch.int8)
    return q, torch.rand((m,), generator=g, device=DEV) * 0.03 + 0.01


def _inputs(case, seed):
    """The plain inputs of a case: everything later laid out, packed or padded."""
    g, op, m, k = _gen(seed), case["op"], case["m"], case["k"]
    if op == "norm":
        x = torch.randn((m, k), generator=g, device=DEV)
        # a residual stream: wider than a linear's output, with a few dominant channels
        res = torch.randn((m, k), generator=g, device=DEV) * 4.0 if case["residual"] else None
        if res is not None:
            res[:, :: max(1, k // 3)] *= 12.0
        return {"x": x, "residual": res, "weight": torch.rand((k,), generator=g, device=DEV) + 0.5}
    if op == "quant":
        return {"x": (torch.randn((m, k), generator=g, device=DEV) * 0.7).to(torch.float16)}
    n = case["n"]
    if op == "linear":
        q, qs = _q8(g, m, k)
        return {"q": q, "q_scale": qs, "codes": _codes(g, n, k), "scale": _scales(g, n)}
    if op == "gateup":
        q, qs = _q8(g, m, k)
        # scales that keep gate outputs of order one, where silu bends
        return {"q": q, "q_scale": qs * (2.0 / math.sqrt(k)), "gate": _codes(g, n, k), "up": _codes(g, n, k),
                "gate_scale": _scales(g, n), "up_scale": _scales(g, n)}
    r, na = case["rank"], case["adapters"]
    y = torch.randn((m, n), generator=g, device=DEV)
    x = torch.randn((m, k), generator=g, device=DEV).to(torch.float16)
    a = (torch.randn((na, r, k), generator=g, device=DEV) / math.sqrt(k)).to(torch.float16)
    b = (torch.randn((na, n, r), generator=g, device=DEV) / math.sqrt(r)).to(torch.float16)
    # -1: a request without an adapter
    ids = torch.randint(-1, na, (m,), generator=g, device=DEV, dtype=torch.int32)
    if case["runs"]:
        ids = ids.sort().values
    return {"y": y, "x": x, "ids": ids, "a": a, "b": b, "scale": torch.rand((na,), generator=g, device=DEV) + 0.5}


def _shifts():
    """Place of code j of a 16-code word: pair j // 2 from the top of half j % 2."""
    j = torch.arange(16, device=DEV, dtype=torch.int32)
    return 16 * (j % 2) + 14 - 2 * (j // 2)


def _pack(codes):
    """The library's packed words (2 bits a code, rows of whole 16-byte chunks) from codes [n, k]."""
    n, k = codes.shape
    words = 4 * ((k + 63) // 64)
    c = torch.zeros((n, words * 16), dtype=torch.int32, device=DEV)
    c[:, :k] = codes
    return ((c.view(n, words, 16) & 3) << _shifts()).sum(-1).to(torch.int32)


def _pad_rows(q):
    """8-bit rows as the library keeps them: padded with zeros to a multiple of 64 bytes."""
    m, k = q.shape
    out = torch.zeros((m, 64 * ((k + 63) // 64)), dtype=torch.int8, device=DEV)
    out[:, :k] = q
    return out


def prepare(case, seed):
    s, op, m, k = _inputs(case, seed), case["op"], case["m"], case["k"]
    n = case.get("n")
    kp = 64 * ((k + 63) // 64)
    # output buffers that a serving loop keeps from step to step
    if op == "norm":
        s["residual_out"] = torch.empty((m, k), device=DEV)
        s["h"] = torch.empty((m, k), device=DEV, dtype=torch.float16) if case["h"] else None
        s["q"] = torch.empty((m, kp), device=DEV, dtype=torch.int8) if case["q"] else None
        s["q_scale"] = torch.empty((m,), device=DEV) if case["q"] else None
    elif op == "quant":
        s["q"] = torch.empty((m, kp), device=DEV, dtype=torch.int8)
        s["q_scale"] = torch.empty((m,), device=DEV)
    elif op == "linear":
        s["packed"], s["q"] = _pack(s.pop("codes")), _pad_rows(s["q"])
        s["out"] = torch.empty((m, n), device=DEV)
    elif op == "gateup":
        s["gate"], s["up"], s["q"] = _pack(s["gate"]), _pack(s["up"]), _pad_rows(s["q"])
        s["out"] = torch.empty((m, n), device=DEV, dtype=torch.float16)
    else:
        s["out"] = torch.empty((m, n), device=DEV)
        # room for the products x A^T of every row, in fp32 and split over the columns where rows are few
        s["workspace"] = torch.zeros((m * case["rank"] * 16,), device=DEV)
    s["op"], s["k"] = op, k
    return s


# ---- one pass --------------------------------------------------------------


def run(s):
    if own:
        return _own(s)
    return {"norm": _norm, "quant": _quant, "linear": _linear, "gateup": _gateup, "lora": _lora}[s["op"]](s)


def _own(s):
    import packed_bit_gemv_amd as pbg

    op, k = s["op"], s["k"]
    if op == "norm":
        res, h, q, qs = pbg.add_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["residual_out"],
                                        h=s["h"], q=s["q"], q_scale=s["q_scale"])
        return {"residual": res, "h": h, "q": None if q is None else q[:, :k], "q_scale": qs}
    if op == "quant":
        q, qs = pbg.quantize_rows(s["x"], s["q"], s["q_scale"])
        return {"q": q[:, :k], "q_scale": qs}
    if op == "linear":
        return pbg.ternary_gemm_i8(s["packed"], s["scale"], k, s["q"], s["q_scale"], s["out"])
    if op == "gateup":
        return pbg.ternary_swiglu_gate_up_i8(s["gate"], s["gate_scale"], s["up"], s["up_scale"], k, s["q"], s["q_scale"],
                                             s["out"])
    return pbg.lora_add(s["y"], s["x"], s["ids"], s["a"], s["b"], s["scale"], s["out"], s["workspace"])


def _quantized(p):
    """Codes of fp32 rows p and the largest magnitude of each row (0 for a row of nothing)."""
    top = p.abs().amax(dim=1, keepdim=True)
    some = top >= TINY
    q = torch.where(some, torch.round(p * (127.0 / torch.where(some, top, torch.ones_like(top)))), torch.zeros_like(p))
    return q.to(torch.int8), torch.where(some, top, torch.zeros_like(top))


def _norm(s):
    r = s["x"] if s["residual"] is None else s["x"] + s["residual"]
    rms = torch.rsqrt((r * r).mean(dim=1, keepdim=True) + EPS)
    p = r * s["weight"]
    out = {"residual": r, "h": None, "q": None, "q_scale": None}
    if s["h"] is not None:
        out["h"] = (p * rms).to(torch.float16)
    if s["q"] is not None:
        out["q"], top = _quantized(p)
        out["q_scale"] = (top * rms / 127.0).squeeze(1)
    return out


def _quant(s):
    q, top = _quantized(s["x"].float())
    return {"q": q, "q_scale": (top / 127.0).squeeze(1)}


def _unpacked(packed, k):
    """Codes of packed words, as fp32 [n, k]."""
    f = (packed.unsqueeze(-1) >> _shifts()) & 3
    return (f - 4 * (f == 3)).view(packed.shape[0], -1)[:, :k].float()


def _product(packed, scale, k, q, q_scale):
    # whole numbers below 2^24: the fp32 product is exact
    return (q[:, :k].float() @ _unpacked(packed, k).t()) * q_scale.unsqueeze(1) * scale


def _linear(s):
    return _product(s["packed"], s["scale"], s["k"], s["q"], s["q_scale"])


def _gateup(s):
    g = _product(s["gate"], s["gate_scale"], s["k"], s["q"], s["q_scale"])
    u = _product(s["up"], s["up_scale"], s["k"], s["q"], s["q_scale"])
    return (g / (1.0 + torch.exp(-g)) * u).to(torch.float16)


def _lora(s):
    a, b = s["a"].float(), s["b"].float()
    na, r, k = a.shape
    m, n = s["y"].shape
    v = (s["x"].float() @ a.view(na * r, k).t()).view(m, na, r)
    mine = s["ids"].unsqueeze(1) == torch.arange(na, device=DEV, dtype=torch.int32)
    v = v * (mine * s["scale"]).unsqueeze(2)
    return s["y"] + v.view(m, na * r) @ b.permute(0, 2, 1).reshape(na * r, n)


# ---- what a pass cannot do without -----------------------------------------


def work(case):
    op, m, k, n = case["op"], case["m"], case["k"], case.get("n", 0)
    words = 4 * ((k + 63) // 64)
    if op == "norm":
        each = 4 + 4 + (4 if case["residual"] else 0) + (2 if case["h"] else 0) + (1 if case["q"] else 0)
        return {"bytes": m * k * each + 4 * k + (4 * m if case["q"] else 0), "flops": m * k * (4 + (1 if case["residual"] else 0))}
    if op == "quant":
        return {"bytes": 3 * m * k + 4 * m, "flops": 3 * m * k}
    if op == "linear":
        return {"bytes": n * (4 * words + 4) + m * (k + 4) + 4 * m * n, "flops": 2 * m * n * k}
    if op == "gateup":
        return {"bytes": 2 * n * (4 * words + 4) + m * (k + 4) + 2 * m * n, "flops": 4 * m * n * k}
    r, used = case["rank"], min(case["adapters"], m)
    return {"bytes": 2 * m * k + 8 * m * n + 4 * m + used * (2 * r * (n + k) + 4), "flops": 2 * m * r * (n + k)}


# ---- the same from the definitions in 64 bits -------------------------------


def exact(case, seed):
    i, op, k = _inputs(case, seed), case["op"], case["k"]
    if op == "norm":
        r = i["x"].double()
        if i["residual"] is not None:
            r = r + i["residual"].double()
        p = i["weight"].double() * r / (r.pow(2).sum(1, keepdim=True) / k + EPS).sqrt()
        return {"residual": r, "h": p if case["h"] else None, "q": None,
                "q_scale": p.abs().max(dim=1).values / 127 if case["q"] else None}
    if op == "quant":
        return {"q": None, "q_scale": i["x"].double().abs().max(dim=1).values / 127}
    if op in ("linear", "gateup"):
        q = i["q"].double() * i["q_scale"].double()[:, None]
        if op == "linear":
            return torch.mm(q, (i["codes"].double() * i["scale"].double()[:, None]).t().contiguous())
        g = torch.mm(q, (i["gate"].double() * i["gate_scale"].double()[:, None]).t().contiguous())
        u = torch.mm(q, (i["up"].double() * i["up_scale"].double()[:, None]).t().contiguous())
        return g * torch.sigmoid(g) * u
    out = i["y"].double()
    for t in range(case["adapters"]):
        rows = (i["ids"] == t).nonzero().squeeze(1)
        down = torch.mm(i["x"].double()[rows], i["a"][t].double().t().contiguous())
        out[rows] += i["scale"][t].double() * torch.mm(down, i["b"][t].double().t().contiguous())
    return out
