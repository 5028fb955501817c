"""The attention half of a step and penalize_logits without a GPU: argument
checks of the C entry points and of the binding, frequencies, and the oracle's
pins."""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle
from packed_bit_gemv_amd import binding
from test_abi import GOOD, _gpu_visible, no_gpu_only  # noqa: F401 (the marker evaluates _gpu_visible here)


def lib():
    return binding.lib()


def call(name, args, **kw):
    a = {**args, **kw}
    return getattr(lib(), name)(*a.values(), None)


def refusals(name, args, needed, optional, aligned, shapes, values=()):
    """Every needed pointer is required, every pointer's alignment and every size and value is checked."""
    for p in needed:
        assert call(name, args, **{p: None}) == -1, p
    for p in (*needed, *optional):
        for off in (1, 2, 4, 8):
            if off < aligned.get(p, 4):
                assert call(name, args, **{p: GOOD + off}) == -3, (p, off)
    for p, v in shapes:
        assert call(name, args, **{p: v}) == -2, (p, v)
    for p, v in values:
        assert call(name, args, **{p: v}) == -7, (p, v)


PLAN = dict(lengths=GOOD, added=GOOD, requests=3, table=GOOD, table_width=8, free_pages=GOOD, free_capacity=9, free_count=GOOD, pages=40,
            page_size=16, parents=GOOD, m=7, row_start=GOOD, request=GOOD, position=GOOD, slot=GOOD, ancestors=GOOD, free_left=GOOD + 64)


@no_gpu_only
def test_cache_plan_refusals():
    refusals("cache_plan", PLAN, [p for p in PLAN if PLAN[p] in (GOOD, GOOD + 64) and p not in ("parents", "ancestors")], ["parents", "ancestors"],
             dict(slot=8, ancestors=8),
             [("requests", 0), ("requests", 4097), ("table_width", 0), ("table_width", 2 ** 27), ("free_capacity", 0), ("pages", 0),
              ("pages", 2 ** 31), ("page_size", 0), ("page_size", 3), ("page_size", 8192), ("page_size", -16), ("m", 0), ("m", 2 ** 20 + 1)],
             [("free_left", GOOD)])


ROTARY = dict(qkv=GOOD, position=GOOD, slot=GOOD, inv_freq=GOOD, q_weight=GOOD, k_weight=GOOD, eps=1e-6, amplitude=1.0, interleaved=0, m=2,
              heads=4, kv_heads=2, head_dim=64, rotary_dim=64, q=GOOD, k_cache=GOOD, v_cache=GOOD, pages=4, page_size=16)


@no_gpu_only
def test_rotary_refusals():
    refusals("rotary_qkv", ROTARY, ["qkv", "position", "slot", "inv_freq", "q", "k_cache", "v_cache"], ["q_weight", "k_weight"],
             dict(slot=8, inv_freq=8, q=16, k_cache=16, v_cache=16),
             [("m", 0), ("m", 2 ** 20 + 1), ("heads", 0), ("heads", 5), ("heads", 1026), ("kv_heads", 0), ("kv_heads", -2), ("kv_heads", 3),
              ("head_dim", 0), ("head_dim", 60), ("head_dim", 264), ("rotary_dim", 72), ("rotary_dim", 12), ("rotary_dim", -8), ("pages", 0),
              ("page_size", 12)],
             [("eps", 0.0), ("eps", math.nan), ("eps", math.inf), ("amplitude", math.nan), ("amplitude", -math.inf)])
    assert call("rotary_qkv", ROTARY, rotary_dim=0) == -1
    assert call("rotary_qkv", ROTARY, m=2 ** 20, heads=64, kv_heads=32) == -2


ATTENTION = dict(q=GOOD, k_cache=GOOD, v_cache=GOOD, pages=4, page_size=16, table=GOOD, table_width=4, lengths=GOOD, row_start=GOOD, requests=2,
                 ancestors=GOOD, m=5, heads=4, kv_heads=2, head_dim=64, scale=0.125, out=GOOD, workspace=GOOD, workspace_bytes=1 << 30)


@no_gpu_only
def test_attention_refusals():
    refusals("tree_attention", ATTENTION, ["q", "k_cache", "v_cache", "table", "lengths", "row_start", "out", "workspace"], ["ancestors"],
             dict(q=16, k_cache=16, v_cache=16, ancestors=8, out=16, workspace=16),
             [("m", 0), ("m", 2 ** 20 + 1), ("requests", 0), ("requests", 4097), ("heads", 3), ("heads", 1026), ("kv_heads", 0),
              ("head_dim", 4), ("head_dim", 65), ("head_dim", 512), ("pages", 0), ("page_size", 48), ("page_size", 4), ("table_width", 0),
              ("table_width", 2 ** 28)],
             [("scale", 0.0), ("scale", -1.0), ("scale", math.nan), ("scale", math.inf), ("scale", 3e38)])
    size = lib().pbg_attention_workspace_bytes(4, 2, 64)
    assert size > 0 and call("tree_attention", ATTENTION, workspace_bytes=size - 1) == -6


def test_attention_workspace_bytes():
    """Nothing for heads that are refused; more for wider heads."""
    f = lib().pbg_attention_workspace_bytes
    assert f(0, 1, 64) == 0 and f(4, 3, 64) == 0 and f(4, 4, 60) == 0 and f(4, 4, 264) == 0
    sizes = [f(32, 8, d) for d in range(8, 257, 8)]
    assert all(0 < a <= b < 256 << 20 for a, b in zip(sizes, sizes[1:]))


LOGITS = dict(logits=GOOD, request=GOOD, tokens=GOOD, tokens_width=9, prompt_length=GOOD, length=GOOD, repetition=GOOD, frequency=GOOD,
              presence=GOOD, requests=2, drafts=GOOD, row_start=GOOD, ancestors=GOOD, bias_start=GOOD, bias_token=GOOD, bias_value=GOOD,
              bias_entries=3, grammar=GOOD, grammar_row=GOOD, states=2, m=4, n=2000, out=GOOD, token=GOOD, top=GOOD, workspace=GOOD,
              workspace_bytes=64)


@no_gpu_only
def test_logits_refusals():
    pointers = [p for p in LOGITS if LOGITS[p] == GOOD]
    refusals("penalize_logits", LOGITS, pointers, [], dict(ancestors=8, workspace=8),
             [("m", 0), ("m", 2 ** 20 + 1), ("n", 0), ("n", 2 ** 24 + 1), ("n", 2 ** 31), ("requests", 0), ("requests", 4097), ("tokens_width", 0),
              ("tokens_width", 2 ** 24 + 1), ("bias_entries", 0), ("bias_entries", 2 ** 31), ("states", 0), ("states", 2 ** 31)])
    assert call("penalize_logits", LOGITS, workspace_bytes=63) == -6
    assert call("penalize_logits", LOGITS, m=2 ** 20, n=2 ** 13) == -2


def test_binding_rejects_cpu_tensors():
    import torch

    f32, f16, i32, i64 = torch.float32, torch.float16, torch.int32, torch.int64
    z = lambda dt, *s: torch.zeros(s, dtype=dt)  # noqa: E731
    cache = z(f16, 2, 1, 16, 64)
    for f in (lambda: binding.cache_plan(z(i32, 2), z(i32, 2), z(i32, 2, 4), z(i32, 5), z(i32, 1), 16, 9, rows=3),
              lambda: binding.cache_plan(None, None, None, None, None, 16, 9, rows=3),
              lambda: binding.rotary_qkv(z(f32, 2, 256), z(i32, 2), z(i64, 2), z(torch.float64, 32), cache, cache),
              lambda: binding.tree_attention(z(f16, 2, 2, 64), cache, cache, z(i32, 1, 2), z(i32, 1), z(i32, 2)),
              lambda: binding.tree_attention(z(f16, 2, 2, 64), None, cache, z(i32, 1, 2), z(i32, 1), z(i32, 2)),
              lambda: binding.penalize_logits(z(f32, 2, 9), z(i32, 2), z(i32, 1, 4), z(i32, 1), z(i32, 1), z(f32, 1), z(f32, 1), z(f32, 1))):
        with pytest.raises(ValueError):
            f()


def test_rotary_frequencies():
    f, a = binding.rotary_frequencies(8, 10000.0, device="cpu")
    assert a == 1.0 and np.allclose(f.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-14)
    assert np.allclose(binding.rotary_frequencies(8, 10000.0, "linear", 4.0, device="cpu")[0].numpy(), f.numpy() / 4, rtol=1e-14)
    g, a = binding.rotary_frequencies(128, 1e6, "ntk", 4.0, device="cpu")
    base = binding.rotary_frequencies(128, 1e6, device="cpu")[0].numpy()
    assert a == 1.0 and g[0] == 1.0 and np.isclose(float(g[-1]), base[-1] / 4, rtol=1e-12) and (np.diff(g.numpy() / base) <= 0).all()
    y, a = binding.rotary_frequencies(128, 1e6, "yarn", 4.0, 32768, device="cpu")
    ratio, turns = y.numpy() / base, base * 32768 / (2 * math.pi)
    assert np.isclose(a, 1 + 0.1 * math.log(4.0)) and (np.diff(ratio) <= 1e-15).all()
    # a pair off the ramp's ends by the rounding of its number at most
    step = base[0] / base[1]
    assert np.allclose(ratio[turns > 32 * step], 1.0) and np.allclose(ratio[turns < 1 / step], 0.25)
    assert len(binding.rotary_frequencies(0, device="cpu")[0]) == 0
    for bad in (dict(rotary_dim=7), dict(rotary_dim=8, factor=0.5), dict(rotary_dim=8, scaling="other")):
        with pytest.raises(ValueError):
            binding.rotary_frequencies(**bad, device="cpu")


def test_oracle_plan():
    """A worked step: pages of 4, one request in the middle of a page, one that opens two, one that waits, a tree."""
    table = np.full((3, 4), -1, np.int32)
    table[0, :2] = [5, 2]
    table[2, :1] = [7]
    start, request, position, slot, anc, left, out = oracle.cache_plan(
        np.array([6, 0, 3]), np.array([1, 5, 0]), table, np.array([9, 8, 4, 3]), 3, 4, 10, 8)
    assert start.tolist() == [0, 1, 6, 6] and request.tolist() == [0, 1, 1, 1, 1, 1, -1, -1]
    assert position.tolist() == [6, 0, 1, 2, 3, 4, -1, -1]
    assert slot.tolist() == [2 * 4 + 2, 16, 17, 18, 19, 32, -1, -1] and left == 1
    assert out[1].tolist() == [4, 8, -1, -1] and out[0].tolist() == [5, 2, -1, -1]
    assert [int(a) for a in anc[:6]] == [1, 1, 3, 7, 15, 31]
    _, _, position, _, anc, _, _ = oracle.cache_plan(np.array([6]), np.array([5]), table[:1], np.array([9, 8]), 2, 4, 10, 5,
                                                     np.array([-1, 0, 0, 2, 9]))
    assert position.tolist() == [6, 7, 7, 8, 6] and [int(a) for a in anc] == [1, 0b11, 0b101, 0b1101, 0b10000]


def test_oracle_rotary():
    """A turn keeps lengths; scores depend on the distance of positions only; both layouts are the same turn of permuted elements."""
    rng = np.random.default_rng(1)
    d, freq = 16, 1e4 ** (-np.arange(8) / 8)
    x = np.repeat(rng.standard_normal((1, 3 * d)), 6, 0).astype(np.float32)
    q, k, v = oracle.rotary_qkv(x, np.array([0, 1, 5, 100, 101, 105]), freq, 1, 1, d)
    assert np.allclose((q ** 2).sum(-1), (x[:, None, :d].astype(np.float64) ** 2).sum(-1)) and np.array_equal(v[:, 0], x[:, 2 * d:].astype(np.float64))
    s = q[:, 0] @ k[:, 0].T
    assert np.isclose(s[1, 0], s[4, 3]) and np.isclose(s[2, 1], s[5, 4]) and np.allclose(q[0, 0], x[0, :d])
    order = np.arange(d).reshape(2, 8).T.reshape(-1)
    y = x.reshape(6, 3, d)[:, :, order].reshape(6, -1)
    qi, _, _ = oracle.rotary_qkv(y, np.array([0, 1, 5, 100, 101, 105]), freq, 1, 1, d, interleaved=True)
    assert np.allclose(qi[:, 0], q[:, 0][:, order])
    qn, _, _ = oracle.rotary_qkv(x, np.zeros(6), None, 1, 1, d, q_weight=np.full(d, 2, np.float32), eps=0.5)
    mean = (x[0, :d].astype(np.float64) ** 2).mean()
    assert np.allclose(qn[0, 0], 2 * x[0, :d] / math.sqrt(mean + 0.5))


def test_oracle_attention():
    """One token returns its value; equal scores average; a mask leaves its tokens out; an empty row is zero."""
    rng = np.random.default_rng(2)
    k, v = np.zeros((3, 1, 4, 8), np.float16), rng.standard_normal((3, 1, 4, 8)).astype(np.float16)
    q = rng.standard_normal((3, 2, 8)).astype(np.float16)
    c = dict(q=q, k_cache=k, v_cache=v, table=np.array([[2, 0]], np.int32), lengths=np.array([3], np.int32), row_start=np.array([0, 3], np.int32))
    flat = np.concatenate([v[2, 0], v[0, 0]]).astype(np.float64)
    out, _, _ = oracle.tree_attention(**c)
    for a in range(3):
        assert np.allclose(out[a], flat[: 4 + a].mean(0))
    out, _, _ = oracle.tree_attention(**c, ancestors=np.array([0b1, 0b10, 0b101], np.uint64))
    assert np.allclose(out[1, 0], flat[[0, 1, 2, 4]].mean(0)) and np.allclose(out[2, 1], flat[[0, 1, 2, 3, 5]].mean(0))
    out, _, _ = oracle.tree_attention(**{**c, "lengths": np.array([0], np.int32)}, ancestors=np.array([0, 1, 0b10], np.uint64))
    assert (out[0] == 0).all() and np.allclose(out[1], flat[0]) and np.allclose(out[2], flat[1])


def test_oracle_logits():
    c = dict(logits=np.array([[1.0, -1.0, 2.0, 4.0, 0.5]], np.float32), request=np.array([0], np.int32), tokens=np.array([[0, 1, 3, 3, 9]], np.int32),
             prompt_length=np.array([2], np.int32), length=np.array([4], np.int32), repetition=np.array([2.0], np.float32),
             frequency=np.array([0.25], np.float32), presence=np.array([0.5], np.float32))
    out, token, top = oracle.penalize_logits(**c)
    assert out[0].tolist() == [0.5, -2.0, 2.0, 1.0, 0.5] and token[0] == 2 and top[0] == 2.0
    out, token, _ = oracle.penalize_logits(**c, bias_start=np.array([0, 3]), bias_token=np.array([4, 0, 4]), bias_value=np.array([9.0, 1.0, 1.0]),
                                           grammar=np.array([[0b10011]], np.uint32), grammar_row=np.array([0]))
    assert out[0].tolist() == [1.5, -2.0, -math.inf, -math.inf, 1.5] and token[0] == 0
