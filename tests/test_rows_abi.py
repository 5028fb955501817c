"""The 8-bit activation path and the adapters without a GPU: argument checks
of the C entry points and of the binding, and the oracle's pins."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
import synth
from packed_bit_gemv_amd import binding
from test_abi import GOOD, _gpu_visible, no_gpu_only  # noqa: F401 (the marker evaluates _gpu_visible here)


def lib():
    return binding.lib()


def test_row_bytes():
    for k, b in ((1, 64), (64, 64), (65, 128), (4096, 4096), (4100, 4160), (0, 0), (-3, 0)):
        assert lib().pbg_q8_row_bytes(k) == b == binding.q8_row_bytes(k)
    assert lib().pbg_strerror(-7) != b"unknown error code"


NORM = dict(x=GOOD, residual=GOOD, weight=GOOD, eps=1e-6, m=2, k=64, residual_out=GOOD, h=GOOD, q=GOOD, q_scale=GOOD)


def norm(**kw):
    a = {**NORM, **kw}
    return lib().add_rmsnorm(a["x"], a["residual"], a["weight"], a["eps"], a["m"], a["k"], a["residual_out"], a["h"],
                             a["q"], a["q_scale"], None)


@no_gpu_only
@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), -1), (dict(weight=None), -1), (dict(h=None, q=None, q_scale=None), -1), (dict(q=None), -1),
    (dict(q_scale=None), -1), (dict(m=0), -2), (dict(m=2 ** 20 + 1), -2), (dict(k=0), -2), (dict(k=2 ** 17 + 1), -2),
    (dict(x=GOOD + 2), -3), (dict(residual=GOOD + 1), -3), (dict(weight=GOOD + 2), -3), (dict(residual_out=GOOD + 2), -3),
    (dict(h=GOOD + 1), -3), (dict(q=GOOD + 8), -3), (dict(q_scale=GOOD + 2), -3), (dict(eps=0.0), -7),
    (dict(eps=-1.0), -7), (dict(eps=float("inf")), -7), (dict(eps=float("nan")), -7)])
def test_add_rmsnorm_refusals(kw, rc):
    assert norm(**kw) == rc


@no_gpu_only
def test_quantize_rows_refusals():
    f = lib().quantize_rows
    assert f(None, 1, 64, GOOD, GOOD, None) == -1 and f(GOOD, 1, 64, None, GOOD, None) == -1
    assert f(GOOD, 1, 64, GOOD, None, None) == -1
    for m, k in ((0, 64), (-1, 64), (2 ** 20 + 1, 64), (1, 0), (1, 2 ** 17 + 1)):
        assert f(GOOD, m, k, GOOD, GOOD, None) == -2
    assert f(GOOD + 1, 1, 64, GOOD, GOOD, None) == -3 and f(GOOD, 1, 64, GOOD + 4, GOOD, None) == -3
    assert f(GOOD, 1, 64, GOOD, GOOD + 2, None) == -3


@no_gpu_only
def test_gemm_i8_refusals():
    f, g = lib().ternary_gemm_i8, lib().ternary_swiglu_gate_up_i8
    for at in (0, 1, 4, 5, 7):
        args = [GOOD, GOOD, 4, 64, GOOD, GOOD, 3, GOOD]
        args[at] = None
        assert f(*args, None) == -1
    for n, k, m in ((0, 64, 1), (4, 0, 1), (4, 64, 0), (2 ** 24 + 1, 64, 1), (4, 2 ** 17 + 1, 1), (4, 64, 2 ** 20 + 1),
                    (2 ** 24, 64, 2 ** 13)):
        assert f(GOOD, GOOD, n, k, GOOD, GOOD, m, GOOD, None) == -2
        assert g(GOOD, GOOD, GOOD, GOOD, k, n, GOOD, GOOD, m, GOOD, None) == -2
    for at, off in ((0, 8), (1, 2), (4, 8), (5, 2), (7, 2)):
        args = [GOOD, GOOD, 4, 64, GOOD, GOOD, 3, GOOD]
        args[at] += off
        assert f(*args, None) == -3
    for at in (0, 1, 2, 3, 6, 7, 9):
        args = [GOOD, GOOD, GOOD, GOOD, 64, 4, GOOD, GOOD, 3, GOOD]
        args[at] = None
        assert g(*args, None) == -1
        args[at] = GOOD + 1
        assert g(*args, None) == -3


@no_gpu_only
def test_lora_refusals():
    f = lib().lora_add
    ws = lib().pbg_lora_workspace_bytes(5, 16)
    assert ws >= 4 * 5 * 16
    for m, r in ((0, 16), (5, 0), (5, 129), (2 ** 20 + 1, 16)):
        assert lib().pbg_lora_workspace_bytes(m, r) == 0

    def call(p=None, m=5, n=32, k=64, na=3, r=16, nbytes=ws, put=None):
        a = [GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, m, n, k, na, r, GOOD, GOOD, nbytes]
        if p is not None:
            a[p] = put
        return f(*a, None)

    for p in (0, 1, 2, 3, 4, 5, 11, 12):
        assert call(p, put=None) == -1
        assert call(p, put=GOOD + 1) == -3
    assert call(m=0) == -2 and call(n=0) == -2 and call(k=0) == -2 and call(k=2 ** 17 + 1) == -2
    assert call(na=0) == -2 and call(na=65537) == -2 and call(r=0) == -2 and call(r=129) == -2
    assert call(nbytes=ws - 1) == -6


def test_binding_rejects_cpu_tensors():
    import torch

    f32, f16, i8, i32 = torch.float32, torch.float16, torch.int8, torch.int32
    x, h, q, ids = torch.zeros((2, 64), dtype=f32), torch.zeros((2, 64), dtype=f16), torch.zeros((2, 64), dtype=i8), torch.zeros(2, dtype=i32)
    for call in (lambda: binding.add_rmsnorm(x, torch.ones(64)), lambda: binding.quantize_rows(h),
                 lambda: binding.ternary_gemm_i8(torch.zeros((4, 4), dtype=i32), torch.ones(4), 64, q, torch.ones(2)),
                 lambda: binding.lora_add(x, h, ids, torch.zeros((1, 8, 64), dtype=f16), torch.zeros((1, 64, 8), dtype=f16),
                                          torch.ones(1))):
        with pytest.raises(ValueError):
            call()


def test_oracle_codes():
    """Codes are within half a step of the value (plus fp32 rounding), the largest one is 127."""
    rng = np.random.default_rng(3)
    p = rng.standard_normal((50, 333)).astype(np.float32) * np.exp(rng.uniform(-60, 60, (50, 1))).astype(np.float32)
    p[7] = 0.0
    q, top = oracle.row_codes(p)
    step = top.astype(np.float64)[:, None] / 127.0
    assert np.all(np.abs(q * step - p) <= step * (0.5 + 127 * 2.0 ** -22))
    assert np.all(np.abs(q.astype(int)).max(axis=1) == np.where(np.arange(50) == 7, 0, 127)) and top[7] == 0.0
    p[3, 5], p[4, 6] = np.nan, -np.inf
    q, top = oracle.row_codes(p)
    assert np.isnan(top[[3, 4]]).all() and not q[[3, 4]].any()
    assert oracle.row_codes(np.full((1, 4), 1e-31, np.float32))[1][0] == 0.0


def test_oracle_norm_and_products():
    rng = np.random.default_rng(4)
    x, res = rng.standard_normal((3, 40)).astype(np.float32), rng.standard_normal((3, 40)).astype(np.float32)
    w = rng.uniform(0.5, 1.5, 40).astype(np.float32)
    r, h, q, qs = oracle.add_rmsnorm(x, w, 1e-6, res)
    for i in range(3):
        mean = sum(float(v) ** 2 for v in r[i]) / 40
        assert np.allclose(h[i], [float(a) * float(b) / (mean + 1e-6) ** 0.5 for a, b in zip(r[i], w)], rtol=1e-12)
    assert np.all(np.abs(q * qs[:, None] - h) <= 0.501 * qs[:, None])
    codes, s = synth.ternary_codes(1, 9, 40), synth.row_scales(2, 9)
    y = oracle.ternary_gemm_i8(oracle.pack(codes)[0], s, 40, q, qs.astype(np.float32))
    for i in range(3):
        for j in range(9):
            t = sum(int(c) * int(v) for c, v in zip(codes[j], q[i]))
            assert y[i, j] == t * float(np.float32(qs[i])) * float(s[j])
    ids = np.array([1, -1, 0], np.int32)
    a, b = rng.standard_normal((2, 4, 40)).astype(np.float16), rng.standard_normal((2, 9, 4)).astype(np.float16)
    out = oracle.lora_add(y, x.astype(np.float16), ids, a, b, np.array([1.0, 2.0], np.float32))
    assert np.array_equal(out[1], y[1])
    w0 = b[1].astype(np.float64) @ a[1].astype(np.float64)
    assert np.allclose(out[0] - y[0], 2.0 * w0 @ x[0].astype(np.float16).astype(np.float64), rtol=1e-9, atol=1e-9)


def test_lora_workspace_grows_with_rows_and_rank():
    """A workspace for the most rows and the highest rank serves every smaller call."""
    f = lib().pbg_lora_workspace_bytes
    rows = [*range(1, 9001), *range(9001, 2 ** 20, 4999), 2 ** 20]
    for r in (1, 3, 4, 8, 16, 17, 33, 64, 128):
        sizes = [f(m, r) for m in rows]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), r
    for m in (1, 16, 17, 64, 65, 2048, 2049, 4097, 9000):
        sizes = [f(m, r) for r in range(1, 129)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), m
