"""penalize_logits on the GPU, bit for bit: zeros of both signs, numbers below the normals, infinities; `top` of a zero is +0."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from logits_helpers import only_zeros, same_bits, zeros_case
from test_step_gpu import LOGITS, dev, host, logits_case, pbg, say  # noqa: F401 (pbg is a fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def check_bits(pbg, c):  # noqa: F811
    for in_place in (False, True):
        d = {k: dev(v) for k, v in c.items()}
        out, token, top = pbg.penalize_logits(**d, out=d["logits"] if in_place else None, greedy=True)
        ref, tok, best = oracle.penalize_logits(**c)
        live = tok != -2
        assert same_bits(host(out)[live], ref[live])
        assert np.array_equal(host(token)[live], tok[live])
        assert same_bits(host(top)[live], (best + np.float32(0.0))[live])  # -0 + 0 is +0


@pytest.mark.parametrize("r,rows,n,hist,bias,grammar", LOGITS)
def test_bits(pbg, r, rows, n, hist, bias, grammar):  # noqa: F811
    say(f"logits bits r={r} rows={rows} n={n}")
    check_bits(pbg, logits_case(n + r, r, rows, n, hist, rows > 1, bias, grammar))


@pytest.mark.parametrize("r,rows,n,hist", [(3, 2, 2000, 700), (6, 4, 9001, 9000), (1, 1, 64, 40), (8, 1, 30011, 20000)])
def test_bits_of_zeros(pbg, r, rows, n, hist):  # noqa: F811
    say(f"logits zeros r={r} rows={rows} n={n}")
    for seed in range(4):
        c = zeros_case(seed, r, rows, n, hist)
        check_bits(pbg, c)
        check_bits(pbg, only_zeros(c))
