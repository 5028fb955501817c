"""rotary_qkv on the GPU: norms of heads whose squares leave fp32."""
from __future__ import annotations

import numpy as np
import pytest

import oracle  # noqa: F401
from test_step_gpu import check_rotary, pbg, rotary_case, say  # noqa: F401 (pbg is a fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("m,heads,kv,d,rot,inter", [(9, 4, 2, 64, 64, False), (300, 32, 8, 128, 128, False), (600, 20, 5, 80, 32, True),
                                                    (5, 3, 1, 256, 256, False), (4, 1, 1, 8, 0, False)])
def test_norm_of_large_heads(pbg, m, heads, kv, d, rot, inter):  # noqa: F811
    """Elements of 1e19 to 3e38 in some heads: their quotient by the norm is of order one. Neighbours keep theirs."""
    say(f"rotary large m={m} heads={heads}/{kv} d={d}")
    c, pages, page = rotary_case(m, m, heads, kv, d, rot, 3)
    x = c["qkv"].reshape(m, heads + 2 * kv, d)
    rng = np.random.default_rng(1)
    for a in range(0, m, 2):
        x[a, rng.integers(0, heads + kv)] *= 1e19
        x[a, heads] *= 3e37 / np.abs(x[a, heads]).max()
        x[a, 0, rng.integers(0, d)] = 3.4e38
    c["qkv"] = x.reshape(m, -1)
    check_rotary(pbg, c, pages, page, heads, kv, d, inter)
    check_rotary(pbg, c, pages, page, heads, kv, d, inter, eps=3e37)
