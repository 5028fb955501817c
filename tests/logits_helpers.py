"""A strict comparison for penalize_logits, and cases full of zeros of both signs."""
from __future__ import annotations

import numpy as np


def same_bits(got, ref) -> bool:
    """The same fp32 bits, zeros' signs among them, and NaN exactly where the reference is NaN."""
    nan = np.isnan(ref)
    return got.dtype == ref.dtype == np.float32 and got.shape == ref.shape and bool(
        np.array_equal(np.isnan(got), nan) and np.array_equal(got.view(np.uint32)[~nan], ref.view(np.uint32)[~nan]))


def zeros_case(seed, r, rows, n, hist):
    """Logits, penalties and biases whose results are zeros of either sign, numbers below the normals, infinities and NaN."""
    rng = np.random.default_rng(seed)
    m = r * rows
    pick = np.array([0.0, -0.0, 1.5, -1.5, 0.5, -0.5, 1e-40, -1e-40, 3e-45, 1e38, -1e38, np.inf, -np.inf, np.nan], np.float32)
    c = dict(logits=rng.choice(pick, (m, n)).astype(np.float32), request=np.repeat(np.arange(r), rows).astype(np.int32),
             tokens=rng.integers(0, n, (r, hist)).astype(np.int32), length=np.full(r, hist, np.int32),
             prompt_length=np.full(r, hist // 2, np.int32), repetition=rng.choice(np.array([1.0, -1.0, 0.5, 1e-30, 1e30, 0.0], np.float32), r),
             frequency=rng.choice(np.array([0.0, -0.0, 0.5, -1.5, 1.5], np.float32), r),
             presence=rng.choice(np.array([0.0, -0.0, 0.5, 1.5], np.float32), r))
    c["drafts"] = rng.integers(0, n, m).astype(np.int32)
    c["row_start"] = (np.arange(r + 1) * rows).astype(np.int32)
    c["ancestors"] = rng.integers(0, 2 ** rows, m).astype(np.uint64)
    c["bias_start"] = (np.arange(r + 1) * (n // 4)).astype(np.int32)
    c["bias_token"] = rng.integers(0, n, r * (n // 4)).astype(np.int32)
    c["bias_value"] = rng.choice(pick[:11], r * (n // 4)).astype(np.float32)
    return c


def only_zeros(c):
    """The same with no logit above zero, so that the best of a row is a zero of one sign or the other."""
    x = c["logits"]
    zero = np.where(np.arange(x.size).reshape(x.shape) % 3, np.float32(0.0), np.float32(-0.0))
    return {**{k: c[k] for k in ("request", "tokens", "length", "prompt_length")}, "logits": np.where(x > 0, zero, x),
            **{k: np.full(len(c["length"]), v, np.float32) for k, v in (("repetition", 1), ("frequency", 0), ("presence", 0))}}
