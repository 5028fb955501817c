"""The strict comparison of penalize_logits on the CPU: what it notices, and that its cases have what it looks for."""
from __future__ import annotations

import numpy as np

import oracle
from logits_helpers import only_zeros, same_bits, zeros_case


def test_strict_comparison():
    """A planted zero of the other sign, a NaN too many, one too few and the last bit are noticed; a NaN's payload does not matter."""
    c = zeros_case(1, 3, 2, 2000, 700)
    ref, token, top = oracle.penalize_logits(**c)
    assert same_bits(ref.copy(), ref)
    negative, positive = (ref == 0) & np.signbit(ref), (ref == 0) & ~np.signbit(ref)
    small = (ref != 0) & (np.abs(ref) < 2.0 ** -126)
    assert negative.sum() > 100 and positive.sum() > 100 and small.sum() > 100 and np.isnan(ref).any() and np.isinf(ref).any()
    for where, value in ((negative, 0.0), (positive, -0.0), (np.isnan(ref), 1.0), (positive, np.nan), (small, 0.0)):
        wrong = ref.copy()
        wrong[tuple(np.argwhere(where)[-1])] = value
        assert not same_bits(wrong, ref)
    wrong = ref.copy()
    wrong.view(np.uint32)[tuple(np.argwhere(ref == 1.5)[0])] += 1
    assert not same_bits(wrong, ref)
    other = ref.copy()
    other.view(np.uint32)[np.isnan(ref)] = 0x7FC12345
    assert same_bits(other, ref)


def test_best_of_zeros():
    """The best of a row of zeros and less is its first zero, whatever its sign."""
    c = only_zeros(zeros_case(2, 4, 4, 3000, 5))
    ref, token, top = oracle.penalize_logits(**c)
    assert (top == 0).all() and np.signbit(ref[np.arange(16), token]).any() and not np.signbit(ref[np.arange(16), token]).all()
    for a in range(16):
        assert token[a] == np.flatnonzero(ref[a] == 0)[0]
