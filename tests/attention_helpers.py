"""Cases and the tolerance that the tests of tree_attention's ends share."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
# bits that a weight keeps below the row's largest before it is lost to the second product: 25 of fp16's and the kernels' lift
LOST = 2.0 ** -33


def attention_bound(q, lengths, row_start, ref, size, far, total, high, scale):
    """How far an output may be off. A weight's exponent is off by the score's sum of d products, (d + 4) u scale sum |q_j k_j|, in the
    weight and in the largest, by the exponential's and its argument's roundings (30 u), and the weight by its rounding to fp16
    (2^-11; below the normals no more than LOST of the row's largest, of `total` of which the row has the sum). Numerator and denominator
    are off by that share of the sums of w |v| and w, and by n / 32 + 64 roundings of sums (blocks of 32 tokens one after another, in
    as many pieces as there are; merging p pieces adds p roundings and takes as many from the longest piece). Then fp16's rounding."""
    d = q.shape[2]
    n = int(np.max(lengths, initial=0)) + int(np.diff(row_start).max(initial=0))
    e = 2 * (d + 4) * U * scale * far + 30 * U + 2.0 ** -11 + (n / 32 + 64) * U
    off = e[:, :, None] * (size + np.abs(ref)) * 1.01 + n * LOST * high / np.maximum(total, 1.0)[:, :, None]
    return off + (np.abs(ref) + off) * 2.0 ** -11 + 2.0 ** -25
