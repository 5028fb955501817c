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

BLOCK = 64  # tokens; every unit of work of every kernel is one or more of these

# heads, kv heads, head_dim, rows of each request, tokens of each request: up to 235 units of 128 tokens or 470 of 64, so
# that every workgroup of a launch has a piece of the same rows
LONG = [(4, 1, 128, 1, [30001]), (4, 2, 64, 6, [30001]), (2, 1, 256, 3, [30001]), (12, 2, 128, 4, [30001]), (4, 1, 128, 40, [30001]),
        (2, 1, 64, 33, [30001]), (2, 1, 256, 40, [30001]), (4, 1, 128, 1, [9000, 12, 14001]), (4, 2, 64, 80, [9000, 12, 14001])]


def long_case(heads, kv, d, rows, lengths):
    """Scores of about one, and values that say where they stand: 1 in the column of the token's block, 0 elsewhere."""
    from test_step_gpu import attention_case

    c = attention_case(d + rows, lengths, [rows] * len(lengths), heads, kv, d, 16, spread=0.25)
    c["v_cache"][:] = 0
    for i, n in enumerate(lengths):
        t = np.arange(n + rows)
        c["v_cache"][c["table"][i, t // 16], :, t % 16, t // BLOCK % d] = 1
    return c
