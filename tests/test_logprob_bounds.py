"""How far dt_token_logprobs may be off, from the distances of a row's logits alone, and what that bound refuses.

With y = m - x >= 0 the distance of a logit from the row's largest, and averages E over the row's softmax, in units of 2^-24:
an exponent is the difference to the reference, rounded, times log2 e, which is rounded, and the product: 2.5 times the distance from the
reference, which a logit passes by 8 log2 units (5.6) at most: 2.5 (y + 5.6). The reference moves by 5.5 or more at a time, and in
all by no more than y + 5.6, so that the factors of the sums are off by as much once more, and each by 4 (exp2) and 1 (the product), y / 5.5 + 1.02
of them and one where pieces are put together. exp2 of a weight: 4. Sums: 16 terms, 8 steps, two halves, five shuffles: 30
(pieces are added in 64 bits). So S is off by a factor within 1 +- u, u = 5 (E y + 5.6) + 5 (E y / 5.5 + 2.02) + 34.
log S adds 2 (the mantissa rounded, and its logarithm below 1), the result its own rounding.

The entropy's second sum has terms weight times distance. With Y = y + 5.6, which no distance from a reference on a term's way
passes: 2.5 Y for the distance, (4 + 30 + 10.1) Y + 5.91 Y Y for the weight and the sums as above, and 8 (y / 5.5 + 2.02) Y where references move
(a sum, two products and the factor): 62.8 E Y + 7.4 E Y Y in all. It is divided by S: u E y.

Nothing goes by the logits themselves. Where the largest logit times log2 e is rounded before it is subtracted, exponents are off
by 2^-24 of that product: such sums are refused by the bound for large logits.
"""
import math

import numpy as np
import pytest

H = 2.0 ** -24


def bounds(x):
    """x: a row of logits in 64 bits, no NaN, one finite at least: (log S, entropy, tolerance of log S, of the entropy)."""
    y = x.max() - x[x > -math.inf]
    w = np.exp(-y)
    S = w.sum()
    p = w / S
    ent = math.log(S) + float((p * y).sum())
    Ey, Y = float((p * y).sum()), y + 5.6
    u = H * (5 * (Ey + 5.6) + 5 * (Ey / 5.5 + 2.02) + 34)
    log_s = u + 2 * H
    return math.log(S), ent, log_s, log_s + Ey * u + H * (62.8 * float((p * Y).sum()) + 7.4 * float((p * Y * Y).sum())) + H * abs(ent)


def _sums(x, rounded):
    """S relative to the largest logit as fp32 makes it, terms added in 64 bits."""
    f = np.float32
    c, m = f(1.4426950408889634), x.max()
    if rounded:
        d = f(x.astype(np.float64) * np.float64(c) - np.float64(f(m * c)))
    else:
        d = f(f(x - m) * c)
    return float(np.exp2(d.astype(np.float64)).sum())


@pytest.mark.parametrize("spread,offset", [(0.5, 0.0), (3.0, 0.0), (60.0, 0.0), (3000.0, 0.0), (3.0, 5000.0), (3.0, -1e6)])
def test_the_bound_refuses_a_rounded_reference(spread, offset):
    rng = np.random.default_rng(3)
    refused = 0
    for _ in range(40):
        x = (rng.standard_normal(3000) * spread + offset).astype(np.float32)
        log_s, _, tol, _ = bounds(x.astype(np.float64))
        assert abs(math.log(_sums(x, False)) - log_s) <= tol
        refused += abs(math.log(_sums(x, True)) - log_s) > tol
    assert refused >= 30 or abs(offset) + 3 * spread < 4000, refused
