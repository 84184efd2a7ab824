"""Verification of drafted tokens in exact arithmetic: the residuals as distributions of their own, each
made from the one before it, as whole numbers over a common denominator."""
from __future__ import annotations

import math
from fractions import Fraction

ONE = 1 << 200   # every fp32 number is a whole multiple of 1 / ONE


def _weights(row):
    """A row's probabilities times ONE: what is not positive and finite counts as zero."""
    return [int(math.ldexp(x, 200)) if x > 0 and math.isfinite(x) else 0 for x in map(float, row)]


def _pick(r, sample):
    """The least index whose running sum passes sample * sum; None where there is no weight."""
    total, u = sum(r), Fraction(float(sample))
    if not total:
        return None
    run = 0
    for k, x in enumerate(r):
        run += x
        if run * u.denominator > u.numerator * total:
            return k


def verified(p, q, tokens, parents, accept, sample):
    """One sequence: (accepted path, next token or -1).  p: rows after the last accepted token and after
    each node; q: rows the children were drawn from, or None."""
    vocab = len(p[0])
    cur, path = 0, []
    r, whole = _weights(p[0]), ONE   # the distribution r / whole; a target's row is taken as it is
    for j, x in enumerate(tokens):
        if parents[j] + 1 != cur or not 0 <= x < vocab:
            continue
        u = Fraction(float(accept[j]))
        draw = None if q is None else _weights(q[cur])
        asked = u.numerator * (ONE if draw is None else draw[x]) * whole
        if r[x] > 0 and asked < r[x] * ONE * u.denominator:
            cur = j + 1
            path.append(j)
            r, whole = _weights(p[cur]), ONE
            continue
        if draw is None:
            r[x] = 0
        else:
            r = [max(y * ONE - z * whole, 0) for y, z in zip(r, draw)]
        whole = sum(r) or 1
    token = _pick(r, sample)
    if token is None:
        token = _pick(_weights(p[cur]), sample)
    return path, -1 if token is None else token
