"""The exact reference of drafted tokens' verification, pinned: by hand, and by what the method is for (the first
emitted token is distributed as the target alone would sample it)."""
from fractions import Fraction
from itertools import product

import pytest

from _verify import verified


def test_by_hand():
    p, q = [[0.25, 0.375, 0.25, 0.125], [0, 0, 1, 0]], [[0.5, 0.25, 0.125, 0.125]]
    assert verified(p, q, [0], [-1], [0.49], 0.0) == ([0], 2)     # 0.49 * 0.5 < 0.25
    assert verified(p, q, [0], [-1], [0.5], 0.0) == ([], 1)       # on the border: refused; residual 0, 1/8, 1/8, 0
    assert verified(p, q, [0], [-1], [0.5], 0.5) == ([], 2)       # the running sum has to pass the number
    assert verified(p, None, [0], [-1], [0.24], 0.5) == ([0], 2)
    assert verified(p, None, [0], [-1], [0.25], 0.0) == ([], 1)   # without token 0: 3/8, 1/4, 1/8 of 3/4
    assert verified(p, None, [0], [-1], [0.25], 0.5) == ([], 2)
    assert verified(p, None, [7], [-1], [0.0], 0.0) == ([], 0)    # a padding node: p itself
    assert verified([[0.0] * 3] * 2, None, [1], [-1], [0.0], 0.3) == ([], -1)
    assert verified([[0.5, 0.5]] * 3, [[0.5, 0.5]] * 2, [0, 1], [-1, 0], [0.9, 0.9], 0.75) == ([0, 1], 1)


def emitted(p, q, n_children, accepts, samples):
    """Distribution of the first emitted token over drafted tokens drawn from q and grids of the random numbers."""
    out = [Fraction(0)] * 4
    share = Fraction(1, len(accepts) ** n_children * len(samples))
    rows = [p] + [[0, 0, 0, 1]] * n_children
    for tokens in product(range(4), repeat=n_children):
        weight = share
        for x in tokens:
            weight *= Fraction(q[x]) if q else Fraction(1, 4)
        for us in product(accepts, repeat=n_children):
            for s in samples:
                path, nxt = verified(rows, [q] * n_children if q else None, list(tokens), [-1] * n_children, list(us), s)
                out[tokens[path[0]] if path else nxt] += weight
    return out


@pytest.mark.parametrize("n_children", [1, 2])
def test_the_first_token_is_the_targets(n_children):
    # ratios and residuals that the grids meet exactly: p / q is 1/2 or at least 1; (0, 1/2, 1/2, 0), then (0, 2/5, 3/5, 0)
    p, q = [0.25, 0.375, 0.25, 0.125], [0.5, 0.25, 0.125, 0.125]
    accepts, samples = [0.25, 0.75], [(k + 0.5) / 10 for k in range(10)]
    assert emitted(p, q, n_children, accepts, samples) == [Fraction(x) for x in p]


def test_certain_drafts_keep_the_targets_distribution():
    # any proposal, certain: accepted with its probability, else drawn from the rest (of 3/4, 5/8, 3/4, 7/8: 105 parts)
    p = [0.25, 0.375, 0.25, 0.125]
    accepts, samples = [(k + 0.5) / 8 for k in range(8)], [(k + 0.5) / 210 for k in range(210)]
    assert emitted(p, None, 1, accepts, samples) == [Fraction(x) for x in p]
