"""Verification next to borders, and where a residual is a small part of its row: whole numbers, equal to those of
rational arithmetic wherever a number is farther from its border than the sums are documented to be off."""
import random

import numpy as np
import pytest
import torch

from copy_write_forked_gb300.dendrite import Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()
    torch.cuda.set_device(0)


@pytest.fixture(scope="module")
def pool():
    p = Pool(16, 16, 1, 128, torch.bfloat16, max_branches=4)
    yield p
    p.sync()
    p.close()


def test_a_border_between_two_ctas(pool):
    """Half of a row's sum ends with one CTA's share, and the next share is empty: however the two halves' sums are
    rounded (they have the same terms in another order), one token is given, on one side of the border."""
    rng, n, vocab = random.Random(1), 16, 32768     # 16 CTAs a sequence, of 2,048 tokens each
    tokens, accept = torch.full((n, 1), -1, dtype=torch.int32, device="cuda"), torch.zeros(n, 1, device="cuda")
    sample = torch.full((n,), 0.5, device="cuda")
    for _ in range(16):
        p = np.zeros((n, 2, vocab), np.float32)
        for i in range(n):
            big = [np.float32(rng.uniform(0.02, 0.06) * 2.0 ** rng.choice([0, 0, -1, -3])) for _ in range(7)]
            pairs = [(x, np.float32(float(x) * 2.0 ** -25 * rng.uniform(0.1, 0.9))) for x in big]
            for first, some in ((0, pairs), (8, rng.sample(pairs, 7))):
                for k, (x, y) in enumerate(some):
                    p[i, 0, 2048 * (first + k)], p[i, 0, 2048 * (first + k) + 1] = x, y
        got = pool.verify_draft(tokens, torch.from_numpy(p).cuda(), [-1], accept, sample)[2].tolist()
        # the border: behind the last token of the seventh share, before the first of the ninth
        assert all(x in (2048 * 6 + 1, 2048 * 8) for x in got), got
