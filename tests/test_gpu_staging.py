"""Rotating appends whose arguments fill most of the staging buffer: the metadata's
and the rows' go in one region, which has its place before anything is launched."""
import numpy as np
import pytest
import torch

import _rows as R
from copy_write_forked_gb300.dendrite import Pool, Rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()
    torch.cuda.set_device(0)


# A branch of 64 drafted tokens with a tree of its own takes 12 bytes of the
# metadata's arguments and 76 of the rows'.  27,700 of them: 2,105,200 bytes of
# the rows', more than half of the 4 MiB buffer.  27,000 after six decode steps
# (324,096 bytes each): two regions would begin at 1,944,576, and at 0 for the
# second's 2,052,000 bytes, which reach into the first.
@pytest.mark.parametrize("n,steps", [(27_700, 0), (27_000, 6)])
def test_a_tree_for_each_of_many_branches(n, steps):
    new, base, d = 64, 5, 128
    lens = base + steps
    pool = Pool(n * 6 + 4, 16, 1, d, torch.bfloat16, max_branches=n + 8, max_blocks_per_branch=8)
    g = torch.Generator(device="cuda").manual_seed(n)
    rows = lambda *s: torch.randn(*s, 1, d, generator=g, device="cuda").bfloat16()  # noqa: E731
    root = pool.new_branch()
    past = rows(1, base)
    pool.append_kv([root], past, past)
    br = pool.fork(root, n)
    decoded = [rows(n, 1) for _ in range(steps)]
    K, V = rows(n, new), rows(n, new)
    parents = torch.randint(-1, 1 << 20, (n, new), dtype=torch.int32, generator=torch.Generator().manual_seed(n))
    parents = (parents % (torch.arange(new, dtype=torch.int32) + 1)) - 1   # -1 .. j - 1
    rope = Rope(d)
    torch.cuda.synchronize()
    for x in decoded:   # (queued at once: the arguments of the last calls are still on their way)
        pool.append_kv(br, x, x)
    pool.append_rope(br, K, V, rope, parents=parents)
    pool.sync()
    assert {pool.branch_len(b) for b in br} == {lens + new}
    k, v = pool.read_kv(br, [lens] * n, [new] * n)
    assert torch.equal(v.view_as(V), V)
    for i in (0, 1, n // 2, n - 1):
        y, size = R.rotate(R.f64(K[i]), lens + np.array(R.depths(parents[i].tolist())), R.frequencies(d)[0], d, False)
        assert (np.abs(R.f64(k[i * new:(i + 1) * new]) - y) <= R.ROPE_ERR * size + 2.0 ** -8 * (np.abs(y) + R.ROPE_ERR * size)).all()
    k, v = pool.read_kv(br, [0] * n, [lens] * n)
    want = torch.cat([past.expand(n, -1, -1, -1)] + decoded, 1)
    assert torch.equal(k.view_as(want), want) and torch.equal(v.view_as(want), want)
    pool.free([root] + br)
    pool.sync()
    assert sum(pool.read_refcounts()) == 0
    pool.close()
