"""Forks onto selected rows through the C-ABI library: rows bit for bit, tables, reference counts and the free stack
as the documented order gives them, and children that live on like any other branch."""
import random

import numpy as np
import pytest
import torch

import _rows as R
from copy_write_forked_gb300 import workloads as W
from copy_write_forked_gb300.dendrite import DendriteError, Pool, Rope

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "fp8", "fp32"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()
    torch.cuda.set_device(0)


class Case:
    """A pool with branches of the given lengths, and its rows as the pool gives them back."""

    def __init__(self, kind, lens, kv=2, dim=128, layers=1, blocks=600, seed=0, **kw):
        self.kind, self.kv, self.dim, self.layers = kind, kv, dim, layers
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = Pool(blocks, 16, kv, dim, R.POOL_DTYPE[kind], n_layers=layers, **{"max_branches": 64, "max_blocks_per_branch": 512, **kw})
        self.br = [self.pool.new_branch() for _ in lens]
        for b, x in zip(self.br, lens):
            if x:
                self.append([b], x)

    def append(self, br, n):
        lead = (self.layers,) if self.layers > 1 else ()
        k, v = (torch.randn(*lead, len(br), n, self.kv, self.dim, generator=self.g, device="cuda").to(R.ROW_DTYPE[self.kind])
                for _ in range(2))
        self.pool.append_kv(br, k, v)

    def rows(self, b):
        """[layer][K, V][length][kv][dim], and the stored bytes where the values are not all there is."""
        n = self.pool.branch_len(b)
        return [self.pool.read_kv([b], [0], [n], layer=l) for l in range(self.layers)]

    def state(self, br):
        return [self.pool.read_table(b) for b in br], self.pool.read_refcounts(), self.pool.read_free_stack()

    def fork(self, parents, starts, lists, per_head=False):
        """fork_rows with lists of rows (per_head: [layer][count][kv]), checked against the parents' rows and the order of blocks."""
        before = [self.rows(b) for b in parents]
        tables, counts, stack = self.state(parents)
        if per_head:
            flat = torch.cat([x.reshape(self.layers, -1, self.kv) for x in lists], 1).int().cuda()
            flat = flat[0].contiguous() if self.layers == 1 else flat.contiguous()
            sizes = [x.shape[-2] for x in lists]
        else:
            flat, sizes = torch.tensor([r for x in lists for r in x], dtype=torch.int32, device="cuda"), [len(x) for x in lists]
        kids = self.pool.fork_rows(parents, starts, sizes, flat)
        self.pool.sync()
        for i, kid in enumerate(kids):
            want, shared, total = [], starts[i] // 16, starts[i] + sizes[i]
            for blk in tables[i][:shared]:
                counts[blk] += 1
                want.append(blk)
            for _ in range(-(-total // 16) - shared):
                want.append(stack.pop())
                counts[want[-1]] = 1
            assert self.pool.read_table(kid) == want and self.pool.branch_len(kid) == total
            for l, (k, v) in enumerate(self.rows(kid)):
                for got, old in zip((k, v), before[i][l]):
                    assert torch.equal(got[:starts[i]], old[:starts[i]])
                    for h in range(self.kv):
                        at = lists[i].reshape(self.layers, -1, self.kv)[l, :, h].long().cuda() if per_head else torch.tensor(lists[i], device="cuda").long()
                        assert torch.equal(got[starts[i]:, h], old[at, h]), (i, l, h)
        assert self.state(parents) == (tables, counts, stack)
        for b, old in zip(parents, before):   # the parents stand as they were
            for x, y in zip(self.rows(b), old):
                assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
        return kids


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("fp8", 128), ("fp32", 128), ("fp32", 32), ("fp32", 96), ("fp32", 256)])
@pytest.mark.parametrize("kv", [1, 3, 8])
@pytest.mark.parametrize("per_head", [False, True])
def test_selected_rows(kind, dim, kv, per_head):
    rng = random.Random(kv)
    c = Case(kind, [100, 16, 37, 1, 200], kv=kv, dim=dim)
    all0 = c.state([])
    parents = [c.br[i] for i in (0, 1, 2, 3, 4, 4, 0, 0)]
    starts = [0, 16, 15, 1, 33, 200, 99, 4]
    sizes = [17, 5, 16, 3, 100, 0, 1, 31]
    lens = [c.pool.branch_len(b) for b in parents]
    if per_head:
        lists = [torch.tensor([[rng.randrange(n) for _ in range(kv)] for _ in range(s)], dtype=torch.int32).reshape(1, s, kv)
                 for n, s in zip(lens, sizes)]
    else:
        lists = [sorted(rng.sample(range(n), s)) if s <= n and i % 2 else [rng.randrange(n) for _ in range(s)]
                 for i, (n, s) in enumerate(zip(lens, sizes))]
    kids = c.fork(parents, starts, lists, per_head)
    c.append(kids, 3)                      # children live on
    grand = c.pool.fork(kids[0], 2)
    c.append(grand, 20)
    c.fork(grand, [0, 20], [torch.zeros(1, 5, kv, dtype=torch.int32)] * 2 if per_head else [[36, 0, 20]] * 2, per_head)
    c.pool.free(kids)
    c.pool.sync()
    assert len(c.state([])[2]) < len(all0[2])
    c.pool.close()


@pytest.mark.parametrize("kind", KINDS)
def test_layers_with_lists_of_their_own(kind):
    rng = random.Random(3)
    c = Case(kind, [50, 70], kv=4, layers=3)
    lists = [torch.tensor([[[rng.randrange(n) for _ in range(4)] for _ in range(s)] for _ in range(3)], dtype=torch.int32) for n, s in ((50, 20), (70, 33))]
    c.fork(c.br, [5, 16], lists, per_head=True)
    c.fork(c.br, [5, 16], [[49, 3, 3], list(range(70))])
    c.pool.close()


def test_every_count_around_a_block():
    c = Case("bf16", [64], blocks=3000, max_branches=1200)
    starts, lists = [], []
    for start in (0, 1, 15, 16, 17, 31, 32, 33, 63, 64):
        for count in (0, 1, 2, 14, 15, 16, 17, 31, 32, 33, 64):
            starts.append(start)
            lists.append([(7 * k + start) % 64 for k in range(count)])
    c.fork([c.br[0]] * len(starts), starts, lists)   # more arguments than the small parameter block holds
    c.fork([c.br[0]] * 4 * len(starts), starts * 4, lists * 4)   # staged
    c.pool.close()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_compaction(kind):
    """Thinned and the parents freed: all but the kept blocks come back, and the kept rows attend as they should."""
    rng = random.Random(5)
    c = Case(kind, [300, 280, 333])
    root = c.pool.fork_batch(c.br, [2, 1, 1])
    br = [x for ch in root for x in ch]
    c.pool.free(c.br)
    lens = [c.pool.branch_len(b) for b in br]
    lists = [sorted(rng.sample(range(40, n), 61)) for n in lens]
    kids = c.fork(br, [40] * 4, lists)
    c.pool.free(br)
    c.pool.sync()
    used = sum(x > 0 for x in c.pool.read_refcounts())
    assert used == 2 * 3 + 4 * 5   # the whole blocks before row 40, of the forked pair once, and 61 + 8 rows each in 5 blocks
    for step in range(3):
        c.append(kids, 2)
        q = torch.randn(4, 2, 8, 128, generator=c.g, device="cuda").bfloat16()
        out = c.pool.tree_attn_decode(q, kids)
        for i, b in enumerate(kids):
            K, V = (R.f64(x) for x in c.rows(b)[0])
            see = np.arange(len(K)) <= len(K) - 2 + np.arange(2)[:, None]
            ref = R.attention(R.f64(q[i]), K, V, see)
            assert (np.abs(R.f64(out[i]) - ref[0]) <= R.attention_bound(kind, *ref)).all()
    c.pool.free(kids)
    c.pool.sync()
    assert sum(c.pool.read_refcounts()) == 0 and sorted(c.pool.read_free_stack()) == list(range(600))
    c.pool.close()


@pytest.mark.parametrize("kind", KINDS)
def test_children_and_parents_do_not_touch_one_another(kind):
    c = Case(kind, [45])
    b = c.br[0]
    kid, twin = c.fork([b, b], [40, 32], [[1, 2, 3], []])
    kept = [c.rows(x) for x in (kid, twin)]
    c.append([b], 30)
    c.pool.truncate([b], [20])
    c.append([b], 5)
    for x, old in zip((kid, twin), kept):
        assert all(torch.equal(p, q) for p, q in zip(c.rows(x)[0], old[0]))
    own = c.rows(b)
    c.append([kid, twin], 3)
    c.pool.truncate([kid], [10])           # below what it shares
    c.append([kid], 9)
    assert all(torch.equal(p, q) for p, q in zip(c.rows(b)[0], own[0]))
    c.pool.free([b])
    assert all(torch.equal(p[:32], q) for p, q in zip(c.rows(twin)[0], kept[1][0]))
    c.fork([twin, kid], [3, 18], [[34, 0], [18]])
    c.pool.close()


def test_a_child_cut_below_the_parents_own_fork():
    """Shares blocks that its parent has from a grandparent; plans over the whole family read each block once."""
    c = Case("bf16", [128])
    mid = c.pool.fork(c.br[0], 2)
    c.append(mid, 50)
    kids = c.fork([mid[0], mid[1], mid[0]], [64, 140, 17], [[150, 100], [0, 177], list(range(170, 178))])
    every = c.br + mid + kids
    q = torch.randn(len(every), 1, 8, 128, generator=c.g, device="cuda").bfloat16()
    for br in (every, every[::-1], kids):
        out = c.pool.tree_attn_decode(q[:len(br)], br)
        for i, b in enumerate(br):
            K, V = (R.f64(x) for x in c.rows(b)[0])
            ref = R.attention(R.f64(q[i]), K, V, np.ones((1, len(K)), bool))
            assert (np.abs(R.f64(out[i]) - ref[0]) <= R.attention_bound("bf16", *ref)).all()
    distinct = {blk for b in every for blk in c.pool.read_table(b)}
    c.pool.tree_attn_decode(q, every)
    assert c.pool.last_plan_stats()["unique_tiles"] == 2 * len(distinct)
    # drafts accepted on a child: its own rows may move
    c.append([kids[0]], 6)
    rows = [torch.cat((x[:66], x[66 + torch.tensor([1, 4], device="cuda")])) for x in c.rows(kids[0])[0]]
    c.pool.accept_draft([kids[0]], 6, [[1, 4]])
    assert all(torch.equal(x, y) for x, y in zip(c.rows(kids[0])[0], rows))
    c.pool.close()


def test_compressed_pools():
    """Records move as they are."""
    pool = Pool(64, 16, 2, 128, torch.bfloat16, turbo=W.turbo_codec(1), max_branches=8)
    b = pool.new_branch()
    x = torch.randn(1, 50, 2, 128, device="cuda").bfloat16()
    pool.append_kv([b], x, x + 1)
    rows = [49, 3, 17, 17, 0, 30] * 4
    kid = pool.fork_rows([b], [18], [len(rows)], torch.tensor(rows, dtype=torch.int32, device="cuda"))[0]
    pool.sync()

    def records(branch):
        n = pool.branch_len(branch)
        blocks = [pool.read_block(x) for x in pool.read_table(branch)]
        return [torch.cat([blk[i] for blk in blocks], 1)[:, :n] for i in range(2)]

    for old, new in zip(records(b), records(kid)):
        assert torch.equal(new[:, :18], old[:, :18]) and torch.equal(new[:, 18:], old[:, torch.tensor(rows)])
    assert pool.read_table(kid)[0] == pool.read_table(b)[0]
    pool.close()


def test_rows_that_are_not_finite():
    """Rows of NaN are moved like any other, and a child's unwritten slots do not hold what its blocks held before."""
    pool = Pool(8, 16, 1, 128, torch.bfloat16, max_branches=8)
    a = pool.new_branch()
    x = torch.randn(1, 128, 1, 128, device="cuda").bfloat16()
    pool.append_kv([a], x, torch.full_like(x, float("nan")))
    pool.free([a])
    b = pool.new_branch()
    y = x[:, :40].contiguous()
    y[0, 39] = float("inf")
    pool.append_kv([b], y, y)
    kid = pool.fork_rows([b], [3], [7], torch.tensor([38, 1, 2, 3, 4, 5, 39], dtype=torch.int32, device="cuda"))[0]
    k, v = pool.read_kv([kid], [0], [10])
    want = y[0, [0, 1, 2, 38, 1, 2, 3, 4, 5, 39]]
    assert torch.equal(k, want) and torch.equal(v, want)
    pool.truncate([kid], [9])
    clean = pool.fork_rows([kid], [0], [9], torch.arange(9, dtype=torch.int32, device="cuda"))[0]
    q = torch.randn(1, 1, 4, 128, device="cuda").bfloat16()
    for br in (clean, kid):
        out = pool.tree_attn_decode(q, [br])
        ref = R.attention(R.f64(q[0]), R.f64(k[:9]), R.f64(v[:9]), np.ones((1, 9), bool))
        assert (np.abs(R.f64(out[0]) - ref[0]) <= R.attention_bound("bf16", *ref)).all()
    pool.close()


def test_a_long_shared_prefix():
    """More shared entries than one chunk of the table, for several children of one parent."""
    c = Case("fp8", [6000], kv=1, blocks=900)
    c.fork([c.br[0]] * 5, [5999, 4096, 4112, 16, 0], [[0], [5999] * 3, [], [1, 2], list(range(0, 6000, 3))])
    c.pool.close()


def test_past_32_bit_offsets():
    blocks = 136_000   # 64 KiB of K a block: past 4 GiB of elements' bytes
    pool = Pool(blocks + 64, 16, 8, 128, torch.bfloat16, max_branches=64)
    x = torch.randn(1, 65536, 8, 128, device="cuda").bfloat16()
    for lo in range(0, blocks, 4096):
        pool.append_kv([pool.new_branch()], *[x[:, :16 * min(4096, blocks - lo)].contiguous()] * 2)
    b = pool.new_branch()
    pool.append_kv([b], x[:, :200].contiguous(), x[:, 200:400].contiguous())
    rows = torch.randint(0, 200, (300, 8), dtype=torch.int32, device="cuda")
    kid = pool.fork_rows([b], [0], [300], rows)[0]
    assert min(pool.read_table(kid)) >= blocks
    k, v = pool.read_kv([kid], [0], [300])
    for h in range(8):
        assert torch.equal(k[:, h], x[0, rows[:, h].long(), h]) and torch.equal(v[:, h], x[0, 200 + rows[:, h].long(), h])
    pool.close()


def test_another_stream_and_the_lists_memory():
    pools = [Case("bf16", [400, 300], seed=1) for _ in range(2)]
    lists = [torch.randint(0, 300, (500,), dtype=torch.int32, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    kids, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for c, s, l in zip(pools, streams, lists):   # two calls at once
        kids.append(c.pool.fork_rows(c.br, [8, 16], [250, 250], l, stream=s))
    torch.cuda.synchronize()
    for c, ks, l in zip(pools, kids, lists):
        for i, start in enumerate((8, 16)):
            old, new = c.rows(c.br[i])[0][0], c.rows(ks[i])[0][0]
            assert torch.equal(new[start:], old[l[250 * i:250 * i + 250].long()])
        c.pool.close()


def test_too_few_blocks_and_bad_rows_are_reported():
    c = Case("bf16", [64], blocks=10)
    kid = c.fork([c.br[0]], [0], [list(range(64))])   # 8 of 10 blocks
    c.fork([c.br[0]], [32], [[0] * 32])
    assert c.pool.fork_rows([c.br[0]], [64], [0], None)
    stack, counts = c.pool.read_free_stack(), c.pool.read_refcounts()
    c.pool.fork_rows([c.br[0]], [0], [1], torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert c.pool.sync_status() == -2
    assert c.pool.read_free_stack() == stack and c.pool.read_refcounts() == counts
    with pytest.raises(DendriteError):
        c.pool.fork(kid[0], 1)
    c.pool.close()
    for bad in (64, -1, 2147483647, -2147483648):
        c = Case("bf16", [64])
        c.pool.fork_rows([c.br[0]], [3], [2], torch.tensor([0, bad], dtype=torch.int32, device="cuda"))
        assert c.pool.sync_status() == -1
        c.pool.close()


def test_refusals():
    c = Case("bf16", [20, 0], kv=2, max_branches=6, max_blocks_per_branch=8)
    a, empty = c.br
    rows = torch.zeros(4, dtype=torch.int32, device="cuda")
    state = c.state([a])
    wide = torch.zeros(40, dtype=torch.int32, device="cuda")
    bad = [([a], [0], [4], rows.long()), ([a], [0], [4], rows.cpu()), ([a], [0], [3], rows), ([a], [21], [4], rows), ([a], [-1], [4], rows),
           ([a], [0], [-4], rows), ([a], [0, 0], [4], rows), ([99], [0], [4], rows), ([empty], [0], [4], rows), ([a], [0], [4], None),
           ([a], [0], [4], torch.zeros(4, 3, dtype=torch.int32, device="cuda")), ([a], [0], [4], wide[::10]),
           ([a] * 5, [20] * 5, [0] * 5, None), ([a], [0], [129], torch.zeros(129, dtype=torch.int32, device="cuda"))]
    for args in bad:
        with pytest.raises(DendriteError):
            c.pool.fork_rows(*args)
    assert c.state([a]) == state
    c.pool.append_begin([a], 1)
    with pytest.raises(DendriteError):
        c.pool.fork_rows([a], [0], [4], rows)
    z = torch.zeros(1, 1, 2, 128, device="cuda", dtype=torch.bfloat16)
    c.pool.append_layer(0, z, z)
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        graph.capture_begin()
        try:
            with pytest.raises(DendriteError):
                c.pool.fork_rows([a], [0], [4], rows)
            rows.add_(0)
        finally:
            graph.capture_end()
    assert c.pool.fork_rows([], [], [], None) == []
    kids = c.pool.fork_rows([a, a, empty], [21, 0, 0], [0, 0, 0], None)   # nothing copied
    assert [c.pool.branch_len(b) for b in kids] == [21, 0, 0]
    c.pool.sync()
    c.pool.close()


def test_thinned_branches_go_on_at_their_old_positions():
    """After rows are dropped, new rows are turned by positions that go on from the parent's."""
    c = Case("fp32", [90], kv=1)
    kid = c.fork([c.br[0]], [4], [list(range(60, 90))])[0]
    x = torch.randn(1, 3, 1, 128, device="cuda")
    at = torch.tensor([[90, 91, 92]], dtype=torch.int32, device="cuda")
    c.pool.append_rope([kid], x, x, Rope(128), positions=at)
    c.pool.append_rope([c.br[0]], x, x, Rope(128))
    assert torch.equal(c.pool.read_kv([kid], [34], [3])[0], c.pool.read_kv([c.br[0]], [90], [3])[0])
    c.pool.close()
