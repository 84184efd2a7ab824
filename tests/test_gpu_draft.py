"""Draft trees through the C-ABI library: attention of drafted tokens against 64 bits,
accepted paths kept row for row, and whole steps (rotary append, attention,
acceptance, read back) on every kind of pool."""
import random

import numpy as np
import pytest
import torch

import _rows as R
from copy_write_forked_gb300.dendrite import DendriteError, Pool, Rope

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "fp8", "fp32"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()
    torch.cuda.set_device(0)


class Case:
    """A pool of branches with drafted tokens behind them, and what it holds in 64 bits."""

    def __init__(self, kind, lens, new, kv, group, seed=0, dim=128, **kw):
        self.kind, self.new, self.kv, self.nq, self.dim = kind, new, kv, kv * group, dim
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = Pool(sum(2 * ((x + new) // 16 + 4) for x in lens) + 16, 16, kv, dim, R.POOL_DTYPE[kind],
                         max_branches=4 * len(lens) + 16, **kw)
        self.br = [self.pool.new_branch() for _ in lens]
        self.K, self.V = {}, {}
        for b, x in zip(self.br, lens):
            self.K[b] = self.V[b] = np.zeros((0, kv, dim))
            if x:
                self.append([b], x)

    def rows(self, *shape):
        return torch.randn(*shape, self.dim, generator=self.g, device="cuda").to(R.ROW_DTYPE[self.kind])

    def append(self, br, n):
        k, v = self.rows(len(br), n, self.kv), self.rows(len(br), n, self.kv)
        self.pool.append_kv(br, k, v)
        for i, b in enumerate(br):
            self.K[b] = np.concatenate((self.K[b], R.held(R.f64(k[i]), self.kind)))
            self.V[b] = np.concatenate((self.V[b], R.held(R.f64(v[i]), self.kind)))

    def fork(self, b, n):
        kids = self.pool.fork(b, n)
        for c in kids:
            self.K[c], self.V[c] = self.K[b], self.V[b]
        return kids

    def check(self, br, trees, out, q):
        for i, b in enumerate(br):
            t = trees[i] if isinstance(trees[0], (list, tuple)) else trees
            see = R.seen(t, len(self.K[b]) - len(t))
            ref = R.attention(R.f64(q[i]), self.K[b], self.V[b], see)
            err, bound = np.abs(R.f64(out[i]) - ref[0]), R.attention_bound(self.kind, *ref)
            assert (err <= bound).all(), (i, float(err.max()), float((err / bound).max()))

    def attend(self, br, trees, **kw):
        q = self.rows(len(br), self.new, self.nq)
        out = self.pool.tree_attn_draft(q, br, trees, **kw)
        self.pool.sync()
        self.check(br, trees, out, q)
        return q, out


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new", [1, 2, 7, 8, 16, 17, 33, 63, 64])
@pytest.mark.parametrize("kv,group", [(1, 1), (2, 4), (1, 8), (2, 5)])
def test_sizes(kind, new, kv, group):
    rng = random.Random(new)
    lens = [0, 1, 15, 16, 131]
    c = Case(kind, lens, new, kv, group, seed=new)
    c.append(c.br, new)
    c.attend(c.br, [R.tree(rng, new) for _ in lens])
    c.attend(c.br, R.tree(rng, new))          # one tree for all
    c.attend(c.br, R.tree(rng, new, "star"))
    c.pool.close()


@pytest.mark.parametrize("dim", [32, 96, 256])
def test_head_dims_of_fp32_pools(dim):
    rng = random.Random(dim)
    c = Case("fp32", [3, 40], 11, 2, 3, dim=dim)
    c.append(c.br, 11)
    c.attend(c.br, [R.tree(rng, 11) for _ in range(2)])
    c.pool.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new", [5, 20, 40])
def test_a_chain_is_the_causal_call(kind, new):
    c = Case(kind, [0, 33, 700], new, 2, 4)
    c.append(c.br, new)
    q, out = c.attend(c.br, R.tree(None, new, "chain"))
    same = c.pool.tree_attn_decode(q, c.br)
    err = np.abs(R.f64(out) - R.f64(same))
    for i, b in enumerate(c.br):     # both within the bound of the same answer
        ref = R.attention(R.f64(q[i]), c.K[b], c.V[b], R.seen(R.tree(None, new, "chain"), len(c.K[b]) - new))
        assert (err[i] <= 2 * R.attention_bound(kind, *ref)).all()
    c.pool.close()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("opts", [dict(tc_min_rows=-1), dict(tc_min_rows=1), dict(device_planning=1), dict(device_planning=-1),
                                  dict(pack_segments=-1), dict(fold_segments=-1), dict(tc_sms=8)])
def test_planning_options(kind, opts):
    """The kernels of every class, plans made on the host and on the device, packed and not."""
    rng = random.Random(7)
    c = Case(kind, [500, 37, 250], 9, 2, 4, **opts)
    kids = [x for b in c.br for x in c.fork(b, 3)]
    c.append(kids, 4)
    c.append(kids, 9)
    c.attend(kids, [R.tree(rng, 9) for _ in kids])
    c.attend(kids[::-1], R.tree(rng, 9))
    c.pool.close()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_wide_trees_over_a_shared_prefix(kind):
    """Hundreds of rows per kv head on shared blocks, drafted blocks of their own."""
    rng = random.Random(2)
    c = Case(kind, [900], 48, 2, 8)
    kids = c.fork(c.br[0], 5)
    c.append(kids, 48)
    c.attend(kids, [R.tree(rng, 48) for _ in kids])
    c.pool.close()


@pytest.mark.parametrize("kind", KINDS)
def test_trees_change_while_the_branches_do_not(kind):
    """The plan is kept from call to call: other trees, causal calls and appends between must not see its masks."""
    rng = random.Random(3)
    c = Case(kind, [60, 9, 200], 12, 2, 4)
    c.append(c.br, 12)
    first = [R.tree(rng, 12) for _ in c.br]
    q, out = c.attend(c.br, first)
    for trees in ([R.tree(rng, 12) for _ in c.br], R.tree(rng, 12), first):
        c.attend(c.br, trees)
    causal = c.pool.tree_attn_decode(q, c.br)
    assert torch.equal(c.pool.tree_attn_draft(q, c.br, first), out)
    assert torch.equal(c.pool.tree_attn_decode(q, c.br), causal)
    for n in (1, 2, 16, 40):      # lengths move: inside the tail block, then into new blocks
        c.append(c.br, n)
        c.attend(c.br, first)
    c.attend([c.br[2], c.br[0]], first[:2])
    c.pool.close()


@pytest.mark.parametrize("kind", KINDS)
def test_drafted_tokens_shared_by_children(kind):
    """Children forked behind the drafts read the same drafted blocks through trees of their own."""
    rng = random.Random(4)
    c = Case(kind, [70], 40, 2, 2)
    c.append(c.br, 40)
    kids = c.fork(c.br[0], 3)
    c.attend(kids + c.br, [R.tree(rng, 40) for _ in range(4)])
    c.pool.close()


def test_unseen_keys_that_are_not_finite():
    """A drafted key of NaN or infinity changes only the nodes that see it (values have to be finite)."""
    for kind in KINDS:
        c = Case(kind, [30], 6, 1, 2)
        k, v = c.rows(1, 6, 1), c.rows(1, 6, 1)
        k[0, 2] = float("nan")
        k[0, 4, 0, 0] = float("inf")
        c.pool.append_kv(c.br, k, v)
        out = R.f64(c.pool.tree_attn_draft(c.rows(1, 6, 2), c.br, [-1, 0, 0, 2, 1, 0]))[0]
        assert np.isfinite(out[[0, 1, 5]]).all(), kind
        assert not np.isfinite(out[[2, 3]]).any(), kind
        c.pool.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new", [1, 5, 16, 31, 64])
@pytest.mark.parametrize("layers", [1, 3])
def test_accept_keeps_rows_bit_for_bit(kind, new, layers):
    rng = random.Random(new)
    lens = [0, 3, 15, 16, 50]
    dt = R.ROW_DTYPE[kind]
    pool = Pool(128, 16, 2, 128, R.POOL_DTYPE[kind], max_branches=16, n_layers=layers)
    br = [pool.new_branch() for _ in lens]
    lead = (layers,) if layers > 1 else ()
    for b, x in zip(br, lens):
        if x:
            z = torch.randn(*lead, 1, x, 2, 128, device="cuda").to(dt)
            pool.append_kv([b], z, z)
    K, V = (torch.randn(*lead, len(lens), new, 2, 128, device="cuda").to(dt) for _ in range(2))
    pool.append_kv(br, K, V)
    trees = [R.tree(rng, new) for _ in lens]
    keep = [R.path_to(t, rng.randrange(new)) for t in trees]
    keep[1] = []
    keep[2] = list(range(new))               # nothing moves
    before = [[pool.read_kv([b], [0], [lens[i] + new], layer=l) for l in range(layers)] for i, b in enumerate(br)]
    pool.accept_draft(br, new, keep)
    for i, b in enumerate(br):
        assert pool.branch_len(b) == lens[i] + len(keep[i])
        rows = list(range(lens[i])) + [lens[i] + j for j in keep[i]]
        for l in range(layers):
            got = pool.read_kv([b], [0], [len(rows)], layer=l)
            for x, y in zip(got, before[i][l]):
                assert torch.equal(x, y[rows])
    held = sum((lens[i] + len(k) + 15) // 16 for i, k in enumerate(keep))
    assert sum(pool.read_refcounts()) == held
    pool.free(br)
    assert sum(pool.read_refcounts()) == 0
    pool.close()


@pytest.mark.parametrize("kind", KINDS)
def test_accept_beside_branches_that_share(kind):
    """Siblings that share a half-full tail draft and accept on their own; the parent's rows and the other
    siblings' stay.  What would move rows in shared blocks is refused."""
    rng = random.Random(5)
    c = Case(kind, [23], 9, 2, 2)
    root = c.br[0]
    kids = c.fork(root, 3)
    c.append(kids, 9)
    trees = [R.tree(rng, 9) for _ in kids]
    keep = [[0, 3, 8], [1], [2, 5, 6, 7]]
    c.pool.accept_draft(kids, 9, keep)
    for i, b in enumerate(kids):
        rows = list(range(23)) + [23 + j for j in keep[i]]
        c.K[b], c.V[b] = c.K[b][rows], c.V[b][rows]
    for b in kids + [root]:
        k, v = c.pool.read_kv([b], [0], [len(c.K[b])])
        assert np.array_equal(R.f64(k), c.K[b]) and np.array_equal(R.f64(v), c.V[b])
    # a next step on top
    c.append(kids, 9)
    c.attend(kids, trees)
    # forked behind the base: rows may not move, a prefix of the drafts may be kept
    grand = c.fork(kids[0], 1)[0]
    with pytest.raises(DendriteError):
        c.pool.accept_draft([kids[0]], 9, [[1]])
    with pytest.raises(DendriteError):
        c.pool.accept_draft([grand], 9, [[1]])
    assert c.pool.branch_len(kids[0]) == len(c.K[kids[0]])
    c.pool.accept_draft([kids[0]], 9, [[0, 1]])
    k, _ = c.pool.read_kv([grand], [0], [len(c.K[grand])])
    assert np.array_equal(R.f64(k), c.K[grand])
    # once the child is gone the branch's rows are its own again
    c.append([kids[1]], 1)
    g2 = c.fork(kids[1], 2)
    c.pool.free(g2)
    c.pool.accept_draft([kids[1]], 10, [[9]])
    rows = list(range(len(c.K[kids[1]]) - 10)) + [len(c.K[kids[1]]) - 1]
    k, v = c.pool.read_kv([kids[1]], [0], [len(rows)])
    assert np.array_equal(R.f64(k), c.K[kids[1]][rows]) and np.array_equal(R.f64(v), c.V[kids[1]][rows])
    c.pool.close()


def test_accept_of_many_branches():
    # more arguments than travel as kernel parameters
    rng = random.Random(6)
    n, new = 150, 60
    pool = Pool(n * 8, 16, 1, 128, torch.bfloat16, max_branches=n + 1)
    br = [pool.new_branch() for _ in range(n)]
    K = torch.randn(n, new, 1, 128, device="cuda").bfloat16()
    pool.append_kv(br, K, K)
    keep = [sorted(rng.sample(range(new), rng.randint(0, new))) for _ in range(n)]
    pool.accept_draft(br, new, keep)
    k, v = pool.read_kv(br, [0] * n, [len(x) for x in keep])
    want = torch.cat([K[i, x] for i, x in enumerate(keep)])
    assert torch.equal(k, want) and torch.equal(v, want)
    pool.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
def test_steps_of_speculative_decoding(kind, interleaved):
    """Drafts appended at their depths' positions, attended, one path accepted, again and again: keys, values
    and outputs against a 64-bit cache that is kept beside the pool's own rounding."""
    rng = random.Random(8)
    c = Case(kind, [40, 7, 0], 12, 2, 4)
    rope = Rope(64, interleaved=interleaved, scaling="linear", factor=2.0)
    freq, m = R.frequencies(64, 10000.0, "linear", 2.0)
    for step in range(4):
        trees = [R.tree(rng, 12) for _ in c.br]
        k, v, q = c.rows(3, 12, 2), c.rows(3, 12, 2), c.rows(3, 12, 8)
        tq = c.pool.append_rope(c.br, k, v, rope, Q=q, parents=trees)
        base = [len(c.K[b]) for b in c.br]
        for i, b in enumerate(c.br):
            pos = base[i] + np.array(R.depths(trees[i]))
            y, size = R.rotate(R.f64(q[i]), pos, freq, 64, interleaved, m)
            half = {"fp32": 2.0 ** -24}.get(kind, 2.0 ** -8)
            assert (np.abs(R.f64(tq[i]) - y) <= R.ROPE_ERR * size + half * (np.abs(y) + R.ROPE_ERR * size) + 1e-38).all()
            got = c.pool.read_kv([b], [base[i]], [12])
            y, size = R.rotate(R.f64(k[i]), pos, freq, 64, interleaved, m)
            # the stored keys themselves are checked in the append's own tests: near, and then taken as they are
            assert np.abs(R.f64(got[0]) - y).max() <= 2.0 ** -3 * np.abs(y).max()
            assert np.array_equal(R.f64(got[1]), R.held(R.f64(v[i]), kind))
            c.K[b] = np.concatenate((c.K[b], R.f64(got[0])))
            c.V[b] = np.concatenate((c.V[b], R.f64(got[1])))
        out = c.pool.tree_attn_draft(tq, c.br, trees)
        c.check(c.br, trees, out, tq)
        keep = [R.path_to(t, rng.randrange(12)) for t in trees]
        c.pool.accept_draft(c.br, 12, keep)
        for i, b in enumerate(c.br):
            rows = list(range(base[i])) + [base[i] + j for j in keep[i]]
            c.K[b], c.V[b] = c.K[b][rows], c.V[b][rows]
            got = c.pool.read_kv([b], [0], [len(rows)])
            assert np.array_equal(R.f64(got[0]), c.K[b]) and np.array_equal(R.f64(got[1]), c.V[b])
    # the accepted rows stand as an ordinary decode sees them
    q = c.rows(3, 1, 8)
    c.append(c.br, 1)
    out = c.pool.tree_attn_decode(q, c.br)
    c.check(c.br, [[-1]] * 3, out, q)
    c.pool.sync()
    c.pool.close()


def test_layers_of_a_step():
    """Several layers: one plan, the drafts turned layer by layer, accepted in all of them."""
    rng = random.Random(9)
    pool = Pool(64, 16, 2, 128, torch.float8_e4m3fn, max_branches=8, n_layers=3)
    br = [pool.new_branch() for _ in range(2)]
    x = torch.randn(3, 2, 21, 2, 128, device="cuda").bfloat16()
    pool.append_kv(br, x, x)
    trees = [R.tree(rng, 10) for _ in br]
    k, v = (torch.randn(3, 2, 10, 2, 128, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(3, 2, 10, 8, 128, device="cuda").bfloat16()
    pool.append_begin(br, 10)
    for l in range(3):
        tq = pool.append_layer_rope(l, k[l].contiguous(), v[l].contiguous(), Rope(128), Q=q[l].contiguous(), parents=trees)
        out = pool.tree_attn_draft(tq, br, trees, layer=l)
        if l < 2:
            with pytest.raises(DendriteError):
                pool.tree_attn_draft(tq, br, trees, layer=2)
            with pytest.raises(DendriteError):
                pool.accept_draft(br, 10, [[0], [0]])
        for i, b in enumerate(br):
            K, V = (R.f64(t) for t in pool.read_kv([b], [0], [31], layer=l))
            ref = R.attention(R.f64(tq[i]), K, V, R.seen(trees[i], 21))
            assert (np.abs(R.f64(out[i]) - ref[0]) <= R.attention_bound("fp8", *ref)).all()
    before = [[pool.read_kv([b], [0], [31], layer=l) for l in range(3)] for b in br]
    pool.accept_draft(br, 10, [R.path_to(t, 9) for t in trees])
    for i, b in enumerate(br):
        rows = list(range(21)) + [21 + j for j in R.path_to(trees[i], 9)]
        for l in range(3):
            assert all(torch.equal(a, w[rows]) for a, w in zip(pool.read_kv([b], [0], [len(rows)], layer=l), before[i][l]))
    pool.close()


def test_refusals():
    c = Case("bf16", [20, 20], 4, 2, 2)
    c.append(c.br, 4)
    q = c.rows(2, 4, 4)
    for trees in (None, [-1, 0, 1], [-1, 0, 2, 1], [-1, 0, 1, 3], [[-1, 0, 1, 2]] * 3, [-2, 0, 0, 0]):
        with pytest.raises(DendriteError):
            c.pool.tree_attn_draft(q, c.br, trees)
    long = c.rows(2, 65, 4)
    c.append(c.br, 61)
    with pytest.raises(DendriteError):
        c.pool.tree_attn_draft(long, c.br, list(range(-1, 64)))
    short = c.pool.new_branch()
    with pytest.raises(DendriteError):      # fewer tokens than drafts
        c.pool.tree_attn_draft(q[:1].contiguous(), [short], [-1, 0, 0, 0])
    with pytest.raises(DendriteError):
        c.pool.tree_attn_draft(q, [c.br[0], c.br[0]], [-1, 0, 0, 0])
    for keep in ([[0], [4]], [[0], [-1]], [[1, 1], [0]], [[2, 1], [0]], [[0]], [[0, 1, 2, 3, 4], []]):
        with pytest.raises(DendriteError):
            c.pool.accept_draft(c.br, 4, keep)
    with pytest.raises(DendriteError):
        c.pool.accept_draft(c.br, 65, [[0], [0]])
    with pytest.raises(DendriteError):
        c.pool.accept_draft([c.br[0], c.br[0]], 4, [[0], [0]])
    with pytest.raises(DendriteError):
        c.pool.accept_draft([short], 4, [[0]])
    assert [c.pool.branch_len(b) for b in c.br] == [85, 85]
    c.pool.accept_draft(c.br, 0, [[], []])
    c.pool.accept_draft([], 4, [])
    assert [c.pool.branch_len(b) for b in c.br] == [85, 85]
    c.pool.sync()
    c.pool.close()


@pytest.mark.parametrize("kind,new,decode_tc,draft_tc", [("bf16", 4, False, False), ("bf16", 5, False, True), ("bf16", 16, False, True),
                                                         ("bf16", 17, True, True), ("fp8", 8, False, False), ("fp8", 9, True, True)])
def test_rows_per_head_choose_the_kernel(kind, new, decode_tc, draft_tc):
    """4 rows per drafted token: the tcgen05 kernel from the documented rows on, for each kind of call, and for each its own."""
    rng = random.Random(11)
    c = Case(kind, [100, 33, 7], new, 2, 4)
    c.append(c.br, new)
    q = torch.randn(len(c.br), new, 8, 128, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):      # a draft call after a decode call of the same rows, and the other way round
        c.pool.tree_attn_decode(q, c.br)
        assert (c.pool.last_plan_stats()["n_tc_units"] > 0) == decode_tc
        c.attend(c.br, [R.tree(rng, new) for _ in c.br])
        assert (c.pool.last_plan_stats()["n_tc_units"] > 0) == draft_tc
    c.pool.close()


@pytest.mark.parametrize("kind,blocks", [("fp8", 270_000), ("bf16", 136_000)])
def test_offsets_past_32_bits(kind, blocks):
    """A step on blocks more than 4 GiB into the pools gives what it gives on the first ones."""
    g = torch.Generator(device="cuda").manual_seed(9)
    kv, nq, new = 8, 32, 20
    x = torch.randn(1, 65536, kv, 128, generator=g, device="cuda").bfloat16()
    q = torch.randn(1, new, nq, 128, generator=g, device="cuda").bfloat16()
    parents = R.tree(random.Random(5), new)
    path, j = [], new - 1
    while j >= 0:
        path, j = [j] + path, parents[j]
    results = []
    for filled in (0, blocks):
        pool = Pool(filled + 64, 16, kv, 128, R.POOL_DTYPE[kind], max_branches=256)
        for lo in range(0, filled, 4096):
            pool.append_kv([pool.new_branch()], *[x[:, :16 * min(4096, filled - lo)].contiguous()] * 2)
        b = pool.new_branch()
        pool.append_kv([b], x[:, :333].contiguous(), x[:, 333:666].contiguous())
        turned = pool.append_rope([b], x[:, :new].contiguous(), x[:, new:2 * new].contiguous(), Rope(128), Q=q, parents=parents)
        out = pool.tree_attn_draft(turned, [b], parents)
        pool.accept_draft([b], new, [path])
        one = pool.tree_attn_decode(q[:, :1].contiguous(), [b])
        if filled:
            assert min(pool.read_table(b)[:20]) >= filled
        results.append([turned, out, one, *pool.read_kv([b], [0], [333 + len(path)])])
        pool.sync()
        pool.close()
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("kind", KINDS)
def test_the_most_rows_of_a_tree(kind):
    """64 drafted tokens of 64 query heads a kv head: 4,096 rows, many units of every kernel."""
    rng = random.Random(4)
    c = Case(kind, [50, 3], 64, 1, 64)
    c.append(c.br, 64)
    c.attend(c.br, [R.tree(rng, 64) for _ in c.br])
    c.pool.close()
