"""What a block still holds behind a branch's end (left by its last owner, by a
roll-back or by an acceptance) touches no output: with rows there that are not
finite, every attention call gives the bits it gives over a pool whose blocks were
never used before."""
import random

import pytest
import torch

import _rows as R
from copy_write_forked_gb300.dendrite import Pool, Rope
from copy_write_forked_gb300.workloads import turbo_codec

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "fp8", "fp32"]
KV, D = 2, 128


def new_pool(kind, blocks, **kw):
    if kind == "turbo":
        return Pool(blocks, 16, KV, D, torch.bfloat16, turbo=turbo_codec(), **kw)
    return Pool(blocks, 16, KV, D, R.POOL_DTYPE[kind], **kw)


def row_dtype(kind):
    return torch.bfloat16 if kind == "turbo" else R.ROW_DTYPE[kind]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()
    torch.cuda.set_device(0)


class Pools:
    """The same calls on a pool of untouched blocks and on one whose every block holds `fill`."""

    def __init__(self, kind, blocks, fill, **kw):
        self.dtype = row_dtype(kind)
        self.turbo = kind == "turbo"
        self.fill = fill
        self.pools = [new_pool(kind, blocks, max_branches=64, **kw) for _ in range(2)]
        self.g = torch.Generator(device="cuda").manual_seed(3)
        p = self.pools[1]
        b = p.new_branch()
        x = self.junk(blocks * 16)
        p.append_kv([b], x, x)
        p.free([b])

    def junk(self, n, branches=1):
        return torch.full((branches, n, KV, D), self.fill, dtype=self.dtype, device="cuda")

    def rows(self, *shape):
        return torch.randn(*shape, D, generator=self.g, device="cuda").to(self.dtype)

    def new(self):
        a, b = (p.new_branch() for p in self.pools)
        assert a == b
        return a

    def each(self, name, *args, **kw):
        return [getattr(p, name)(*args, **kw) for p in self.pools][0]

    def append(self, br, n):
        k, v = self.rows(len(br), n, KV), self.rows(len(br), n, KV)
        self.each("append_kv", br, k, v)

    def leave(self, br, n):
        """n rows appended and rolled back: in the used pool they are junk."""
        for p, x in zip(self.pools, (torch.zeros_like(self.junk(n, len(br))), self.junk(n, len(br)))):
            p.append_kv(br, x, x)
            if self.turbo:
                p.truncate(br, [p.branch_len(b) - n for b in br])
            else:
                p.accept_draft(br, n, [[] for _ in br])

    def same(self, name, *args, **kw):
        a, b = (getattr(p, name)(*args, **kw) for p in self.pools)
        for p in self.pools:
            p.sync()
        assert torch.isfinite(a).all() and torch.equal(a, b)

    def attend(self, br, group, q_len, **kw):
        self.same("tree_attn_decode", self.rows(len(br), q_len, KV * group), br, **kw)

    def close(self):
        for p in self.pools:
            p.close()


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("rows", [-1, 1])
@pytest.mark.parametrize("group,q_len", [(1, 1), (4, 5), (8, 3), (16, 4), (8, 30), (16, 17)])
@pytest.mark.parametrize("kind", KINDS + ["turbo"])
def test_last_owners_and_roll_backs(kind, group, q_len, rows, fill):
    """Row groups of 1 to 272 rows: every row tile of both kernels; ends at each place in a stage of four tiles."""
    p = Pools(kind, 40, fill, tc_min_rows=rows)
    b = p.new()
    for n in (30, 1, 16, 15, 2, 49, 70):     # ends at 30, 31, 47, 62, 64, 113, 183
        p.append([b], n)
        p.attend([b], group, q_len)
        p.leave([b], 21)
        p.attend([b], group, q_len)
        c = p.each("fork", b, 1)             # a copied tail
        p.append(c, 1)
        p.attend(c, group, q_len)
        p.each("free", c)
    p.close()


@pytest.mark.parametrize("opts", [dict(), dict(pack_segments=1_000_000, tc_min_rows=8), dict(pack_segments=1_000_000, tc_min_rows=-1),
                                  dict(pack_segments=-1), dict(fold_segments=1_000_000), dict(device_planning=1)])
@pytest.mark.parametrize("width,q_len", [(3, 1), (7, 2), (5, 9)])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "turbo"])
def test_forks_of_one_prefix(kind, width, q_len, opts):
    """Leaves of 1 to 40 tokens behind a prefix: extra tiles of a packed segment end in them."""
    p = Pools(kind, 60 + 8 * width, float("nan"), **opts)
    root = p.new()
    p.append([root], 16 * 13)
    kids = p.each("fork", root, width)
    for i, k in enumerate(kids):
        p.append([k], 9 + (11 * i) % 32)
        p.leave([k], 5)
    p.attend(kids, 4, q_len)
    p.append(kids, 3)                        # lengths refreshed, segments grown
    p.attend(kids, 4, q_len)
    p.each("free", kids[:1])
    p.attend(kids[1:], 4, q_len)
    p.close()


@pytest.mark.parametrize("rows", [-1, 0, 1])
@pytest.mark.parametrize("new", [1, 6, 17, 45])
@pytest.mark.parametrize("kind", KINDS)
def test_draft_trees(kind, new, rows):
    rng = random.Random(new)
    p = Pools(kind, 80, float("nan"), tc_min_rows=rows)
    br = [p.new() for _ in range(3)]
    for b, n in zip(br, (5, 40, 111)):
        p.append([b], n)
    for _ in range(3):
        trees = [R.tree(rng, new) for _ in br]
        p.append(br, new)
        p.same("tree_attn_draft", p.rows(3, new, KV * 4), br, trees)
        p.each("accept_draft", br, new, [R.path_to(t, new // 2) for t in trees])
        p.leave(br, 4)
        p.attend(br, 4, 1)
    p.close()


@pytest.mark.parametrize("rolled_back", [False, True])
@pytest.mark.parametrize("rows", [-1, 1])
@pytest.mark.parametrize("kind", KINDS)
def test_the_allocation_free_call(kind, rows, rolled_back):
    p = Pools(kind, 20, float("nan"), tc_min_rows=rows)
    b = p.new()
    p.append([b], 37)
    if rolled_back:
        p.leave([b], 9)
    q = p.rows(1, 1, KV * 4)
    outs = [torch.zeros_like(q) for _ in range(2)]
    for pool, o in zip(p.pools, outs):
        pool.tree_attn_decode_noalloc(q, [b], o)
        pool.sync()
    assert torch.isfinite(outs[0]).all() and torch.equal(*outs)
    p.close()


@pytest.mark.parametrize("kind,how", [(k, h) for k in KINDS + ["turbo"] for h in ("kv", "rope", "layers", "layers_rope")
                                      if k != "turbo" or "rope" not in h])   # compressed pools do not rotate
def test_every_way_of_appending(kind, how):
    """Junk brought in by, and written over by, each kind of append, in every layer."""
    layers, dt, rope = 2, row_dtype(kind), Rope(D)
    g = torch.Generator(device="cuda").manual_seed(5)
    rows = lambda *s: torch.randn(*s, D, generator=g, device="cuda").to(dt)  # noqa: E731

    def append(p, br, k, v):
        if how == "kv":
            p.append_kv(br, k, v)
        elif how == "rope":
            p.append_rope(br, k, v, rope)
        else:
            p.append_begin(br, k.shape[2])
            for y in range(layers):
                if how == "layers":
                    p.append_layer(y, k[y], v[y])
                else:
                    p.append_layer_rope(y, k[y], v[y], rope)

    data = {n: (rows(layers, 1, n, KV), rows(layers, 1, n, KV)) for n in (37, 3, 1, 9)}
    q = rows(1, 2, KV * 4)
    outs = []
    for junk in (False, True):
        p = new_pool(kind, 8, max_branches=8, n_layers=layers)
        if junk:
            b = p.new_branch()
            k = rows(layers, 1, 128, KV) * 0
            append(p, [b], k, torch.full_like(k, float("nan")))
            p.free([b])
        out = []

        def attend(b):
            out.extend(p.tree_attn_decode(q, [b], layer=y) for y in range(layers))

        b = p.new_branch()
        append(p, [b], *data[37])     # new blocks
        attend(b)
        append(p, [b], *data[3])      # in place
        attend(b)
        c = p.fork(b, 1)[0]
        append(p, [c], *data[1])      # a copied tail
        attend(c)
        attend(b)
        append(p, [b], *data[9])      # in place again, into the next block
        attend(b)
        p.sync()
        outs.append(torch.stack(out))
        p.close()
    assert torch.isfinite(outs[0]).all() and torch.equal(*outs)


def test_large_values_behind_a_branch_of_a_compressed_pool():
    """Its weights are kept in units of the largest value's size: one that nothing sees has no say in them."""
    p = Pools("turbo", 8, 1e30)
    b = p.new()
    p.append([b], 37)
    p.attend([b], 4, 1)
    p.leave([b], 4)
    p.attend([b], 4, 3)
    p.close()
