"""Appends with rotary positions through the C-ABI library: queries and stored keys
against 64 bits within what fp32 angles and products and one rounding allow, values
untouched, tables as a plain append leaves them."""
import random

import numpy as np
import pytest
import torch

import _rows as R
from copy_write_forked_gb300.dendrite import DendriteError, Pool, Rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()
    torch.cuda.set_device(0)


def _close(kind, got, y, size, stored):
    """got against the turned rows y: fp32 error, then the rounding of where it is stored."""
    err = np.abs(got - y)
    slack = R.ROPE_ERR * size
    if stored and kind == "fp8":
        # the row's exponent may be the next one where its largest element is within the
        # fp32 error of a border: a step is 2^-3 of a value, or of 2^-6 of the scale
        top = (np.abs(y) + slack).max(-1, keepdims=True)
        e = np.ceil(np.log2(np.maximum(top, 1e-300) / 448))
        half = np.maximum(2.0 ** -4 * (np.abs(y) + slack), 2.0 ** (e - 10))
        bound = slack + half
    else:
        bound = slack + {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp8": 2.0 ** -8}[kind] * (np.abs(y) + slack)
    assert (err <= bound + 1e-38).all(), float((err / (bound + 1e-38)).max())


def _case(kind, dim, rot, interleaved, scaling, kv, nq, lens, new, trees, seed=0, layers=1, in_place=False, split=False):
    dt, rows = R.POOL_DTYPE[kind], R.ROW_DTYPE[kind]
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = len(lens)
    pool = Pool(sum((x + new) // 16 + 3 for x in lens) + 8, 16, kv, dim, dt, max_branches=n + 8, n_layers=layers,
                max_blocks_per_branch=(max(lens) + new) // 16 + 2)
    lead = (layers,) if layers > 1 else ()
    br = [pool.new_branch() for _ in lens]
    for b, x in zip(br, lens):
        if x:
            z = torch.randn(*lead, 1, x, kv, dim, generator=g, device="cuda").to(rows)
            pool.append_kv([b], z, z)
    kw = dict(base=500000.0, factor=4.0, original_len=8192.0)
    rope = Rope(rot, interleaved=interleaved, scaling=scaling, **kw)
    freq, m = R.frequencies(rot, 500000.0, scaling, 4.0, 8192.0)
    K, V = (torch.randn(*lead, n, new, kv, dim, generator=g, device="cuda").to(rows) for _ in range(2))
    Q = torch.randn(*lead, n, new, nq, dim, generator=g, device="cuda").to(rows) if nq else None
    q64, k64, v64 = (R.f64(x).reshape(layers, n, new, -1, dim) if x is not None else None for x in (Q, K, V))
    parents = None if trees is None else torch.tensor(trees, dtype=torch.int32)
    if split:
        pool.append_begin(br, new)
        outs = [pool.append_layer_rope(l, K[l].contiguous(), V[l].contiguous(), rope, Q=Q[l].contiguous() if nq else None,
                                       parents=parents) for l in range(layers)]
        out = torch.stack(outs) if nq else None
    else:
        out = pool.append_rope(br, K, V, rope, Q=Q, parents=parents, out=Q if in_place else None)
    pool.sync()
    for i in range(n):
        if trees is None:
            pos = lens[i] + np.arange(new)
        else:
            pos = lens[i] + np.array(R.depths(trees[i] if isinstance(trees[0], list) else trees))
        for l in range(layers):
            if nq:
                y, size = R.rotate(q64[l, i], pos, freq, rot, interleaved, m)
                _close(kind, R.f64(out).reshape(layers, n, new, nq, dim)[l, i], y, size, False)
                assert rot == dim or np.array_equal(R.f64(out).reshape(layers, n, new, nq, dim)[l, i][..., rot:], q64[l, i][..., rot:])
            k, v = pool.read_kv([br[i]], [lens[i]], [new], layer=l)
            y, size = R.rotate(k64[l, i], pos, freq, rot, interleaved, m)
            _close(kind, R.f64(k), y, size, True)
            assert np.array_equal(R.f64(v), R.held(v64[l, i], kind))
        assert pool.branch_len(br[i]) == lens[i] + new
    pool.close()


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("fp8", 128), ("fp32", 128), ("fp32", 32), ("fp32", 96), ("fp32", 256)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", ["all", "half", 16])
def test_types_and_layouts(kind, dim, interleaved, rot):
    rot = {"all": dim, "half": dim // 2}.get(rot, rot)
    _case(kind, dim, rot, interleaved, "none", 2, 6, [0, 5, 31], 19, None, seed=dim + rot)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
@pytest.mark.parametrize("new", [1, 2, 3, 15, 16, 17, 40])
@pytest.mark.parametrize("kv,nq", [(1, 0), (1, 7), (3, 3), (8, 32)])
def test_sizes(kind, new, kv, nq):
    _case(kind, 128, 128, False, "none", kv, nq, [0, 1, 15, 16, 100], new, None, seed=new)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "bands"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(scaling, interleaved):
    # angles of 60,000 radians, whose fp32 product alone would be off by 2^-9
    _case("fp32", 64, 64, interleaved, scaling, 1, 2, [60011, 7, 32768], 5, None, seed=3)
    _case("bf16", 128, 64, interleaved, scaling, 1, 2, [40007], 18, None, seed=4)


def test_far_positions_by_large_frequencies():
    # positions near 2^30 as frequencies: a whole turn more or less changes nothing at whole positions
    pool = Pool(16, 16, 1, 128, torch.float32, max_branches=4)
    b = pool.new_branch()
    x = torch.randn(1, 20, 1, 128, device="cuda")
    f = [2 * np.pi * 10 ** 6 + 0.125 * i for i in range(16)] + [-0.5] * 48
    rope = Rope(128, inv_freq=f)
    pool.append_rope([b], x, x, rope)
    k, _ = pool.read_kv([b], [0], [20])
    y, size = R.rotate(R.f64(x[0]), np.arange(20), [0.125 * i for i in range(16)] + [-0.5] * 48, 128, False)
    # 2 pi 10^6 as a double is off by 2^-31 radians per position at most, 20 positions
    assert (np.abs(R.f64(k) - y) <= R.ROPE_ERR * size + 2.0 ** -24 * np.abs(y) + 20 * 2.0 ** -30 * size).all()
    pool.close()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
@pytest.mark.parametrize("new", [1, 2, 9, 33, 64])
@pytest.mark.parametrize("shape", ["random", "chain", "star"])
@pytest.mark.parametrize("shared", [False, True])
def test_draft_trees(kind, new, shape, shared):
    rng = random.Random(new)
    lens = [3, 0, 16, 77]
    trees = R.tree(rng, new, shape) if shared else [R.tree(rng, new, shape) for _ in lens]
    _case(kind, 128, 128, False, "none", 2, 4, lens, new, trees, seed=new)


def test_many_branches():
    # more arguments than travel as kernel parameters, trees among them
    rng = random.Random(0)
    lens = [i % 37 for i in range(600)]
    _case("bf16", 128, 128, False, "none", 1, 2, lens, 3, None)
    _case("fp8", 128, 64, True, "none", 1, 1, lens[:200], 40, [R.tree(rng, 40) for _ in range(200)])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
def test_layers_in_place_and_split(kind):
    tree = [-1, 0, 0, 1, 1]
    _case(kind, 128, 128, False, "none", 2, 4, [9, 20], 5, tree, layers=3)
    _case(kind, 128, 64, True, "none", 2, 4, [9, 20], 5, None, layers=3, in_place=True)
    _case(kind, 128, 128, False, "none", 2, 4, [9, 20], 5, tree, layers=3, split=True)
    _case(kind, 128, 128, False, "none", 2, 0, [9, 20], 5, None, layers=2, split=True)
    _case(kind, 128, 128, False, "yarn", 2, 8, [9, 20, 0], 21, None, in_place=True)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
def test_copy_on_write_keeps_the_older_rows(kind):
    """Children of a half-full tail: each turns its own token, the shared rows stay as they were, and
    tables and refcounts are those of a plain append."""
    rows = R.ROW_DTYPE[kind]
    pools = [Pool(64, 16, 2, 128, R.POOL_DTYPE[kind], max_branches=16) for _ in range(2)]
    rope = Rope(128)
    x = torch.randn(1, 23, 2, 128, device="cuda").to(rows)
    y = torch.randn(3, 2, 2, 128, device="cuda").to(rows)
    state = []
    for turned, pool in zip((True, False), pools):
        root = pool.new_branch()
        pool.append_kv([root], x, x)
        kids = pool.fork(root, 3)
        pool.free([root])
        if turned:
            pool.append_rope(kids, y, y, rope)
        else:
            pool.append_kv(kids, y, y)
        state.append(([pool.read_table(b) for b in kids], pool.read_refcounts(), pool.read_free_stack()))
        k, v = pool.read_kv(kids, [0] * 3, [25] * 3)
        old = R.held(R.f64(x[0]), kind)
        for i in range(3):
            assert np.array_equal(R.f64(k)[25 * i:25 * i + 23], old) and np.array_equal(R.f64(v)[25 * i:25 * i + 23], old)
            if turned:
                t, size = R.rotate(R.f64(y[i]), 23 + np.arange(2), R.frequencies(128)[0], 128, False)
                _close(kind, R.f64(k)[25 * i + 23:25 * i + 25], t, size, True)
            assert np.array_equal(R.f64(v)[25 * i + 23:25 * i + 25], R.held(R.f64(y[i]), kind))
    assert state[0] == state[1]
    for p in pools:
        p.close()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
@pytest.mark.parametrize("how", ["append", "rope", "split"])
def test_branches_of_different_lengths_in_one_shared_tail(kind, how):
    """Siblings of a half-full tail, one of them rolled back inside it, appended to in one call: the one served last
    writes in place and must not overwrite what the others still have to copy.  Tables are those of one call each."""
    rows = R.ROW_DTYPE[kind]
    g = torch.Generator(device="cuda").manual_seed(3)
    layers, kv = (2, 8) if how == "split" else (1, 8)
    x = torch.randn(layers, 1, 44, kv, 128, generator=g, device="cuda").to(rows)
    y = torch.randn(layers, 9, 20, kv, 128, generator=g, device="cuda").to(rows)
    for cut in (33, 40, 43):
        state = []
        for one_call in (True, False):
            pool = Pool(128, 16, kv, 128, R.POOL_DTYPE[kind], max_branches=16, n_layers=layers)
            root = pool.new_branch()
            pool.append_kv([root], *[x if layers > 1 else x[0]] * 2)
            kids = pool.fork(root, 8)
            pool.free([root])
            pool.truncate([kids[3]], [cut])
            order = kids[:3] + kids[4:] + pool.fork(kids[3], 1) + [kids[3]]   # the shortest hold the block last
            for br in ([order] if one_call else [[b] for b in order]):
                at = [order.index(b) for b in br]
                new = y[:, at].contiguous()
                if how == "split":
                    pool.append_begin(br, 20)
                    for layer in range(layers):
                        pool.append_layer(layer, new[layer], new[layer])
                elif how == "rope":
                    pool.append_rope(br, new[0], new[0], Rope(128))
                else:
                    pool.append_kv(br, new[0], new[0])
            state.append(([pool.read_table(b) for b in order], pool.read_refcounts(), pool.read_free_stack()))
            for layer in range(layers):
                lens = [pool.branch_len(b) for b in order]
                k, v = (R.f64(z) for z in pool.read_kv(order, [0] * 9, lens, layer=layer))
                for i, n in enumerate(lens):
                    old, start = R.held(R.f64(x[layer, 0]), kind)[:n - 20], sum(lens[:i])
                    assert np.array_equal(k[start:start + n - 20], old) and np.array_equal(v[start:start + n - 20], old), (cut, i)
                    assert np.array_equal(v[start + n - 20:start + n], R.held(R.f64(y[layer, i]), kind))
            pool.close()
        assert state[0] == state[1]


def test_another_stream_and_two_calls_at_once():
    pools = [Pool(64, 16, 4, 128, torch.bfloat16, max_branches=8) for _ in range(2)]
    rope = Rope(128)
    x = torch.randn(4, 50, 4, 128, device="cuda").bfloat16()
    q = torch.randn(4, 50, 16, 128, device="cuda").bfloat16()
    torch.cuda.synchronize()
    outs, reads = [], []
    for p in pools:
        s = torch.cuda.Stream()
        br = [p.new_branch() for _ in range(4)]
        out = torch.empty_like(q)
        p.append_rope(br, x, x, rope, Q=q, out=out, stream=s)
        outs.append(out)
        with torch.cuda.stream(s):
            reads.append(p.read_kv(br, [0] * 4, [50] * 4))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(reads[0][0], reads[1][0])
    y, size = R.rotate(R.f64(q[1]), np.arange(50), R.frequencies(128)[0], 128, False)
    _close("bf16", R.f64(outs[0][1]), y, size, False)
    for p in pools:
        p.close()


def test_rows_that_are_not_finite_stay_in_their_row():
    x = torch.randn(1, 4, 1, 128, device="cuda").bfloat16()
    x[0, 1, 0, 5] = float("inf")
    x[0, 2, 0, 9] = float("nan")
    for kind in ("bf16", "fp8"):
        pool = Pool(8, 16, 1, 128, R.POOL_DTYPE[kind], max_branches=4)
        b = pool.new_branch()
        pool.append_rope([b], x, torch.zeros_like(x), Rope(128))
        k = R.f64(pool.read_kv([b], [0], [4])[0])[:, 0]
        assert np.isfinite(k[[0, 3]]).all()
        for row, col in ((1, 5), (2, 9)):
            bad = np.flatnonzero(~np.isfinite(k[row])).tolist()
            assert bad == list(range(128)) if kind == "fp8" else set(bad) <= {col, col + 64} and bad
        pool.close()


def test_refusals():
    pool = Pool(64, 16, 2, 128, torch.bfloat16, max_branches=8)
    b = pool.new_branch()
    x = torch.zeros(1, 4, 2, 128, device="cuda", dtype=torch.bfloat16)
    q = torch.zeros(1, 4, 8, 128, device="cuda", dtype=torch.bfloat16)
    r = Rope(128)
    flat = torch.zeros(2 * q.numel(), device="cuda", dtype=torch.bfloat16)
    bad = [dict(rope=Rope(256)), dict(Q=q.float()), dict(Q=q[:, :3].contiguous()), dict(out=q[:, :, :4].contiguous(), Q=q),
           dict(parents=[-1, 0, 1]), dict(parents=[-1, 1, 0, 0]), dict(parents=[-2, 0, 0, 0]), dict(parents=[[-1] * 4] * 2),
           dict(Q=flat[:q.numel()].view_as(q), out=flat[64:64 + q.numel()].view_as(q)), dict(V=x[:, :3].contiguous()), dict(rope=None),
           dict(Q=q.cpu())]
    for kw in bad:
        a = dict(K=x, V=x, rope=r) | kw
        with pytest.raises(DendriteError):
            pool.append_rope([b], a.pop("K"), a.pop("V"), a.pop("rope"), **a)
        assert pool.branch_len(b) == 0
    long = torch.zeros(1, 65, 2, 128, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(DendriteError):
        pool.append_rope([b], long, long, r, parents=list(range(-1, 64)))
    pool.append_rope([b], long, long, r)   # without a tree any length goes
    for attr, val in (("rot_dim", 24), ("interleaved", 2), ("scale", float("inf"))):
        broken = Rope(128)
        setattr(broken._c, attr, val)
        with pytest.raises(DendriteError):
            pool.append_rope([b], x, x, broken)
    broken = Rope(128)
    broken._c.inv_freq[3] = float("nan")
    with pytest.raises(DendriteError):
        pool.append_rope([b], x, x, broken)
    mixed = torch.zeros(x.numel() + q.numel(), device="cuda", dtype=torch.bfloat16)   # the rotated queries over K's last rows
    over = mixed[x.numel() - 128:][:q.numel()].view_as(q)
    for a in (dict(K=mixed[:x.numel()].view_as(x), V=x), dict(K=x, V=mixed[:x.numel()].view_as(x))):
        with pytest.raises(DendriteError):
            pool.append_rope([b], a["K"], a["V"], r, Q=q, out=over)
    pool.append_rope([], x[:0].contiguous(), x[:0].contiguous(), r)   # nothing to do
    assert pool.branch_len(b) == 65
    with pytest.raises(DendriteError):
        pool.append_layer_rope(0, x, x, r)   # nothing is pending
    pool.sync()
    pool.close()
