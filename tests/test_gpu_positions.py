"""Appends turned by given positions, of one axis and several, through the C-ABI library: against 64 bits within what
fp32 products and one rounding allow, and bit for bit the plain call where the positions are the lengths."""
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


def turned(x, angles, rot, interleaved, m):
    """x [tokens][heads][d] (float64) turned by angles [tokens][rot / 2]; and m (|x1| + |x2|) of each element."""
    y, size = x.copy(), np.zeros_like(x)
    c, s = np.cos(angles)[:, None], np.sin(angles)[:, None]
    i = np.arange(rot // 2)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    u, v = x[..., p], x[..., q]
    y[..., p], y[..., q] = m * (u * c - v * s), m * (v * c + u * s)
    size[..., p] = size[..., q] = abs(m) * (np.abs(u) + np.abs(v))
    return y, size


def _close(kind, got, y, size, stored, far):
    """far: the largest |position|.  inv_freq (at most 1) as turns is rounded once and cut to 64 bits, 2^-53 and 2^-64 of a
    turn, and the reference's own product by 2^-53 of the angle: 2^-50 radians a position are more than both."""
    slack = (R.ROPE_ERR + far * 2.0 ** -50) * size
    if stored and kind == "fp8":
        # (as in the plain call's tests: the row's exponent may be the next one)
        top = (np.abs(y) + slack).max(-1, keepdims=True)
        e = np.ceil(np.log2(np.maximum(top, 1e-300) / 448))
        bound = slack + np.maximum(2.0 ** -4 * (np.abs(y) + slack), 2.0 ** (e - 10))
    else:
        bound = slack + {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp8": 2.0 ** -8}[kind] * (np.abs(y) + slack)
    err = np.abs(got - y)
    assert (err <= bound + 1e-38).all(), float((err / (bound + 1e-38)).max())


def _case(kind, dim, rot, interleaved, axes, kv, nq, lens, new, at, scaling="none", seed=0, layers=1, split=False, in_place=False):
    """at: positions [n][new][axes] (or [n][new]) as an int32 CUDA tensor of any strides."""
    rows = R.ROW_DTYPE[kind]
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, lead = len(lens), (layers,) if layers > 1 else ()
    pool = Pool(sum((x + new) // 16 + 3 for x in lens) + 8, 16, kv, dim, R.POOL_DTYPE[kind], max_branches=n + 8, n_layers=layers,
                max_blocks_per_branch=(max(lens) + new) // 16 + 2)
    br = [pool.new_branch() for _ in lens]
    for b, x in zip(br, lens):
        if x:
            z = torch.randn(*lead, 1, x, kv, dim, generator=g, device="cuda").to(rows)
            pool.append_kv([b], z, z)
    rope = Rope(rot, base=500000.0, interleaved=interleaved, scaling=scaling, factor=4.0, original_len=8192.0, axes=axes)
    freq, m = R.frequencies(rot, 500000.0, scaling, 4.0, 8192.0)
    K, V = (torch.randn(*lead, n, new, kv, dim, generator=g, device="cuda").to(rows) for _ in range(2))
    Q = torch.randn(*lead, n, new, nq, dim, generator=g, device="cuda").to(rows) if nq else None
    q64, k64, v64 = (R.f64(x).reshape(layers, n, new, -1, dim) if x is not None else None for x in (Q, K, V))
    if split:
        pool.append_begin(br, new)
        outs = [pool.append_layer_rope(l, K[l].contiguous(), V[l].contiguous(), rope, Q=Q[l].contiguous() if nq else None, positions=at)
                for l in range(layers)]
        out = torch.stack(outs) if nq else None
    else:
        out = pool.append_rope(br, K, V, rope, Q=Q, positions=at, out=Q if in_place else None)
    pool.sync()
    p = at.cpu().numpy().astype(float).reshape(n, new, -1)
    far = np.abs(p).max(initial=0)
    for i in range(n):
        angles = p[i][:, axes or [0] * (rot // 2)] * np.asarray(freq)
        for l in range(layers):
            if nq:
                o = R.f64(out).reshape(layers, n, new, nq, dim)[l, i]
                _close(kind, o, *turned(q64[l, i], angles, rot, interleaved, m), False, far)
                assert rot == dim or np.array_equal(o[..., rot:], q64[l, i][..., rot:])
            k, v = pool.read_kv([br[i]], [lens[i]], [new], layer=l)
            _close(kind, R.f64(k), *turned(k64[l, i], angles, rot, interleaved, m), True, far)
            assert np.array_equal(R.f64(v), R.held(v64[l, i], kind))
        assert pool.branch_len(br[i]) == lens[i] + new
    pool.close()


def _at(n, new, axes, top=5000, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, top, (n, new, axes), generator=g, device="cuda").int()


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("fp8", 128), ("fp32", 128), ("fp32", 32), ("fp32", 96), ("fp32", 256)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", ["all", 16])
@pytest.mark.parametrize("n_axes,woven", [(1, False), (2, True), (3, False), (3, True), (4, True)])
def test_types_layouts_and_axes(kind, dim, interleaved, rot, n_axes, woven):
    rot = {"all": dim}.get(rot, rot)
    pairs = rot // 2
    axes = [i % n_axes if woven else i * n_axes // pairs for i in range(pairs)]
    _case(kind, dim, rot, interleaved, axes, 2, 6, [0, 5, 31], 19, _at(3, 19, n_axes, seed=dim + rot), seed=dim + rot)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
@pytest.mark.parametrize("new", [1, 2, 3, 15, 16, 17, 40])
@pytest.mark.parametrize("kv,nq", [(1, 0), (1, 7), (8, 32)])
def test_sizes(kind, new, kv, nq):
    axes = [0] * 16 + [1] * 24 + [2] * 24
    _case(kind, 128, 128, False, axes, kv, nq, [0, 1, 15, 16, 100], new, _at(5, new, 3, seed=new), seed=new)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn", "bands"])
def test_scalings(scaling):
    _case("fp32", 64, 64, False, [i % 3 for i in range(32)], 1, 2, [7, 30], 9, _at(2, 9, 3, 60000), scaling=scaling)


@pytest.mark.parametrize("interleaved", [False, True])
def test_negative_and_far_positions(interleaved):
    at = _at(2, 6, 2, 200000, seed=1) - 100000
    _case("fp32", 128, 128, interleaved, [i % 2 for i in range(64)], 1, 2, [3, 40], 6, at)
    ends = torch.tensor([-2147483648, 2147483647, 0, -1, 1 << 24, -(1 << 24) - 1], dtype=torch.int32, device="cuda")
    _case("fp32", 128, 128, interleaved, None, 1, 2, [0], 6, ends[None])
    _case("bf16", 128, 128, interleaved, [1] * 64, 1, 2, [0], 6, torch.stack((ends.flip(0), ends), -1)[None])


def test_strides():
    n, new = 3, 21
    axes = [0] * 16 + [1] * 24 + [2] * 24
    first = _at(3, n, new).permute(1, 2, 0)                       # axes first, as models keep them
    assert not first.is_contiguous()
    _case("bf16", 128, 128, False, axes, 2, 4, [0, 9, 16], new, first)
    _case("bf16", 128, 128, False, axes, 2, 4, [0, 9, 16], new, _at(1, new, 3).expand(n, -1, -1))      # one for all branches
    _case("bf16", 128, 128, False, axes, 2, 4, [0, 9, 16], new, _at(n, 1, 3).expand(-1, new, -1))
    _case("bf16", 128, 128, False, axes, 2, 4, [0, 9, 16], new, _at(n, new, 1).expand(-1, -1, 3))      # the axes alike
    _case("bf16", 128, 128, False, axes, 2, 4, [0, 9, 16], new, _at(2 * n, 3 * new, 7)[::2, ::3, 1::2])
    _case("fp8", 128, 128, False, None, 2, 4, [0, 9, 16], new, _at(n, new, 2)[:, :, 1])                # [n][new], strided


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
def test_layers_in_place_and_split(kind):
    axes = [i % 3 for i in range(64)]
    _case(kind, 128, 128, False, axes, 2, 4, [9, 20], 5, _at(2, 5, 3), layers=3)
    _case(kind, 128, 128, True, axes, 2, 4, [9, 20], 5, _at(2, 5, 3), layers=3, in_place=True)
    _case(kind, 128, 128, False, axes, 2, 4, [9, 20], 5, _at(2, 5, 3), layers=3, split=True)
    _case(kind, 128, 128, False, axes, 2, 0, [9, 20], 5, _at(2, 5, 3), layers=2, split=True)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
@pytest.mark.parametrize("drafts", [False, True])
def test_lengths_and_depths_as_positions_are_the_plain_call(kind, drafts):
    """The same bits, with the axes pointing at equal positions."""
    rows, new = R.ROW_DTYPE[kind], 30
    g = torch.Generator(device="cuda").manual_seed(4)
    lens = [0, 33, 16]
    x = torch.randn(3, new, 2, 128, generator=g, device="cuda").to(rows)
    q = torch.randn(3, new, 8, 128, generator=g, device="cuda").to(rows)
    trees = [R.tree(random.Random(i), new) for i in range(3)] if drafts else None
    got = []
    for given in (False, True):
        pool = Pool(64, 16, 2, 128, R.POOL_DTYPE[kind], max_branches=8)
        br = [pool.new_branch() for _ in lens]
        for b, n in zip(br, lens):
            if n:
                pool.append_kv([b], x[:1, :1].expand(1, n, 2, 128).contiguous(), x[:1, :1].expand(1, n, 2, 128).contiguous())
        if given:
            at = torch.tensor([[n + d for d in (R.depths(trees[i]) if drafts else range(new))] for i, n in enumerate(lens)],
                              dtype=torch.int32, device="cuda")
            out = pool.append_rope(br, x, x, Rope(128, axes=[0, 1, 2, 3] * 16), Q=q, positions=at[..., None].expand(-1, -1, 4))
        else:
            out = pool.append_rope(br, x, x, Rope(128), Q=q, parents=None if trees is None else torch.tensor(trees, dtype=torch.int32))
        got.append((out, *pool.read_kv(br, lens, [new] * 3)))
        pool.close()
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_many_branches():
    # more arguments than travel as kernel parameters
    lens = [i % 37 for i in range(600)]
    _case("bf16", 128, 128, False, [i % 3 for i in range(64)], 1, 2, lens, 3, _at(600, 3, 3))


def test_another_stream():
    pool = Pool(64, 16, 4, 128, torch.bfloat16, max_branches=8)
    x = torch.randn(4, 50, 4, 128, device="cuda").bfloat16()
    q = torch.randn(4, 50, 16, 128, device="cuda").bfloat16()
    at = _at(4, 50, 1)[..., 0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    br = [pool.new_branch() for _ in range(4)]
    out = pool.append_rope(br, x, x, Rope(128), Q=q, positions=at, stream=s)
    del at
    torch.randint(0, 9, (4, 50), device="cuda")   # would take the positions' memory
    torch.cuda.synchronize()
    twin = Pool(64, 16, 4, 128, torch.bfloat16, max_branches=8)
    br2 = [twin.new_branch() for _ in range(4)]
    same = twin.append_rope(br2, x, x, Rope(128), Q=q, positions=_at(4, 50, 1)[..., 0])
    assert torch.equal(out, same)
    pool.close()
    twin.close()


def test_refusals():
    pool = Pool(64, 16, 2, 128, torch.bfloat16, max_branches=8)
    b = pool.new_branch()
    x = torch.zeros(1, 4, 2, 128, device="cuda", dtype=torch.bfloat16)
    q = torch.zeros(1, 4, 8, 128, device="cuda", dtype=torch.bfloat16)
    three = Rope(128, axes=[i % 3 for i in range(64)])
    at = torch.zeros(1, 4, 3, dtype=torch.int32, device="cuda")
    flat = torch.zeros(4 * q.numel(), device="cuda", dtype=torch.bfloat16)
    bad = [dict(rope=three), dict(rope=three, positions=at.long()), dict(rope=three, positions=at.cpu()), dict(rope=three, positions=at[..., :2]),
           dict(rope=three, positions=at[:, :3]), dict(rope=three, positions=at[..., 0]), dict(rope=Rope(128), positions=at),
           dict(rope=three, positions=at, parents=[-1, 0, 1, 2]), dict(rope=three, positions=[[0, 1, 2]] * 4),
           # positions inside the rotated queries
           dict(rope=Rope(128), Q=q, out=flat[:q.numel()].view_as(q), positions=flat.view(torch.int32)[64:68].view(1, 4))]
    for kw in bad:
        with pytest.raises(DendriteError):
            pool.append_rope([b], x, x, **kw)
        assert pool.branch_len(b) == 0
    for axes in ([0] * 63, [4] + [0] * 63, [-1] + [0] * 63):
        with pytest.raises(DendriteError):
            Rope(128, axes=axes)
    broken = Rope(128, axes=[i % 3 for i in range(64)])
    broken._axis = bytes([0, 1, 3] + [2] * 125)   # an axis past the rope's
    with pytest.raises(DendriteError):
        pool.append_rope([b], x, x, broken, positions=at)
    with pytest.raises(DendriteError):
        pool.append_layer_rope(0, x, x, three, positions=at)   # nothing is pending
    pool.append_rope([b], x, x, three, positions=at)
    pool.sync()
    pool.close()
