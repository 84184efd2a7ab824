"""8-bit pools through the C-ABI library: stored tiles bit for bit (fresh rows,
copy-on-write copies, rows at the edges of the format), rows read back, and tree
decode attention against 64 bits within the bound its roundings allow."""
import random

import numpy as np
import pytest
import torch

import _rows as R
from copy_write_forked_gb300 import workloads as W
from copy_write_forked_gb300.dendrite import DendriteError, Pool
from copy_write_forked_gb300.runner import pool_for, run_script
from oracle.block_pool import run_script_pool

from _harness import oracle_tree, pool_state_matches

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()
    torch.cuda.set_device(0)


def _check_tiles(pool, handle, K, V, layer=0):
    """The stored rows of a branch against rows K, V [len][n_kv][128] (float64)."""
    tab = pool.read_table(handle)
    for blk in range((len(K) + 15) // 16):
        raw = pool.read_block(tab[blk], layer=layer)
        for x, r in zip((K, V), raw):
            rows = x[16 * blk:16 * blk + 16]
            codes, e = R.untile(r.numpy())
            want, we = R.quantise(rows.transpose(1, 0, 2))
            n = len(rows)
            assert R.same_codes(codes[:, :n], want), blk
            assert np.array_equal(e[:, :n], we), blk


@pytest.mark.parametrize("seed", range(6))
def test_tiles_and_tables_match_the_reference(seed):
    w = W.random_script(300 + seed, n_ops=28, max_live=6, max_append=40, n_kv=[1, 2, 3][seed % 3], n_q=6, d=128, bs=16,
                        dtype=torch.bfloat16, truncates=seed % 2 == 1)
    pool = pool_for(w, dtype=F8)
    h = run_script(pool, w)
    pool.sync()
    ref = run_script_pool(w, pool.num_blocks, kv_source=lambda idx: w.kv(idx, "cuda"))
    pool_state_matches(pool, h, ref, check_bytes=False)
    tree = oracle_tree(w, list(ref.table), "cuda")
    for b in ref.table:
        K, V = tree.materialise(b)
        _check_tiles(pool, h[b], K, V)
    pool.close()


def _edge_rows():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(64, 2, 128, generator=g)
    x *= torch.exp2(torch.arange(-100, 28, 2).float()[:, None, None])
    x[0] = 0.0
    x[1, :, 3] = float("inf")
    x[2, :, 5] = float("-inf")
    x[3, :, 7] = float("nan")
    x[4] = float("nan")
    x[5] = 0.0
    x[5, :, 0] = 2.0 ** -133
    x[6, :, 9] = 3.3895e38
    x[7] = 0.0
    x[7, 0, :16] = torch.tensor([448., 447, 432, 416, 240, 15.5, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 1.0625, 1.1875, -448, -0.0, 0.0, 17, 464 / 2])
    x[8] = x[7] * 2.0 ** 60
    x[9] = x[7] * (449 / 448)
    x[10] = -0.0
    return x.to(torch.bfloat16)


def test_rows_at_the_edges_of_the_format():
    rows = _edge_rows()
    pool = Pool(64, 16, 2, 128, F8, max_branches=4)
    b = pool.new_branch()
    K = rows[None].cuda()
    V = rows.flip(0)[None].cuda().contiguous()
    pool.append_kv([b], K, V)
    _check_tiles(pool, b, R.f64(K[0]), R.f64(V[0]))
    k, v = pool.read_kv([b], [0], [64])
    for got, x in ((k, K[0]), (v, V[0])):
        want = R.dequantise(*R.quantise(R.f64(x)))
        assert np.array_equal(R.f64(got), want, equal_nan=True)   # bf16 holds code * 2^e exactly
    pool.close()


@pytest.mark.parametrize("dtype,d", [(torch.float32, 32), (torch.float32, 96), (torch.float32, 256),
                                     (torch.bfloat16, 128), (F8, 128)])
@pytest.mark.parametrize("layers", [1, 3])
def test_read_kv(dtype, d, layers):
    rng = random.Random(d)
    rows = torch.bfloat16 if dtype == F8 else dtype
    g = torch.Generator(device="cuda").manual_seed(d)
    pool = Pool(400, 16, 3, d, dtype, max_branches=16, n_layers=layers)
    root = pool.new_branch()
    data = {}
    shape = (layers,) if layers > 1 else ()
    K, V = (torch.randn(*shape, 1, 101, 3, d, generator=g, device="cuda").to(rows) for _ in range(2))
    pool.append_kv([root], K, V)
    data[root] = (K.view(layers, 101, 3, d), V.view(layers, 101, 3, d))
    kids = pool.fork(root, 3)
    K2, V2 = (torch.randn(*shape, 3, 20, 3, d, generator=g, device="cuda").to(rows) for _ in range(2))
    pool.append_kv(kids, K2, V2)
    for i, b in enumerate(kids):
        data[b] = tuple(torch.cat((x, y.view(layers, 3, 20, 3, d)[:, i]), 1) for x, y in zip(data[root], (K2, V2)))
    for _ in range(8):
        br = [rng.choice([root] + kids) for _ in range(rng.randint(1, 40))]
        starts, counts = [], []
        for b in br:
            n = 101 if b == root else 121
            s = rng.randint(0, n)
            starts.append(s)
            counts.append(rng.choice([0, 1, n - s, rng.randint(0, n - s)]) if s < n else 0)
        layer = rng.randrange(layers)
        got = pool.read_kv(br, starts, counts, layer=layer)
        for x, which in zip(got, (0, 1)):
            want = torch.cat([data[b][which][layer, s:s + c] for b, s, c in zip(br, starts, counts)])
            if dtype == F8:
                assert np.array_equal(R.f64(x), R.held(R.f64(want), "fp8"))
            else:
                assert torch.equal(x, want)
    # one row each, no row at all, every row of many branches (arguments past the kernel parameters)
    assert pool.read_kv([root], [101], [0])[0].shape == (0, 3, d)
    assert pool.read_kv([], [], [])[0].shape == (0, 3, d)
    many = [root] * 700
    k, v = pool.read_kv(many, [i % 101 for i in range(700)], [1] * 700)
    idx = torch.tensor([i % 101 for i in range(700)])
    want = data[root][1][0].cpu()[idx]
    assert np.array_equal(R.f64(v), R.held(R.f64(want), "fp8" if dtype == F8 else "same"))
    pool.close()


def test_read_kv_leaves_what_is_behind_its_rows():
    pool = Pool(16, 16, 2, 128, F8, max_branches=4)
    b = pool.new_branch()
    K = torch.randn(1, 30, 2, 128, device="cuda").bfloat16()
    pool.append_kv([b], K, K)
    from copy_write_forked_gb300.dendrite import _arr, _ptr, lib
    out = torch.full((2, 40, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ba, sa, ca = _arr([b]), _arr([3]), _arr([11])
    st = torch.cuda.current_stream().cuda_stream
    assert lib().dendrite_read_kv(pool._h, 0, _ptr(ba), _ptr(sa), _ptr(ca), 1, out[0].data_ptr(), out[1].data_ptr(), st) == 0
    pool.sync()
    assert (out[:, 11:] == 7.0).all() and not (out[:, :11] == 7.0).all()
    # overlapping and misaligned outputs, and ranges past the branch, are refused
    assert lib().dendrite_read_kv(pool._h, 0, _ptr(ba), _ptr(sa), _ptr(ca), 1, out.data_ptr(), out.data_ptr() + 256, st) == -1
    assert lib().dendrite_read_kv(pool._h, 0, _ptr(ba), _ptr(sa), _ptr(ca), 1, out[0].data_ptr() + 2, out[1].data_ptr(), st) == -1
    for s, c in ((-1, 2), (0, 31), (31, 0), (5, -1), (2 ** 31 - 1, 2 ** 31 - 1)):
        with pytest.raises(DendriteError):
            pool.read_kv([b], [s], [c])
    with pytest.raises(DendriteError):
        pool.read_kv([b + 1], [0], [1])
    with pytest.raises(DendriteError):
        pool.read_kv([b], [0], [1], layer=1)
    pool.close()


def _attend(kind, branches_kv, q, out, q_len):
    """Checks out [n][q_len][heads][d] of branches that hold the rows branches_kv[i] = (K, V) (float64, as held)."""
    worst = 0.0
    for i, (K, V) in enumerate(branches_kv):
        n = len(K)
        see = np.arange(n) <= n - q_len + np.arange(q_len)[:, None]
        ref = R.attention(R.f64(q[i]), K, V, see)
        err = np.abs(R.f64(out[i]) - ref[0])
        bound = R.attention_bound(kind, *ref)
        worst = max(worst, float((err / bound).max()))
        assert (err <= bound).all(), (i, float(err.max()), float((err / bound).max()))
    return worst


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 300, 1111])
@pytest.mark.parametrize("kv,group,q_len", [(1, 1, 1), (2, 4, 1), (1, 8, 1), (2, 5, 1), (1, 16, 2), (2, 7, 3), (1, 4, 16), (1, 3, 40)])
def test_attention_lengths_and_groups(length, kv, group, q_len):
    if length < q_len:
        pytest.skip("the queries are the last q_len positions")
    g = torch.Generator(device="cuda").manual_seed(length * 100 + group)
    pool = Pool(256, 16, kv, 128, F8, max_branches=4)
    br = [pool.new_branch() for _ in range(2)]
    K, V = (torch.randn(2, length, kv, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    pool.append_kv(br, K, V)
    q = torch.randn(2, q_len, kv * group, 128, generator=g, device="cuda").bfloat16()
    out = pool.tree_attn_decode(q, br)
    pool.sync()
    _attend("fp8", [(R.held(R.f64(K[i]), "fp8"), R.held(R.f64(V[i]), "fp8")) for i in range(2)], q, out, q_len)
    pool.close()


@pytest.mark.parametrize("width,group,prefix,leaf,q_len", [(2, 4, 100, 9, 1), (4, 4, 517, 33, 1), (7, 5, 48, 1, 1),
                                                           (16, 4, 640, 20, 1), (3, 4, 200, 24, 8), (40, 8, 333, 2, 1)])
def test_attention_over_forks(width, group, prefix, leaf, q_len):
    g = torch.Generator(device="cuda").manual_seed(width)
    kv = 2
    pool = Pool(1000, 16, kv, 128, F8, max_branches=64)
    root = pool.new_branch()
    K, V = (torch.randn(1, prefix, kv, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    pool.append_kv([root], K, V)
    kids = pool.fork(root, width)
    k, v = (torch.randn(width, leaf, kv, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    pool.append_kv(kids, k, v)
    q = torch.randn(width, q_len, kv * group, 128, generator=g, device="cuda").bfloat16()
    held = [tuple(R.held(R.f64(torch.cat((a[0], b[i]))), "fp8") for a, b in ((K, k), (V, v))) for i in range(width)]
    out = pool.tree_attn_decode(q, kids)
    pool.sync()
    _attend("fp8", held, q, out, q_len)
    # the same bits again, on another stream, and in the allocation-free call's fixed scratch
    assert torch.equal(out, pool.tree_attn_decode(q, kids))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = torch.zeros_like(q)
    pool.tree_attn_decode(q, kids, out=again, stream=s)
    s.synchronize()
    assert torch.equal(out, again)
    fixed = torch.zeros_like(q)
    pool.tree_attn_decode_noalloc(q, kids, fixed)
    pool.sync()
    assert torch.equal(out, fixed)
    pool.close()


@pytest.mark.parametrize("case", ["value scales", "key scales", "queries", "zero values", "one token far larger"])
def test_attention_over_rows_of_very_different_size(case):
    """The scales of values spread over 2^80, keys and queries far from one, zero rows."""
    g = torch.Generator(device="cuda").manual_seed(11)
    n, kv, group = 200, 2, 4
    K, V = (torch.randn(1, n, kv, 128, generator=g, device="cuda") for _ in range(2))
    q = torch.randn(1, 1, kv * group, 128, generator=g, device="cuda")
    if case == "value scales":
        V *= torch.exp2(torch.randint(-40, 41, (1, n, kv, 1), generator=g, device="cuda").float())
    elif case == "key scales":
        K *= 2.0 ** 50
        q *= 2.0 ** -50
    elif case == "queries":
        q *= torch.exp2(torch.tensor([-60., -20, -6, 0, 1, 2, 3, 1.5], device="cuda"))[None, None, :, None]
    elif case == "zero values":
        V[:, ::3] = 0
        K[:, ::5] = 0
    else:
        V[:, 17] *= 2.0 ** 20
        K[:, 17] = -K[:, 17].abs() * q[:, :, ::group].sign()   # a token of little weight and huge values
    K, V, q = K.bfloat16(), V.bfloat16(), q.bfloat16()
    pool = Pool(64, 16, kv, 128, F8, max_branches=4)
    b = pool.new_branch()
    pool.append_kv([b], K, V)
    out = pool.tree_attn_decode(q, [b])
    pool.sync()
    _attend("fp8", [(R.held(R.f64(K[0]), "fp8"), R.held(R.f64(V[0]), "fp8"))], q, out, 1)
    pool.close()


@pytest.mark.parametrize("q_len", [1, 12, 70])
@pytest.mark.parametrize("step", [0.05, 0.4, 1.5, -0.4])
def test_running_maximum(step, q_len):
    """Scores that climb (or fall) with the position: the reference moves in every stage, in the middle of stages and not at all."""
    g = torch.Generator(device="cuda").manual_seed(5)
    kv, group, n = 2, 4, 400
    q = torch.randn(1, q_len, kv * group, 128, generator=g, device="cuda")
    q[..., 0] = 8.0
    K = torch.randn(1, n, kv, 128, generator=g, device="cuda") * 0.3
    K[..., 0] = step * torch.arange(n, device="cuda")[None, :, None]
    V = torch.randn(1, n, kv, 128, generator=g, device="cuda")
    K, V, q = K.bfloat16(), V.bfloat16(), q.bfloat16()
    pool = Pool(64, 16, kv, 128, F8, max_branches=4)
    b = pool.new_branch()
    pool.append_kv([b], K, V)
    out = pool.tree_attn_decode(q, [b])
    pool.sync()
    _attend("fp8", [(R.held(R.f64(K[0]), "fp8"), R.held(R.f64(V[0]), "fp8"))], q, out, q_len)
    pool.close()


def test_keys_that_are_not_finite_touch_only_the_rows_that_see_them():
    g = torch.Generator(device="cuda").manual_seed(4)
    pool = Pool(64, 16, 1, 128, F8, max_branches=4)
    b = pool.new_branch()
    K, V = (torch.randn(1, 40, 1, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    K[0, 38, 0, 3] = float("inf")
    pool.append_kv([b], K, V)
    q = torch.randn(1, 4, 4, 128, generator=g, device="cuda").bfloat16()
    out = R.f64(pool.tree_attn_decode(q, [b])[0])
    assert np.isfinite(out[:2]).all() and np.isnan(out[2:]).all()
    pool.close()


@pytest.mark.parametrize("rows", [-1, 1])
@pytest.mark.parametrize("group,q_len", [(1, 1), (8, 3), (8, 40)])
def test_rows_behind_a_branch_touch_nothing(rows, group, q_len):
    """Rows of NaN that a roll-back, an acceptance or a block's last owner left behind a branch's end."""
    g = torch.Generator(device="cuda").manual_seed(8)
    pool = Pool(8, 16, 2, 128, F8, max_branches=8, tc_min_rows=rows)
    nan = torch.full((1, 128, 2, 128), float("nan"), device="cuda", dtype=torch.bfloat16)

    def rows_of(n):
        return torch.randn(1, n, 2, 128, generator=g, device="cuda").bfloat16()

    def attend(b, k, v, q_len):
        q = rows_of(q_len * group).reshape(1, q_len, 2 * group, 128)
        _attend("fp8", [(R.held(R.f64(k[0]), "fp8"), R.held(R.f64(v[0]), "fp8"))], q, pool.tree_attn_decode(q, [b]), q_len)

    b = pool.new_branch()
    pool.append_kv([b], nan, nan)          # every block of the pool holds NaN
    pool.free([b])
    b = pool.new_branch()
    for n, more in ((41, 5), (57, 18)):    # ends inside a block, three blocks in; more rows come and go
        k, v = rows_of(n), rows_of(n)
        pool.append_kv([b], k, v)
        attend(b, k, v, q_len)
        pool.append_kv([b], nan[:, :more].contiguous(), nan[:, :more].contiguous())
        pool.accept_draft([b], more, [[]])
        attend(b, k, v, q_len)
        child = pool.fork(b, 1)            # a copied tail block
        pool.append_kv(child, k[:, :1].contiguous(), v[:, :1].contiguous())
        attend(child[0], torch.cat((k, k[:, :1]), 1), torch.cat((v, v[:, :1]), 1), q_len)
        pool.free(child)
        pool.truncate([b], [0])
    pool.close()


def test_layers_and_the_split_append():
    g = torch.Generator(device="cuda").manual_seed(6)
    L, kv, nq = 3, 2, 8
    pool = Pool(200, 16, kv, 128, F8, max_branches=16, n_layers=L)
    root = pool.new_branch()
    K, V = (torch.randn(L, 1, 70, kv, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    pool.append_kv([root], K, V)
    kids = pool.fork(root, 3)
    k, v = (torch.randn(L, 3, 5, kv, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    pool.append_begin(kids, 5)
    for l in (2, 0, 1):
        with pytest.raises(DendriteError):
            pool.read_kv(kids, [0] * 3, [1] * 3, layer=l)
        pool.append_layer(l, k[l].contiguous(), v[l].contiguous())
        pool.read_kv(kids, [0] * 3, [1] * 3, layer=l)
    q = torch.randn(3, 1, nq, 128, generator=g, device="cuda").bfloat16()
    for l in range(L):
        held = [tuple(R.held(R.f64(torch.cat((a[l, 0], b[l, i]))), "fp8") for a, b in ((K, k), (V, v))) for i in range(3)]
        for i in range(3):
            _check_tiles(pool, kids[i], R.f64(torch.cat((K[l, 0], k[l, i]))), R.f64(torch.cat((V[l, 0], v[l, i]))), layer=l)
        _attend("fp8", held, q, pool.tree_attn_decode(q, kids, layer=l), 1)
    pool.close()


def test_refusals():
    with pytest.raises(DendriteError) as e:
        Pool(16, 16, 2, 64, F8)
    assert e.value.name == "EDTYPE"
    pool = Pool(16, 16, 2, 128, F8, max_branches=4)
    b = pool.new_branch()
    with pytest.raises(DendriteError):
        pool.append_kv([b], torch.zeros(1, 1, 2, 128, device="cuda", dtype=F8), torch.zeros(1, 1, 2, 128, device="cuda", dtype=F8))
    signs, S = W.turbo_codec(0)
    tq = Pool(16, 16, 2, 128, torch.bfloat16, max_branches=4, turbo=(signs, S))
    t = tq.new_branch()
    x = torch.zeros(1, 3, 2, 128, device="cuda", dtype=torch.bfloat16)
    tq.append_kv([t], x, x)
    for call in (lambda: tq.read_kv([t], [0], [1]), lambda: tq.accept_draft([t], 2, [[0]]),
                 lambda: tq.tree_attn_draft(torch.zeros(1, 2, 4, 128, device="cuda", dtype=torch.bfloat16), [t], [-1, 0])):
        with pytest.raises(DendriteError) as e:
            call()
        assert e.value.name == "EDTYPE"
    # a captured call would be replayed with old tables
    pool.append_kv([b], x, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    k = torch.empty(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    from copy_write_forked_gb300.dendrite import _arr, _ptr, lib
    ba, sa, ca = _arr([b]), _arr([0]), _arr([1])
    with torch.cuda.stream(s):
        graph.capture_begin()
        rc = lib().dendrite_read_kv(pool._h, 0, _ptr(ba), _ptr(sa), _ptr(ca), 1, k.data_ptr(), v.data_ptr(), s.cuda_stream)
        graph.capture_end()
    assert rc == -1
    pool.read_kv([b], [0], [1])
    pool.sync()
    pool.close()
    tq.close()


def test_captured_calls_are_refused():
    """Appends and attention of an 8-bit pool on a capturing stream: refused, and nothing of the pool changed."""
    from copy_write_forked_gb300.dendrite import _arr, _ptr, lib
    pool = Pool(16, 16, 2, 128, F8, max_branches=4)
    b = pool.new_branch()
    x = torch.randn(1, 20, 2, 128, device="cuda").bfloat16()
    q = torch.randn(1, 1, 8, 128, device="cuda").bfloat16()
    pool.append_kv([b], x, x)
    want = pool.tree_attn_decode(q, [b])
    out = torch.zeros_like(q)
    ba = _arr([b])
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    L = lib()
    with torch.cuda.stream(s):
        graph.capture_begin()
        rcs = [L.dendrite_append_kv(pool._h, _ptr(ba), 1, 20, x.data_ptr(), x.data_ptr(), s.cuda_stream),
               L.dendrite_append_begin(pool._h, _ptr(ba), 1, 20, s.cuda_stream),
               L.dendrite_tree_attn_decode_layer(pool._h, 0, q.data_ptr(), 8, 1, _ptr(ba), 1, out.data_ptr(), s.cuda_stream)]
        graph.capture_end()
    assert rcs == [-1, -1, -1]
    assert pool.branch_len(b) == 20 and torch.equal(pool.tree_attn_decode(q, [b]), want)
    pool.append_kv([b], x, x)
    k, _ = pool.read_kv([b], [20], [20])
    assert np.array_equal(R.f64(k), R.held(R.f64(x[0]), "fp8"))
    pool.sync()
    pool.close()
