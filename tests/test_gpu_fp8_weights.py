"""Attention over 8-bit pools where one token dwarfs the many beside it: the small ones'
weights, which decide the columns where the large one's value is zero, keep fp16's 11
bits."""
import numpy as np
import pytest
import torch

import _rows as R
from copy_write_forked_gb300.dendrite import Pool

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()
    torch.cuda.set_device(0)


def _bound(out, dev, mag, size, top):
    """As for any 8-bit pool (R.attention_bound), with the weights' rounding taken from
    their range alone: one is at most 2^15 in fp16, rounded by 2^-11 of itself, or under
    2^-14 by 2^-25, that is 2^-40 of a bound on the largest (it may lie up to a factor of
    2 under the whole reference: 2^-39).  A token's scale is under max|v| / 224 and a code
    at most 448: 2 * 2^-39 `top` over all tokens."""
    scores = 2 * 2.0 ** -16 * size * dev + 2.0 ** -18 * mag
    weights = 2.0 ** -11 * mag + 2.0 ** -38 * top
    return scores + weights + 2.0 ** -8 * (np.abs(out) + scores + weights) + 1e-30


def _check(K, V, q):
    n = K.shape[1]
    pool = Pool(n // 16 + 2, 16, K.shape[2], D, torch.float8_e4m3fn, max_branches=4, max_blocks_per_branch=n // 16 + 2)
    b = pool.new_branch()
    pool.append_kv([b], K, V)
    out = pool.tree_attn_decode(q, [b])
    pool.sync()
    k, v = (R.dequantise(*R.quantise(R.f64(x[0]))) for x in (K, V))
    ref = R.attention(R.f64(q[0]), k, v, np.ones((q.shape[1], n), bool))
    err, bound = np.abs(R.f64(out[0]) - ref[0]), _bound(*ref)
    assert np.isfinite(err).all() and (err <= bound).all(), float((err / bound).max())
    pool.close()


# Scores: 0 for the large tokens, -query / sqrt(128) for the others.  With 158, 178 and
# 230 the others' weights are 2^-20.1, 2^-22.7 and 2^-29.3 of the large ones': 14.4, 2.5
# and 0.03 steps of 2^-24.
@pytest.mark.parametrize("query", [40.0, 158.0, 178.0, 230.0])
@pytest.mark.parametrize("n,group", [(64, 1), (2048, 4), (2048, 8), (5000, 16)])
def test_small_weights_beside_a_large_one(query, n, group):
    g = torch.Generator(device="cuda").manual_seed(n)
    kv = 2
    K = torch.zeros(1, n, kv, D, device="cuda")
    K[..., 0] = -1.0
    V = torch.rand(1, n, kv, D, generator=g, device="cuda") + 0.25   # of one sign: errors of one side add up
    V[..., 0] = 0.0
    V[..., 1] = 1.75
    big = torch.arange(0, n, 32, device="cuda")   # one in every pair of tiles: each warp meets one
    K[:, big] = 0.0
    V[:, big] = 0.0
    V[:, big, :, 0] = 1.75
    q = torch.zeros(1, 1, kv * group, D, device="cuda")
    q[..., 0] = query
    _check(K.bfloat16(), V.bfloat16(), q.bfloat16())


def test_one_large_value():
    """The large weight comes from the value's scale, not from the score."""
    g = torch.Generator(device="cuda").manual_seed(1)
    n = 1000
    K = torch.randn(1, n, 1, D, generator=g, device="cuda") * 0.1
    V = torch.rand(1, n, 1, D, generator=g, device="cuda") + 0.25
    big = torch.arange(0, n, 32, device="cuda")
    V[:, big] = 0.0
    V[:, big, :, 0] = 2.0 ** 23 * 1.1
    _check(K.bfloat16(), V.bfloat16(), torch.randn(1, 1, 4, D, generator=g, device="cuda").bfloat16())


@pytest.mark.parametrize("size", [2.0 ** -125, 2.0 ** -100, 2.0 ** 100])
def test_values_of_extreme_size(size):
    g = torch.Generator(device="cuda").manual_seed(1)
    K, V = (torch.randn(1, 100, 1, D, generator=g, device="cuda") for _ in range(2))
    V = (V * size).bfloat16()
    pool = Pool(8, 16, 1, D, torch.float8_e4m3fn, max_branches=4)
    b = pool.new_branch()
    pool.append_kv([b], K.bfloat16(), V)
    q = torch.randn(1, 1, 4, D, generator=g, device="cuda").bfloat16()
    out = R.f64(pool.tree_attn_decode(q, [b])[0])
    pool.sync()
    k, v = (R.dequantise(*R.quantise(R.f64(x[0]))) for x in (K.bfloat16(), V))
    ref = R.attention(R.f64(q[0]), k, v, np.ones((1, 100), bool))
    # (fp32 sums end at 2^-126, bf16 outputs at 2^-133: a few steps of those in absolute terms)
    assert (np.abs(out - ref[0]) <= _bound(*ref) + 100 * 2.0 ** -126).all()
    if size > 2.0 ** -110:
        assert (np.abs(out - ref[0]) <= _bound(*ref)).all()
    pool.close()


@pytest.mark.parametrize("size", [2.0 ** 6, 2.0 ** 12, 2.0 ** 12.5])
def test_scores_of_extreme_size(size):
    """One score far above all others, up to 2^22 (8-bit pools take them to 2^23): the output is its value."""
    K = torch.zeros(1, 100, 1, D, device="cuda")
    K[0, :, 0, 0] = -size
    K[0, 41, 0, 0] = size
    V = torch.randn(1, 100, 1, D, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    q = torch.zeros(1, 1, 4, D, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = size
    pool = Pool(8, 16, 1, D, torch.float8_e4m3fn, max_branches=4)
    b = pool.new_branch()
    pool.append_kv([b], K.bfloat16(), V)
    out = R.f64(pool.tree_attn_decode(q, [b])[0, 0])
    pool.sync()
    v = R.dequantise(*R.quantise(R.f64(V[0, 41])))[0]
    assert np.array_equal(out, np.broadcast_to(v, out.shape))   # a bf16 number, exactly
    pool.close()


@pytest.mark.parametrize("rows", [-1, 1])
@pytest.mark.parametrize("key,query", [(2.0 ** 95, 2.0 ** 50), (2.0 ** 100, 2.0 ** 100), (2.0 ** -100, 2.0 ** -100), (2.0 ** 110, 2.0 ** -110)])
def test_keys_and_queries_of_extreme_size_that_hardly_meet(key, query, rows):
    """Their sizes multiplied may be past fp32's range; the scores, 0 or near it, are not."""
    g = torch.Generator(device="cuda").manual_seed(6)
    K = torch.zeros(1, 75, 2, D, device="cuda")
    K[..., 1] = key
    V = torch.randn(1, 75, 2, D, generator=g, device="cuda")
    q = torch.zeros(1, 1, 8, D, device="cuda")
    q[..., 0] = query
    K, V, q = K.bfloat16(), V.bfloat16(), q.bfloat16()
    pool = Pool(8, 16, 2, D, torch.float8_e4m3fn, max_branches=4, tc_min_rows=rows)
    b = pool.new_branch()
    pool.append_kv([b], K, V)
    out = pool.tree_attn_decode(q, [b])
    pool.sync()
    k, v = (R.dequantise(*R.quantise(R.f64(x[0]))) for x in (K, V))
    ref = R.attention(R.f64(q[0]), k, v, np.ones((1, 75), bool))
    assert (np.abs(R.f64(out[0]) - ref[0]) <= R.attention_bound("fp8", *ref)).all()
    pool.close()
