"""Cross attention beside a decoder's own rows in one pool, layer by layer while branches grow, and over compressed
blocks against the oracle."""
import numpy as np
import pytest
import torch

import _rows as R
from _harness import half_ulp_bf16
from copy_write_forked_gb300 import workloads as W
from copy_write_forked_gb300.dendrite import Pool
from oracle import turbo_quant as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
@pytest.mark.parametrize("new", [1, 7, 70])
def test_decode_and_cross_calls_take_turns(kind, new):
    """Both calls on every layer of every step: their plans replace one another, for as many rows, with lengths that
    grew, in blocks that are new, and over a tree that changed."""
    layers, kv, group = 3, 2, 4
    g = torch.Generator(device="cuda").manual_seed(new)
    pool = Pool(400, 16, kv, 128, R.POOL_DTYPE[kind], max_branches=16, n_layers=layers)
    rows = lambda *s: torch.randn(*s, 128, generator=g, device="cuda").to(R.ROW_DTYPE[kind])   # noqa: E731
    own, states = ([pool.new_branch() for _ in range(3)] for _ in range(2))
    for b, n in zip(states, (150, 0, 33)):
        if n:
            pool.append_kv([b], rows(layers, 1, n, kv), rows(layers, 1, n, kv))
    for step in range(4):
        pool.append_kv(own, rows(layers, 3, new, kv), rows(layers, 3, new, kv))
        if step == 1:      # a streaming encoder: inside a block, and a first row
            pool.append_kv(states[1:], rows(layers, 2, 3, kv), rows(layers, 2, 3, kv))
        if step == 2:      # beams: the tree changes
            states[0] = pool.fork(states[0], 1)[0]
            own[1] = pool.fork(own[0], 1)[0]
        for layer in range(layers):
            q = rows(3, new, kv * group)
            for br, call in ((own, pool.tree_attn_decode), (states, pool.tree_attn_cross)):
                out = call(q, br, layer=layer)
                for i, b in enumerate(br):
                    n = pool.branch_len(b)
                    if n == 0:
                        assert out[i].eq(0).all()
                        continue
                    K, V = (R.f64(x) for x in pool.read_kv([b], [0], [n], layer=layer))
                    see = np.ones((new, n), bool) if br is states else np.arange(n) <= n - new + np.arange(new)[:, None]
                    ref = R.attention(R.f64(q[i]), K, V, see)
                    assert (np.abs(R.f64(out[i]) - ref[0]) <= R.attention_bound(kind, *ref)).all(), (step, layer, i)
    pool.sync()
    pool.close()


@pytest.mark.parametrize("q_len", [1, 6, 40])
@pytest.mark.parametrize("forks", [False, True])
def test_compressed_states_against_the_oracle(q_len, forks):
    """Within the tolerance of decode attention over compressed blocks (5e-3 and half a step of bf16)."""
    signs, S = W.turbo_codec(2)
    s64, S64 = signs.numpy().astype(np.float64), S.numpy()
    pool = Pool(200, 16, 2, 128, torch.bfloat16, turbo=(signs, S), max_branches=16)
    g = torch.Generator(device="cuda").manual_seed(q_len)
    br, lens = [pool.new_branch() for _ in range(4)], [45, 0, 300, 16]
    x = [torch.randn(2, 1, max(n, 1), 2, 128, generator=g, device="cuda").bfloat16() for n in lens]
    for b, n, kv in zip(br, lens, x):
        if n:
            pool.append_kv([b], kv[0], kv[1])
    if forks:
        br, lens, x = br + pool.fork(br[2], 3), lens + lens[2:3] * 3, x + x[2:3] * 3
    q = torch.randn(len(br), q_len, 8, 128, generator=g, device="cuda").bfloat16()
    out = pool.tree_attn_cross(q, br)
    pool.sync()
    for i, n in enumerate(lens):
        if n == 0:
            assert out[i].eq(0).all()
            continue
        K, V = (y[0].float().cpu().numpy() for y in x[i])
        keys, vals = T.pack_key(*T.encode_key(K, s64, S64)), T.pack_value(*T.encode_value(V, s64))
        for j in range(0, q_len, 7):    # each query sees all: as one alone does
            ref = T.attention_compressed(q[i, j:j + 1].double().cpu().numpy(), keys, vals, s64, S64, 2)
            assert (np.abs(out[i, j:j + 1].double().cpu().numpy() - ref) <= 5e-3 + half_ulp_bf16(ref)).all(), (i, j)
    pool.close()
