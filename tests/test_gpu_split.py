"""How a call with wide prefixes and private leaves shares the SMs between the two
attention kernels: by what each pool type's own kernels take."""
import numpy as np
import pytest
import torch

import _rows as R
from copy_write_forked_gb300.dendrite import Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()
    torch.cuda.set_device(0)


def _ctas(kind, prefixes, prefix, width, leaf, **kw):
    pool = Pool(prefixes * (prefix // 16 + width * (leaf // 16 + 1)) + 8, 16, 8, 128, R.POOL_DTYPE[kind],
                max_branches=prefixes * (width + 1) + 1, max_blocks_per_branch=(prefix + leaf) // 16 + 2, **kw)
    roots = [pool.new_branch() for _ in range(prefixes)]
    x = torch.zeros(prefixes, prefix, 8, 128, device="cuda", dtype=torch.bfloat16)
    pool.append_kv(roots, x, x)
    kids = [c for k in pool.fork_batch(roots, [width] * prefixes) for c in k]
    x = torch.zeros(len(kids), leaf, 8, 128, device="cuda", dtype=torch.bfloat16)
    pool.append_kv(kids, x, x)
    pool.tree_attn_decode(torch.zeros(len(kids), 1, 32, 128, device="cuda", dtype=torch.bfloat16), kids)
    pool.sync()
    st = pool.last_plan_stats()
    pool.close()
    return st["n_tc_ctas"], st["n_ctas"]


# 64 rows a kv head on the prefix (bf16: 256, its tcgen05 class begins at 65), 4 on a leaf.
@pytest.mark.parametrize("shape", [(4, 4096, 16, 512), (2, 16384, 64, 1024)])
def test_8_bit_calls_take_no_split_that_the_bf16_kernels_would(shape):
    all_sms = _ctas("fp8", *shape, tc_sms=-1)
    assert _ctas("fp8", *shape) == all_sms
    assert _ctas("fp8", *shape, tc_sms=60)[0] == 60


def test_bf16_calls_split_as_before():
    # tcgen05: 8 kv heads x (1,024 tiles x 3 + 24) weights x 85 SM ns = 2.105 SM ms a prefix; bytes:
    # 8 x (1,024 + 64 x 64) tiles x 8,192 = 335.5 MB a prefix, 50.08 us at 6,700 GB/s.  Both kernels
    # end there from 2105 / 50.08 = 42.04 SMs on: 43.
    n_tc, n = _ctas("bf16", 2, 16384, 64, 1024)
    assert n_tc == 43 and n == 2 * (torch.cuda.get_device_properties(0).multi_processor_count - n_tc)


@pytest.mark.parametrize("width,leaf", [(4, 20), (7, 3)])
def test_8_bit_prefixes_beside_many_short_leaves(width, leaf):
    """A plan whose small kernel has long units of up to 28 rows and many short ones of 4: right, whatever CTA has which."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n, prefix, kv = 4, 1500, 2
    pool = Pool(n * (prefix // 16 + 4 * width), 16, kv, 128, torch.float8_e4m3fn, max_branches=64)
    rows = lambda *s: torch.randn(*s, kv, 128, generator=g, device="cuda").bfloat16()  # noqa: E731
    roots = [pool.new_branch() for _ in range(n)]
    K, V = rows(n, prefix), rows(n, prefix)
    pool.append_kv(roots, K, V)
    kids = [c for k in pool.fork_batch(roots, [width] * n) for c in k]
    k, v = rows(n * width, leaf), rows(n * width, leaf)
    pool.append_kv(kids, k, v)
    q = torch.randn(n * width, 1, 4 * kv, 128, generator=g, device="cuda").bfloat16()
    out = pool.tree_attn_decode(q, kids)
    pool.sync()
    for i in range(n * width):
        kk, vv = (R.held(R.f64(torch.cat((a[i // width], b[i]))), "fp8") for a, b in ((K, k), (V, v)))
        ref = R.attention(R.f64(q[i]), kk, vv, np.ones((1, len(kk)), bool))
        assert (np.abs(R.f64(out[i]) - ref[0]) <= R.attention_bound("fp8", *ref)).all()
    pool.close()
