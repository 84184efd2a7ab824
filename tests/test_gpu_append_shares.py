"""How an append's rows are shared out among CTAs (a CTA per tile, parts of tiles, even shares over tiles' ends) changes
no row: a call of many branches gives what calls of one branch give, bit for bit."""
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


# (layers, branches, tokens, kv heads, query heads): one token; a tile of few turns; parts of tiles; shares over tiles' ends
# below one wave of tiles, just above one and two; one CTA a tile at nearly two waves and at more
SHAPES = [(1, 1, 1, 8, 32), (32, 32, 1, 8, 0), (1, 3, 40, 1, 0), (8, 32, 5, 8, 8), (4, 3, 33, 8, 5), (1, 2, 4096, 2, 3), (2, 30, 190, 2, 2),
          (1, 14, 800, 2, 1), (1, 28, 780, 1, 2), (1, 37, 500, 1, 1), (5, 17, 500, 1, 1), (600, 3, 20, 1, 1)]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
@pytest.mark.parametrize("turned", ["plain", "length", "given"])
@pytest.mark.parametrize("layers,n,new,kv,nq", SHAPES)
def test_many_branches_as_one_by_one(kind, turned, layers, n, new, kv, nq):
    dim = 128
    g = torch.Generator(device="cuda").manual_seed(new)
    rows = lambda h: torch.randn(layers, n, new, h, dim, generator=g, device="cuda").to(R.ROW_DTYPE[kind])   # noqa: E731
    k, v, q = rows(kv), rows(kv), rows(nq) if nq and turned != "plain" else None
    at = torch.randint(-5, 3000, (n, new, 2), generator=g, device="cuda").int()
    rope = Rope(96, axes=[0, 1] * 24) if turned == "given" else Rope(96)
    lens = [3 + 5 * (i % 4) for i in range(n)]
    blocks = sum((x + new) // 16 + 2 for x in lens)
    out = []
    for alone in (False, True):
        pool = Pool(blocks, 16, kv, dim, R.POOL_DTYPE[kind], n_layers=layers, max_branches=n + 1)
        br = [pool.new_branch() for _ in lens]
        lead = (lambda x: x if layers > 1 else x[0])
        for i, b in enumerate(br):   # (rows before: the same in both)
            z = lead(k[:, :1, :1].expand(-1, -1, lens[i], -1, -1).contiguous())
            pool.append_kv([b], z, z)
        turned_q = []
        for i in (range(n) if alone else [slice(None)]):
            s = slice(i, i + 1) if alone else i
            cut = lambda x: lead(x[:, s].contiguous())   # noqa: E731
            if turned == "plain":
                pool.append_kv(br[s], cut(k), cut(v))
            else:
                y = pool.append_rope(br[s], cut(k), cut(v), rope, Q=None if q is None else cut(q), positions=at[s] if turned == "given" else None)
                if y is not None:
                    turned_q.append(y if layers > 1 else y[None])
        got = [pool.read_kv(br, lens, [new] * n, layer=l) for l in range(layers if layers < 50 else 2)]
        pool.sync()
        out.append([x for kv_ in got for x in kv_] + ([torch.cat(turned_q, 1)] if turned_q else []))
        pool.close()
    assert len(out[0]) == len(out[1]) and all(torch.equal(a, b) for a, b in zip(*out))
    assert all(bool(x.float().abs().sum() > 0) for x in out[0])
