"""Cross attention through the C-ABI library: every query sees every row of its branch, of whatever length, against
64 bits within the derived bounds."""
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
    def __init__(self, kind, lens, kv, group, seed=0, dim=128, **kw):
        self.kind, self.kv, self.nq, self.dim = kind, kv, kv * group, dim
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = Pool(sum(3 * (x // 16 + 6) for x in lens) + 16, 16, kv, dim, R.POOL_DTYPE[kind], max_branches=8 * len(lens) + 16, **kw)
        self.br = [self.pool.new_branch() for _ in lens]
        for b, x in zip(self.br, lens):
            if x:
                self.append([b], x)

    def rows(self, *shape):
        return torch.randn(*shape, self.dim, generator=self.g, device="cuda").to(R.ROW_DTYPE[self.kind])

    def append(self, br, n):
        self.pool.append_kv(br, self.rows(len(br), n, self.kv), self.rows(len(br), n, self.kv))

    def attend(self, br, q_len, **kw):
        q = self.rows(len(br), q_len, self.nq)
        out = self.pool.tree_attn_cross(q, br, **kw)
        self.pool.sync()
        for i, b in enumerate(br):
            n = self.pool.branch_len(b)
            got = R.f64(out[i])
            if n == 0:
                assert (got == 0).all()
                continue
            K, V = (R.f64(x) for x in self.pool.read_kv([b], [0], [n]))
            ref = R.attention(R.f64(q[i]), K, V, np.ones((q_len, n), bool))
            err, bound = np.abs(got - ref[0]), R.attention_bound(self.kind, *ref)
            assert (err <= bound).all(), (i, float(err.max()), float((err / bound).max()))
        return q, out


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_len", [1, 2, 5, 16, 33, 130])
@pytest.mark.parametrize("kv,group", [(1, 1), (2, 4), (1, 8), (2, 5)])
def test_sizes(kind, q_len, kv, group):
    c = Case(kind, [0, 1, 15, 16, 17, 131], kv, group, seed=q_len)
    c.attend(c.br, q_len)
    c.attend(c.br[1:], q_len)
    c.attend(c.br[:1], q_len)      # no rows at all
    c.pool.close()


@pytest.mark.parametrize("dim", [32, 96, 256])
def test_head_dims_of_fp32_pools(dim):
    c = Case("fp32", [3, 40, 0], 2, 3, dim=dim)
    c.attend(c.br, 50)
    c.attend(c.br[2:], 5)
    c.pool.close()


@pytest.mark.parametrize("kind", KINDS)
def test_long_queries_and_long_states(kind):
    c = Case(kind, [1500, 700, 0], 1, 4)
    c.attend(c.br, 300)
    c.attend(c.br[:1], 1)
    c.attend(c.br[:1], 448)
    c.pool.close()


@pytest.mark.parametrize("kind", KINDS)
def test_a_single_query_is_the_decode_call(kind):
    """One query sees the whole branch in both calls; more than one see different rows, though the plans look alike."""
    c = Case(kind, [77, 300, 33], 2, 4)
    for q_len in (1, 8):
        q, out = c.attend(c.br, q_len)
        causal = c.pool.tree_attn_decode(q, c.br)
        if q_len == 1 and kind == "fp32":
            # two kernels, two orders of the sums: with |out - x| <= b (checked by attend) and |causal - x| <= b for
            # the exact x and its bound b, |out - causal| <= |out - x| + |x - causal| <= 2 b
            for i, b in enumerate(c.br):
                n = c.pool.branch_len(b)
                K, V = (R.f64(x) for x in c.pool.read_kv([b], [0], [n]))
                ref = R.attention(R.f64(q[i]), K, V, np.ones((1, n), bool))
                assert (np.abs(R.f64(out[i]) - R.f64(causal[i])) <= 2 * R.attention_bound(kind, *ref)).all()
        else:
            assert torch.equal(out[:, -1:], causal[:, -1:]) if q_len == 1 else not torch.equal(out, causal)
        again = c.pool.tree_attn_cross(q, c.br)
        assert torch.equal(again, out)
        trees = list(range(-1, q_len - 1))
        assert c.pool.tree_attn_draft(q, c.br, trees).shape == out.shape
        assert torch.equal(c.pool.tree_attn_cross(q, c.br), out)
    c.pool.close()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("opts", [dict(tc_min_rows=-1), dict(tc_min_rows=1), dict(device_planning=1), dict(device_planning=-1),
                                  dict(pack_segments=-1), dict(fold_segments=-1), dict(tc_sms=8)])
def test_planning_options(kind, opts):
    c = Case(kind, [500, 37, 250], 2, 4, **opts)
    kids = [x for b in c.br for x in c.pool.fork(b, 3)]
    c.attend(kids, 9)
    c.append(kids[1:7], 21)
    c.attend(kids, 9)
    c.attend(kids[::-1], 40)
    c.pool.close()


@pytest.mark.parametrize("kind", KINDS)
def test_states_that_grow(kind):
    """Streaming encoders append between calls: lengths inside a block, new blocks, an empty branch's first rows."""
    c = Case(kind, [0, 5, 31, 200], 2, 2)
    c.attend(c.br, 12)
    for n in (1, 3, 14, 40):
        c.append(c.br[:3], n)
        c.attend(c.br, 12)
    c.pool.truncate(c.br, [3, 0, 16, 170])
    c.attend(c.br, 12)
    c.attend(c.br, 70)
    c.pool.close()


@pytest.mark.parametrize("kind", KINDS)
def test_sequences_that_share_states(kind):
    """Beams and samples of one prompt: forks of the states' branch, read once for all."""
    c = Case(kind, [900], 2, 2)
    kids = c.pool.fork(c.br[0], 6)
    c.attend(kids, 7)
    # 56 whole blocks of 2 heads, read together; the partly filled one counts as each fork's own
    assert c.pool.last_plan_stats()["unique_tiles"] == 2 * (56 + 6)
    c.attend(kids, 100)
    c.pool.close()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_what_stands_behind_the_end_touches_nothing(kind):
    c = Case(kind, [40, 40], 1, 4)
    bad = torch.full((2, 7, 1, 128), float("nan"), device="cuda").to(R.ROW_DTYPE[kind])
    c.pool.append_kv(c.br, bad, bad)
    c.pool.truncate(c.br, [40, 33])
    for q_len in (1, 20, 100):
        c.attend(c.br, q_len)
    c.append(c.br, 2)
    c.attend(c.br, 20)
    c.pool.close()


def test_layers():
    pool = Pool(64, 16, 2, 128, torch.bfloat16, max_branches=8, n_layers=3)
    br = [pool.new_branch() for _ in range(2)]
    x = torch.randn(3, 2, 45, 2, 128, device="cuda").bfloat16()
    pool.append_kv(br, x, x)
    q = torch.randn(2, 11, 8, 128, device="cuda").bfloat16()
    for l in range(3):
        out = pool.tree_attn_cross(q, br, layer=l)
        for i in range(2):
            ref = R.attention(R.f64(q[i]), R.f64(x[l, i]), R.f64(x[l, i]), np.ones((11, 45), bool))
            assert (np.abs(R.f64(out[i]) - ref[0]) <= R.attention_bound("bf16", *ref)).all()
    with pytest.raises(DendriteError):
        pool.tree_attn_cross(q, br, layer=3)
    pool.close()


def test_compressed_pools():
    """Every query of a long call gives what it gives alone."""
    pool = Pool(64, 16, 2, 128, torch.bfloat16, turbo=W.turbo_codec(1), max_branches=8)
    br = [pool.new_branch() for _ in range(3)]
    x = torch.randn(2, 45, 2, 128, device="cuda").bfloat16()
    pool.append_kv(br[:2], x, x)
    q = torch.randn(3, 6, 8, 128, device="cuda").bfloat16()
    out = pool.tree_attn_cross(q, br)
    assert out[2].eq(0).all()
    for j in range(6):
        one = pool.tree_attn_decode(q[:2, j:j + 1].contiguous(), br[:2])
        # both sum the same terms, in fp32 and in tiles of other rows; then half a step of bf16 each
        assert torch.allclose(out[:2, j:j + 1].float(), one.float(), rtol=2.0 ** -7, atol=2.0 ** -12)
    pool.close()


def test_another_stream_and_two_calls_at_once():
    cases = [Case("bf16", [300, 20], 2, 4, seed=s) for s in (1, 2)]
    qs = [c.rows(2, 30, 8) for c in cases]
    want = [c.pool.tree_attn_cross(q, c.br) for c, q in zip(cases, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [c.pool.tree_attn_cross(q, c.br, stream=s) for c, q, s in zip(cases, qs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    empty = cases[0].pool.new_branch()
    z = cases[0].pool.tree_attn_cross(qs[0][:1].contiguous(), [empty], stream=streams[0])
    torch.cuda.synchronize()
    assert z.eq(0).all()
    for c in cases:
        c.pool.close()


def test_refusals():
    c = Case("bf16", [20, 20], 2, 2)
    q = c.rows(2, 4, 4)
    out = torch.empty_like(q)
    for args, kw in (((q, c.br[:1]), {}), ((q, [c.br[0]] * 2), {}), ((q, [c.br[0], 99]), {}), ((q.float(), c.br), {}), ((q.cpu(), c.br), {}),
                     ((q[:, :, :3].contiguous(), c.br), {}), ((q, c.br), dict(out=out[:1])), ((q, c.br), dict(layer=1)),
                     ((q[:, :0].contiguous(), c.br), {})):
        with pytest.raises(DendriteError):
            c.pool.tree_attn_cross(*args, **kw)
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        graph.capture_begin()
        try:
            with pytest.raises(DendriteError):
                c.pool.tree_attn_cross(q, c.br, out=out)
            out.zero_()
        finally:
            graph.capture_end()
    c.attend(c.br, 4)
    c.pool.close()


def test_a_step_with_images_thinning_drafts_and_an_encoder():
    """The calls together, as a decoding loop over image and audio inputs makes them: prompts turned by three axes, rows
    thinned out, drafts at positions that go on from the prompt's, their attention and cross attention, verification,
    acceptance; each against 64 bits."""
    from _verify import verified

    rng = random.Random(11)
    kv, nq, new, vocab = 2, 8, 7, 200
    c = Case("bf16", [60, 45], kv, 4)                      # the encoder's states
    self_pool = Pool(128, 16, kv, 128, torch.bfloat16, max_branches=16)
    rope = Rope(128, axes=[0] * 16 + [1] * 24 + [2] * 24)
    freq, _ = R.frequencies(128)
    br = [self_pool.new_branch() for _ in range(2)]
    at = torch.randint(0, 50, (2, 90, 3), device="cuda").int()
    self_pool.append_rope(br, c.rows(2, 90, kv), c.rows(2, 90, kv), rope, positions=at)
    top = at.amax((1, 2)) + 1
    lists = [sorted(rng.sample(range(8, 90), 40)) for _ in br]
    kids = self_pool.fork_rows(br, [8, 8], [40, 40], torch.tensor(lists, dtype=torch.int32, device="cuda").flatten())
    self_pool.free(br)
    for step in range(3):
        trees = [R.tree(rng, new) for _ in kids]
        depth = torch.tensor([R.depths(t) for t in trees], device="cuda", dtype=torch.int32)
        pos = (top[:, None] + depth).int()[..., None].expand(-1, -1, 3)
        k, v, q = c.rows(2, new, kv), c.rows(2, new, kv), c.rows(2, new, nq)
        lens = [self_pool.branch_len(b) for b in kids]
        tq = self_pool.append_rope(kids, k, v, rope, Q=q, positions=pos)
        out = self_pool.tree_attn_draft(tq, kids, trees)
        for i, b in enumerate(kids):
            y, size = R.rotate(R.f64(q[i]), pos[i, :, 0].cpu().numpy(), freq, 128, False)
            assert (np.abs(R.f64(tq[i]) - y) <= R.ROPE_ERR * size + 2.0 ** -8 * (np.abs(y) + R.ROPE_ERR * size)).all()
            K, V = (R.f64(x) for x in self_pool.read_kv([b], [0], [lens[i] + new]))
            ref = R.attention(R.f64(tq[i]), K, V, R.seen(trees[i], lens[i]))
            assert (np.abs(R.f64(out[i]) - ref[0]) <= R.attention_bound("bf16", *ref)).all()
        c.attend(c.br, new)
        p = torch.softmax(2 * torch.randn(2, 1 + new, vocab, device="cuda"), -1)
        dq = torch.softmax(p[:, :new].log() + 0.3 * torch.randn(2, new, vocab, device="cuda"), -1)
        tokens = torch.stack([torch.multinomial(dq[i, [x + 1 for x in trees[i]]], 1)[:, 0] for i in range(2)]).int()
        u, s = torch.rand(2, new, device="cuda"), torch.rand(2, device="cuda")
        path, size, token = self_pool.verify_draft(tokens, p, trees, u, s, draft=dq)
        keep = [x[:n] for x, n in zip(path.tolist(), size.tolist())]
        for i in range(2):
            assert (keep[i], token[i].item()) == verified(R.f64(p[i]), R.f64(dq[i]), tokens[i].tolist(), trees[i], u[i].tolist(), s[i].item())
        rows = [[x.clone() for x in self_pool.read_kv([b], [0], [lens[i] + new])] for i, b in enumerate(kids)]
        self_pool.accept_draft(kids, new, keep)
        for i, b in enumerate(kids):
            want = list(range(lens[i])) + [lens[i] + j for j in keep[i]]
            assert all(torch.equal(x, y[want]) for x, y in zip(self_pool.read_kv([b], [0], [len(want)]), rows[i]))
        top = top + size + 1
    self_pool.sync()
    self_pool.close()
    c.pool.close()


@pytest.mark.parametrize("dim", range(32, 257, 32))
def test_row_counts_of_fp32_pools(dim):
    """Units of 4, 8, .. 128 rows, filled, just passed and in pieces, over ends on both sides of 32 tokens."""
    c = Case("fp32", [1, 31, 32, 33, 500], 2, 1, dim=dim)
    for q_len in (1, 2, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 130):
        c.attend(c.br, q_len)
    c.pool.close()


def test_fp32_rows_of_several_branches_in_one_unit():
    """Forks of one length share units whose rows end at different positions of a shared block once they are cut."""
    c = Case("fp32", [700], 1, 3)
    kids = c.pool.fork(c.br[0], 9)
    c.pool.truncate(kids, [700, 699, 689, 688, 673, 672, 300, 17, 0])
    for q_len in (1, 2, 5, 11, 40):
        c.attend(kids, q_len)
    c.append(kids, 3)
    c.attend(kids, 5)
    c.pool.close()


def test_what_stands_behind_the_end_touches_nothing_in_fp32():
    c = Case("fp32", [40, 40], 1, 4)
    bad = torch.full((2, 7, 1, 128), float("nan"), device="cuda")
    c.pool.append_kv(c.br, bad, bad)
    kid = c.pool.fork(c.br[0], 1)[0]      # still holds those rows, in the blocks that the first branch reads
    c.pool.truncate(c.br, [40, 33])
    for q_len in (1, 2, 20, 100):
        c.attend(c.br, q_len)
        q = c.rows(3, q_len, 4)
        out = R.f64(c.pool.tree_attn_cross(q, [c.br[0], kid, c.br[1]]))
        assert np.isnan(out[1]).all() and np.isfinite(out[[0, 2]]).all()
        for i, b in ((0, c.br[0]), (2, c.br[1])):
            n = c.pool.branch_len(b)
            K, V = (R.f64(x) for x in c.pool.read_kv([b], [0], [n]))
            ref = R.attention(R.f64(q[i]), K, V, np.ones((q_len, n), bool))
            assert (np.abs(out[i] - ref[0]) <= R.attention_bound("fp32", *ref)).all()
    c.pool.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,q_len", [(13, 64), (25, 65), (19, 10)])
def test_units_shared_by_two_ctas(kind, n, q_len):
    """About as many units as CTAs, so that most CTAs end inside a unit that the next one began: their rows are joined,
    the same way whichever ends first, and every later call finds the counts of their meetings as the first did."""
    c = Case(kind, [300 - 7 * i for i in range(n)], 8, 4, seed=n)
    q, out = c.attend(c.br, q_len)
    for _ in range(20):
        assert torch.equal(c.pool.tree_attn_cross(q, c.br), out)
    c.append(c.br, 9)
    c.attend(c.br, q_len)
    c.pool.close()
