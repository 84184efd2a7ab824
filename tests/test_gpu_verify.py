"""Verification of drafted tokens through the C-ABI library, against rational arithmetic: paths, lengths and next
tokens are whole numbers and have to be equal."""
import random

import numpy as np
import pytest
import torch

import _rows as R
from _verify import verified
from copy_write_forked_gb300.dendrite import DendriteError, Pool

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()
    torch.cuda.set_device(0)


@pytest.fixture(scope="module")
def pool():
    p = Pool(16, 16, 1, 128, torch.bfloat16, max_branches=4)
    yield p
    p.sync()
    p.close()


def _case(n, t, vocab, kind, certain, g, spread=2.0, trees=None, shape="random", seed=0):
    """Inputs whose drafts are drawn from the draft's rows (of what is near the target's)."""
    rng = random.Random(seed)
    logits = spread * torch.randn(n, 1 + t, vocab, generator=g, device="cuda")
    p = torch.softmax(logits, -1).to(TYPES[kind])
    q = torch.softmax(logits[:, :t] + 0.5 * torch.randn(n, t, vocab, generator=g, device="cuda"), -1).to(TYPES[kind])
    trees = trees or [R.tree(rng, t, shape) for _ in range(n)]
    rows = torch.stack([q[i, [x + 1 for x in trees[i]]] for i in range(n)]).float()
    tokens = torch.multinomial(rows.view(n * t, vocab) + 1e-30, 1, generator=g).view(n, t).int()
    accept = torch.rand(n, t, generator=g, device="cuda")
    sample = torch.rand(n, generator=g, device="cuda")
    return tokens, p, torch.tensor(trees, dtype=torch.int32), accept, sample, None if certain else q


def _check(pool, case, got=None, which=None):
    tokens, p, trees, accept, sample, q = case
    path, size, token = got or pool.verify_draft(tokens, p, trees, accept, sample, draft=q)
    pool.sync()
    n, t = tokens.shape
    P, Q = R.f64(p), None if q is None else R.f64(q)
    flat = trees if trees.dim() == 2 else trees.expand(n, -1)
    for i in range(n) if which is None else which:
        want, nxt = verified(P[i], None if Q is None else Q[i], tokens[i].tolist(), flat[i].tolist(), accept[i].tolist(), sample[i].item())
        assert path[i].tolist() == want + [-1] * (t - len(want)), i
        assert size[i].item() == len(want) and token[i].item() == nxt, (i, size[i].item(), token[i].item(), len(want), nxt)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 31, 33, 100, 515, 1001])
@pytest.mark.parametrize("t,shape", [(1, "chain"), (2, "star"), (5, "chain"), (9, "random"), (17, "star"), (64, "random"), (33, "star")])
def test_sizes_and_trees(pool, kind, certain, vocab, t, shape):
    g = torch.Generator(device="cuda").manual_seed(vocab + t)
    _check(pool, _case(3, t, vocab, kind, certain, g, shape=shape, seed=t), which=range(3) if t * vocab < 9000 else [1])


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("vocab", [4097, 50257, 128256, 150001])
@pytest.mark.parametrize("n", [1, 40])
def test_large_vocabularies(pool, kind, certain, vocab, n):
    """Several CTAs a sequence: odd row lengths, rows that start at any address."""
    g = torch.Generator(device="cuda").manual_seed(vocab)
    _check(pool, _case(n, 4, vocab, kind, certain, g, seed=vocab), which=[0] if n == 1 else [3, 39])


@pytest.mark.parametrize("n", [2, 300])
def test_flat_rows_fall_to_the_right_token(pool, n):
    """Equal probabilities: 2^-16 apart, the borders meet the numbers exactly (a number on a border is the next token's)."""
    vocab = 65536
    p = torch.full((n, 2, vocab), 2.0 ** -16, device="cuda")
    sample = torch.arange(n, device="cuda") * (2.0 ** 24 // n) / 2.0 ** 24
    tokens, accept = torch.full((n, 1), -1, dtype=torch.int32, device="cuda"), torch.zeros(n, 1, device="cuda")
    _, size, token = pool.verify_draft(tokens, p, [-1], accept, sample)
    assert size.eq(0).all()
    assert torch.equal(token.long(), torch.floor(sample.double() * vocab).long())
    sample = torch.full((n,), 1 - 2.0 ** -24, device="cuda")
    assert pool.verify_draft(tokens, p, [-1], accept, sample)[2].eq(vocab - 1).all()


def test_borders(pool):
    """Dyadic rows: the comparisons at equality."""
    p = torch.tensor([[0.25, 0.375, 0.25, 0.125], [0, 0, 1, 0]], device="cuda").expand(1, 2, 4).contiguous()
    q = torch.tensor([[0.5, 0.25, 0.125, 0.125]], device="cuda").expand(1, 1, 4).contiguous()
    for x in range(4):
        for u in (0.0, 0.25, 0.49, 0.5, 0.51, 0.99):
            for s in (0.0, 0.25, 0.375, 0.5, 0.625, 0.75, 0.875):
                for draft in (q, None):
                    _check(pool, (torch.tensor([[x]], dtype=torch.int32, device="cuda"), p, torch.tensor([[-1]], dtype=torch.int32),
                                  torch.tensor([[u]], device="cuda"), torch.tensor([s], device="cuda"), draft))


@pytest.mark.parametrize("certain", [False, True])
def test_one_hot_targets_are_greedy_decoding(pool, certain):
    g = torch.Generator(device="cuda").manual_seed(3)
    tokens, p, trees, accept, sample, q = _case(6, 20, 300, "fp32", certain, g, seed=3)
    best = p.argmax(-1, keepdim=True)
    hot = torch.zeros_like(p).scatter_(-1, best, 1.0)
    for i in range(6):   # half of the drafts right
        for j in range(0, 20, 2):
            tokens[i, j] = best[i, trees[i, j] + 1, 0]
    case = (tokens, hot, trees, accept, sample, q)
    _check(pool, case)
    path, size, token = pool.verify_draft(tokens, hot, trees, accept, sample, draft=q)
    for i in range(6):
        row = 0 if size[i] == 0 else path[i, size[i] - 1].item() + 1
        assert token[i].item() == best[i, row, 0].item()


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("certain", [False, True])
def test_rows_that_leave_nothing(pool, kind, certain):
    """Empty rows, residuals without weight, drafted tokens that neither side holds likely, padding, tokens drafted twice,
    entries that are no probabilities."""
    g = torch.Generator(device="cuda").manual_seed(5)
    tokens, p, trees, accept, sample, q = _case(12, 8, 90, kind, certain, g, shape="star", seed=5)
    p[0] = 0                                            # no weight anywhere: -1
    p[1, 0] = 0                                         # none at the root
    if q is not None:
        q[2] = p[2, :8]                                 # the residual is empty: the target itself
        q[3, :, 10:] = 0
    tokens[2] = 89
    p[2, :, 89] = 0
    if q is not None:
        q[2, :, 89] = 0
    tokens[4] = -1                                      # nothing drafted
    tokens[5, 3:] = 90                                  # outside the vocabulary
    tokens[6] = tokens[6, 0]                            # the same token eight times
    p[7, :, ::3] = float("nan")
    p[7, :, 1::3] = -1.0
    p[8, :, 5] = float("inf")
    if q is not None:
        q[7, :, 2::5] = float("nan")
        q[8, :, 7] = float("-inf")
    tokens[9, :] = 2147483647
    tokens[10, :] = -2147483648
    accept[11] = 0.0                                    # accepted wherever there is weight
    _check(pool, (tokens, p, trees, accept, sample, q))
    out = pool.verify_draft(tokens, p, trees, accept, sample, draft=q)
    assert out[2][0].item() == -1 and out[1][0].item() == 0
    chain = torch.arange(-1, 7, dtype=torch.int32)
    _check(pool, (tokens, p, chain, accept, sample, q))   # one tree for all


def test_random_numbers_outside_their_range(pool):
    """Documented as in [0, 1); one that is not picks the first or the last token with weight, and nothing is left unwritten."""
    p = torch.tensor([0.0, 0.5, 0.5, 0.0], device="cuda").expand(4, 2, 4).contiguous()
    tokens = torch.full((4, 1), -1, dtype=torch.int32, device="cuda")
    sample = torch.tensor([1.0, -1.0, float("nan"), float("inf")], device="cuda")
    out = tuple(torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((4, 1), (4,), (4,)))
    path, size, token = pool.verify_draft(tokens, p, [-1], torch.zeros(4, 1, device="cuda"), sample, out=out)
    assert token.tolist() == [2, 1, 1, 2] and size.tolist() == [0] * 4 and path.tolist() == [[-1]] * 4


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_strides(pool, kind):
    """Rows of a padded vocabulary, and views that start at any element."""
    g = torch.Generator(device="cuda").manual_seed(6)
    tokens, p, trees, accept, sample, q = _case(3, 6, 1001, kind, False, g, seed=6)
    want = pool.verify_draft(tokens, p, trees, accept, sample, draft=q)
    for pad, off in ((7, 1), (23, 3), (64, 0)):
        wide = torch.full((3, 7, 1001 + pad), float("nan"), dtype=p.dtype, device="cuda")
        wide[:, :, off:off + 1001] = p
        widq = torch.full((3, 6, 1001 + pad), float("nan"), dtype=p.dtype, device="cuda")
        widq[:, :, off:off + 1001] = q
        got = pool.verify_draft(tokens, wide[:, :, off:off + 1001], trees, accept, sample, draft=widq[:, :, off:off + 1001])
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    one = pool.verify_draft(tokens[1:2], p[1:2], trees[1:2].contiguous(), accept[1:2], sample[1:2], draft=q[1:2])
    assert all(torch.equal(a[1:2], b) for a, b in zip(want, one))


def test_many_sequences(pool):
    """More tree bytes than travel as kernel parameters, and more sequences than run at once."""
    g = torch.Generator(device="cuda").manual_seed(7)
    case = _case(700, 40, 61, "fp32", False, g, seed=7)
    _check(pool, case, which=list(range(0, 700, 41)) + [699])
    _check(pool, _case(2000, 3, 700, "bf16", True, g, seed=8), which=[0, 1, 999, 1999])


def test_the_same_again_and_on_other_streams(pool):
    g = torch.Generator(device="cuda").manual_seed(8)
    cases = [_case(9, 12, 30011, "fp32", False, g, seed=s) for s in (1, 2)]
    want = [pool.verify_draft(c[0], c[1], c[2], c[3], c[4], draft=c[5]) for c in cases]
    torch.cuda.synchronize()
    other = Pool(16, 16, 1, 128, torch.bfloat16, max_branches=4)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):   # two calls at once, of two pools
        got = [p.verify_draft(c[0], c[1], c[2], c[3], c[4], draft=c[5], stream=s) for p, c, s in zip((pool, other), cases, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    other.close()


def test_rows_past_32_bit_offsets(pool):
    """A target of more than 2^32 elements: the last sequence's rows."""
    n, t, vocab = 36, 1, 60_000_001
    p = torch.zeros(n, 1 + t, vocab, dtype=torch.bfloat16, device="cuda")
    p[n - 1, 1, vocab - 1] = 0.5
    p[n - 1, 1, 17] = 0.5
    p[n - 1, 0, 59_999_990] = 1.0
    tokens = torch.full((n, t), 59_999_990, dtype=torch.int32, device="cuda")
    sample = torch.full((n,), 0.6, device="cuda")
    path, size, token = pool.verify_draft(tokens, p, [-1], torch.full((n, t), 0.5, device="cuda"), sample)
    assert size.tolist() == [0] * (n - 1) + [1] and token.tolist() == [-1] * (n - 1) + [vocab - 1]
    del p


def test_refusals(pool):
    g = torch.Generator(device="cuda").manual_seed(9)
    tokens, p, trees, accept, sample, q = _case(3, 5, 40, "fp32", False, g)
    good = dict(tokens=tokens, target=p, parents=trees, accept=accept, sample=sample, draft=q)
    pool.verify_draft(**good)
    mixed = torch.zeros(64, dtype=torch.int32, device="cuda")
    bad = [dict(tokens=tokens.long()), dict(tokens=tokens[:2]), dict(tokens=tokens.cpu()), dict(target=p.half()), dict(target=p[:, :5]),
           dict(target=p.cpu()), dict(parents=None), dict(parents=[-1, 0, 1]), dict(parents=[-1, 1, 0, 0, 0]), dict(parents=[-2, 0, 0, 0, 0]),
           dict(accept=accept[:, :4]), dict(accept=accept.double()), dict(sample=sample[:2]), dict(draft=q.bfloat16()), dict(draft=p),
           dict(target=p.transpose(1, 2).contiguous().transpose(1, 2)), dict(target=p[:, :, ::2]), dict(draft=q[:, :, :39]),
           dict(out=(mixed[:15].view(3, 5), mixed[10:13], mixed[20:23])), dict(out=(mixed[:15].view(3, 5), mixed[16:19], mixed[18:21])),
           dict(out=(tokens, mixed[:3], mixed[3:6])), dict(out=(mixed[:15].view(3, 5), sample.view(torch.int32), mixed[20:23])),
           dict(out=(mixed[:15].view(3, 5), mixed[16:19]))]
    for kw in bad:
        with pytest.raises((DendriteError, ValueError)):
            pool.verify_draft(**(good | kw))
    none = torch.zeros(3, 0, dtype=torch.int32, device="cuda")
    with pytest.raises(DendriteError):
        pool.verify_draft(none, p[:, :1].contiguous(), torch.zeros(3, 0, dtype=torch.int32), accept[:, :0].contiguous(), sample)
    long = _case(1, 65, 4, "fp32", True, g)
    with pytest.raises(DendriteError):
        pool.verify_draft(long[0], long[1], long[2], long[3], long[4])
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    out = tuple(torch.zeros(x, dtype=torch.int32, device="cuda") for x in ((3, 5), (3,), (3,)))
    with torch.cuda.stream(s):
        graph.capture_begin()
        try:
            with pytest.raises(DendriteError):
                pool.verify_draft(**good, out=out)
            out[1].add_(1)   # (a graph of something)
        finally:
            graph.capture_end()
    empty = pool.verify_draft(tokens[:0], p[:0], torch.zeros(0, 5, dtype=torch.int32), accept[:0], sample[:0])
    assert [x.numel() for x in empty] == [0, 0, 0]
    pool.sync()


@pytest.mark.parametrize("vocab", [5, 70000])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_least_weights_still_give_a_token(pool, vocab, kind):
    """One weight of the type's least positive number: its token, however near one the sample is (sample times the
    weight rounds to the weight itself)."""
    least = 2.0 ** (-149 if kind == "fp32" else -133)
    samples = [0.0, 0.5, 1 - 2.0 ** -24]
    n = len(samples)
    for at in (0, 3, vocab - 1):
        p = torch.zeros(n, 2, vocab, device="cuda", dtype=TYPES[kind])
        p[:, 0, at] = least
        tokens, accept = torch.full((n, 1), -1, dtype=torch.int32, device="cuda"), torch.zeros(n, 1, device="cuda")
        out = tuple(torch.full(s, 7, dtype=torch.int32, device="cuda") for s in ((n, 1), (n,), (n,)))
        _, size, token = pool.verify_draft(tokens, p, [-1], accept, torch.tensor(samples, device="cuda"), out=out)
        assert size.tolist() == [0] * n and token.tolist() == [at] * n


@pytest.mark.parametrize("certain", [False, True])
def test_small_rows(pool, certain):
    """Rows that add up to 2^-90: the digits that the sums keep are all there."""
    g = torch.Generator(device="cuda").manual_seed(11)
    tokens, p, trees, accept, sample, q = _case(3, 6, 500, "fp32", certain, g, seed=11)
    _check(pool, (tokens, p * 2.0 ** -90, trees, accept, sample, None if q is None else q * 2.0 ** -90))


@pytest.mark.parametrize("vocab", [6, 30000])
def test_rows_past_the_largest_float(pool, vocab):
    """The sum of such a row is no number: -1, and nothing else is touched."""
    p = torch.full((2, 2, vocab), 1.0 / vocab, device="cuda")
    p[0, 0] = 3e38
    tokens, accept = torch.full((2, 1), -1, dtype=torch.int32, device="cuda"), torch.zeros(2, 1, device="cuda")
    out = tuple(torch.full(s, 7, dtype=torch.int32, device="cuda") for s in ((2, 1), (2,), (2,)))
    path, size, token = pool.verify_draft(tokens, p, [-1], accept, torch.tensor([0.5, 0.0], device="cuda"), out=out)
    assert size.tolist() == [0, 0] and token.tolist() == [-1, 0] and path.eq(-1).all()
