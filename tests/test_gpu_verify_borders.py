"""Verification next to borders, and where a residual is a small part of its row: whole numbers, equal to those of
rational arithmetic wherever a number is farther from its border than the sums are documented to be off."""
import math
import random
from fractions import Fraction

import numpy as np
import pytest
import torch

from _verify import verified
from copy_write_forked_gb300.dendrite import Pool

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
BITS = {"fp32": 24, "bf16": 8}


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


def test_a_border_between_two_ctas(pool):
    """Half of a row's sum ends with one CTA's share, and the next share is empty: however the two halves' sums are
    rounded (they have the same terms in another order), one token is given, on one side of the border."""
    rng, n, vocab = random.Random(1), 16, 32768     # 16 CTAs a sequence, of 2,048 tokens each
    tokens, accept = torch.full((n, 1), -1, dtype=torch.int32, device="cuda"), torch.zeros(n, 1, device="cuda")
    sample = torch.full((n,), 0.5, device="cuda")
    for _ in range(16):
        p = np.zeros((n, 2, vocab), np.float32)
        for i in range(n):
            big = [np.float32(rng.uniform(0.02, 0.06) * 2.0 ** rng.choice([0, 0, -1, -3])) for _ in range(7)]
            pairs = [(x, np.float32(float(x) * 2.0 ** -25 * rng.uniform(0.1, 0.9))) for x in big]
            for first, some in ((0, pairs), (8, rng.sample(pairs, 7))):
                for k, (x, y) in enumerate(some):
                    p[i, 0, 2048 * (first + k)], p[i, 0, 2048 * (first + k) + 1] = x, y
        got = pool.verify_draft(tokens, torch.from_numpy(p).cuda(), [-1], accept, sample)[2].tolist()
        # the border: behind the last token of the seventh share, before the first of the ninth
        assert all(x in (2048 * 6 + 1, 2048 * 8) for x in got), got


def _pieces(x, bits):
    """x > 0 as a sum of numbers of that many bits, each exact, largest first."""
    out = []
    while x > 0:
        e = math.frexp(float(x))[1]
        step = Fraction(2) ** (e - bits)
        y = x // step * step
        if y == 0:   # (x was rounded up to the next power of two)
            y = x // (step / 2) * (step / 2)
        out.append(float(y))
        x -= y
    return out


def _weights(rng, kind, n_before, n_after, ratio, scale, side):
    """Weights of the type's digits, of size about `scale`: the first n_before of them add up to `ratio` (a binary
    fraction) of all, and to side * 2^-38 of all more."""
    bits = BITS[kind]

    def some():
        return Fraction(rng.randrange(2 ** (bits - 1), 2 ** bits)) * Fraction(2) ** (-bits - rng.randrange(5)) * Fraction(scale)

    while True:
        before = [some() for _ in range(n_before)]
        a = sum(before)
        d = Fraction(2) ** -38 * Fraction(2) ** math.frexp(float(a / ratio))[1]   # (at least 2^-38 of the whole, at most 2^-37)
        whole = (a - side * d) / ratio
        after = [some() for _ in range(n_after)]
        left = whole - a - sum(after)
        if left > 0:
            rest = _pieces(left, bits)
            if len(rest) <= 12 and rest[-1] > 2.0 ** -100:
                return [float(x) for x in before], [float(x) for x in after] + rest


# 32 tokens of one thread's share where 200 sequences of 16,384 tokens take a CTA each: 16-byte words 32 lanes apart
# (of the first warp's first lane), and the same number anywhere in the row
PLACES = {"fp32": [128 * k + j for k in range(8) for j in range(4)], "bf16": [256 * k + j for k in range(4) for j in range(8)]}
VOCAB = 16384


def _place(rng, kind, together):
    return PLACES[kind] if together else sorted(rng.sample(range(VOCAB), 32))


def _common(g, n, kind):
    """Rows that target and draft have alike: nothing is left of them."""
    x = torch.softmax(2 * torch.randn(n, VOCAB, generator=g), -1)
    return (x * 0.05).to(TYPES[kind]).double().numpy()


def _run(pool, kind, tokens, p, q, accept, sample, expect, exactly=4):
    """One star of a tree for all sequences; `expect`: the outcome (path, token) by construction, `exactly` of them by
    rational arithmetic too."""
    t = tokens.shape[1]
    P = torch.from_numpy(p).to(TYPES[kind])
    assert (P.double().numpy() == p).all()
    Q = None if q is None else torch.from_numpy(q).to(TYPES[kind])
    assert q is None or (Q.double().numpy() == q).all()
    n = len(p)
    T = torch.zeros(n, 1 + t, VOCAB, dtype=TYPES[kind])
    T[:, 0] = P
    D = None
    if Q is not None:
        D = torch.zeros(n, t, VOCAB, dtype=TYPES[kind])
        D[:, 0] = Q
    path, size, token = pool.verify_draft(tokens.cuda(), T.cuda(), [-1] * t, accept.cuda(), sample.cuda(), draft=None if D is None else D.cuda())
    pool.sync()
    got = [(a[:k], x) for a, k, x in zip(path.tolist(), size.tolist(), token.tolist())]
    for i in range(exactly):
        assert verified(T[i].tolist(), None if D is None else D[i].tolist(), tokens[i].tolist(), [-1] * t, accept[i].tolist(), sample[i].item()) == expect[i]
    wrong = [(i, a, b) for i, (a, b) in enumerate(zip(got, expect)) if a != b]
    assert not wrong, (len(wrong), wrong[:4])


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("refusals", [1, 3])
@pytest.mark.parametrize("scale", [2.0 ** -10, 2.0 ** -16, 2.0 ** -20])
@pytest.mark.parametrize("together", [True, False])
@pytest.mark.parametrize("n", [200, 6])
def test_small_residuals_of_drafts(pool, kind, refusals, scale, together, n):
    """Target and draft agree on a token of 0.9 and on the tail; what is left is a 2^-10th to a 2^-20th of the row, and the
    number falls 2^-38 of it beside a border."""
    rng, g = random.Random(n + refusals), torch.Generator().manual_seed(n)
    p = _common(g, n, kind)
    big = float(torch.tensor(0.9).to(TYPES[kind]))
    q, expect = p.copy(), []
    for i in range(n):
        side = 1 if rng.random() < 0.5 else -1
        before, after = _weights(rng, kind, 9, 9, Fraction(1, 2), scale, side)
        at = _place(rng, kind, together)
        mid = at[len(before)]
        where = at[:len(before)] + at[len(before) + 1:len(before) + 1 + len(after)]
        p[i, mid] = q[i, mid] = big
        p[i, where], q[i, where] = before + after, 0
        expect.append(([], where[8] if side > 0 else where[9]))
    first = VOCAB - refusals
    p[:, first:], q[:, first:] = 0, 2.0 ** -10        # the drafted tokens: the target has none of them
    tokens = torch.arange(first, VOCAB, dtype=torch.int32).expand(n, -1).contiguous()
    _run(pool, kind, tokens, p, q, torch.full((n, refusals), 0.5), torch.full((n,), 0.5), expect)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("scale", [2.0 ** -10, 2.0 ** -16, 2.0 ** -20])
@pytest.mark.parametrize("together", [True, False])
@pytest.mark.parametrize("n", [200, 6])
def test_small_rests_of_certain_drafts(pool, kind, scale, together, n):
    """The refused token had nearly all: the next token's number, and the next draft's, fall 2^-38 of the rest beside a
    border."""
    rng = random.Random(n)
    p, expect = np.zeros((2 * n, VOCAB)), []
    tokens = torch.full((2 * n, 2), -1, dtype=torch.int32)
    for i in range(2 * n):
        side = 1 if rng.random() < 0.5 else -1
        sibling = i >= n                                   # the first token with weight is a draft too, of about half the rest
        before, after = _weights(rng, kind, 1 if sibling else 9, 0 if sibling else 9, Fraction(1, 2), scale, side)
        at = _place(rng, kind, together)
        mid = at[len(before)]
        where = at[:len(before)] + at[len(before) + 1:len(before) + 1 + len(after)]
        p[i, mid] = float(torch.tensor(0.9).to(TYPES[kind]))
        p[i, where] = before + after
        tokens[i, 0] = mid
        if sibling:
            tokens[i, 1] = where[0]
            # accepted where half of the rest is less than its weight; the accepted node's row is empty
            expect.append(([1], -1) if side > 0 else ([], where[1]))
        else:
            expect.append(([], where[8] if side > 0 else where[9]))
    accept = torch.full((2 * n, 2), 0.5)
    accept[:, 0] = 1 - 2.0 ** -24
    sample = torch.full((2 * n,), 0.5)
    sample[n:] = 0.0
    _run(pool, kind, tokens[:n], p[:n], None, accept[:n], sample[:n], expect[:n])
    _run(pool, kind, tokens[n:], p[n:], None, accept[n:], sample[n:], expect[n:])


@pytest.mark.parametrize("n", [200, 6])
def test_siblings_behind_a_small_residual(pool, n):
    """A second child whose number is 2^-38 of the border: 0.5 q(x) S against the weight p(x) - q(x) of some 2^-22."""
    rng, g, kind = random.Random(3), torch.Generator().manual_seed(4), "fp32"
    p = _common(g, n, kind)
    q, expect = p.copy(), []
    tokens = torch.zeros(n, 2, dtype=torch.int32)
    for i in range(n):
        side = 1 if rng.random() < 0.5 else -1
        at = _place(rng, kind, True)
        w = rng.randrange(9, 16) * 2.0 ** -24              # exact above one half
        d = Fraction(2) ** -38 * Fraction(w)
        rest = _pieces(3 * Fraction(w) - 4 * side * d, 24)  # S = 4 w - 4 side d: 0.5 * 0.5 * S < w where side > 0
        rest = [x / 2 for x in rest[:1] * 2] + rest[1:]
        p[i, at[0]], q[i, at[0]] = 0.5 + w, 0.5
        p[i, at[1]] = q[i, at[1]] = float(torch.tensor(0.9))
        where = at[2:2 + len(rest)]
        p[i, where], q[i, where] = rest, 0
        tokens[i, 0], tokens[i, 1] = VOCAB - 1, at[0]
        # refused: c is 1 + S, which leaves nothing of x; the least token of the rest
        expect.append(([1], -1) if side > 0 else ([], where[0]))
    p[:, VOCAB - 1], q[:, VOCAB - 1] = 0, 2.0 ** -10
    _run(pool, kind, tokens, p, q, torch.full((n, 2), 0.5), torch.zeros(n), expect)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("near", [2.0 ** -4, 2.0 ** -10, 2.0 ** -16])
@pytest.mark.parametrize("n,vocab", [(160, 515), (8, 4500)])
def test_drafts_near_the_target(pool, kind, near, n, vocab):
    """Stars whose children are all refused, of drafts near their target: residuals of residuals, a small part of the
    row each.  (Borders are some 2^-12 of S apart, and c / S up to some 2^20: a number is within 2^-24 of one, 2^-44 c / S,
    in one of a thousand sequences or less; these seeds have none.)"""
    g = torch.Generator().manual_seed(int(1 / near) + n)
    logits = 2 * torch.randn(n, vocab, generator=g)
    p = torch.softmax(logits, -1).to(TYPES[kind])
    q = torch.softmax(logits + near * torch.randn(n, vocab, generator=g), -1).to(TYPES[kind])
    t = 5
    target, draft = torch.zeros(n, 1 + t, vocab, dtype=p.dtype), torch.zeros(n, t, vocab, dtype=p.dtype)
    target[:, 0], draft[:, 0] = p, q
    # tokens that the draft holds likelier than the target (those are refused), as far as there are any
    tokens = (q.float() / p.float().clamp(min=1e-30)).topk(t, -1).indices.int()
    accept = torch.full((n, t), 1 - 2.0 ** -24)
    sample = torch.rand(n, generator=g)
    path, size, token = pool.verify_draft(tokens.cuda(), target.cuda(), [-1] * t, accept.cuda(), sample.cuda(), draft=draft.cuda())
    pool.sync()
    for i in range(0, n, 5 if n > 100 else 1):
        want, nxt = verified(target[i].tolist(), draft[i].tolist(), tokens[i].tolist(), [-1] * t, accept[i].tolist(), sample[i].item())
        assert (path[i].tolist()[:size[i]], token[i].item()) == (want, nxt), i


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [200, 6])
def test_many_refusals_of_certain_drafts(pool, kind, n):
    """Sixty-three refused tokens, most of them of digits that a sum of one does not hold, leave some 2^-8.5 of the row;
    the last child's number is 2^-38 of that beside its border."""
    rng = random.Random(5)
    p, expect = np.zeros((n, VOCAB)), []
    tokens = torch.zeros(n, 64, dtype=torch.int32)
    digits = lambda x: float(torch.tensor(x).to(TYPES[kind]))   # noqa: E731
    for i in range(n):
        side = 1 if rng.random() < 0.5 else -1
        w = Fraction(rng.randrange(2 ** (BITS[kind] - 1), 2 ** BITS[kind])) * Fraction(2) ** (-BITS[kind] - 9)
        d = Fraction(2) ** -38 * Fraction(2) ** math.frexp(float(2 * w))[1]
        rest = _pieces(w - 2 * side * d, BITS[kind])      # all that is left: 2 (w - side d)
        at = rng.sample(range(VOCAB), 64 + len(rest))
        lost = [2.0 ** (-26 if kind == "fp32" else -43) * rng.uniform(1, 4) for _ in range(56)] + [rng.uniform(0.05, 0.25) for _ in range(7)]
        p[i, at[:63]] = [digits(x) for x in lost]
        p[i, at[63]] = w
        p[i, at[64:]] = rest
        tokens[i] = torch.tensor(at[:64])
        expect.append(([63], -1) if side > 0 else ([], min(at[64:])))
    accept = torch.full((n, 64), 1 - 2.0 ** -24)
    accept[:, 63] = 0.5
    _run(pool, kind, tokens, p, None, accept, torch.zeros(n), expect)


def _outcome(p, q, tokens, accept, sample):
    """A star's outcome in rational arithmetic, and whether every number is farther from its border than the sums are
    documented to be off: 2^-40 of what is left, 2^-44 c / S from the second refusal on."""
    exact = lambda row: [Fraction(x) for x in row]   # noqa: E731
    p, q = exact(p), exact(q)
    w, S, c, clear = p, Fraction(1), Fraction(0), True
    off = lambda: max(Fraction(1, 2 ** 40), Fraction(1, 2 ** 44) * c / S if c > 1 else Fraction(0))   # noqa: E731
    for j, x in enumerate(tokens):
        asked = Fraction(accept[j]) * q[x] * S
        if w[x] > 0 or c > 1:
            clear &= abs(asked - w[x]) > off() * max(asked, w[x])
        if w[x] > 0 and asked < w[x]:
            return ([j], None), clear
        c += S
        w = [max(a - c * b, Fraction(0)) for a, b in zip(p, q)]
        S = sum(w)
        if S == 0 or off() > Fraction(1, 8):
            return (None, None), False
    goal, run, at = Fraction(sample) * S, Fraction(0), None
    for k, x in enumerate(w):
        run += x
        clear &= abs(run - goal) > off() * S
        if at is None and run > goal:
            at = k
    return ([], at), clear


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab", [2, 3, 17, 300])
@pytest.mark.parametrize("near", [1.0, 2.0 ** -4, 2.0 ** -10, 2.0 ** -17])
def test_residuals_below_the_last_digit_of_their_row(pool, kind, vocab, near):
    """Refusal after refusal a residual shrinks under the last digit of p and c q, which fp32 differences do not hold."""
    g = torch.Generator().manual_seed(vocab)
    n, t = 200, 6
    logits = 2 * torch.randn(n, vocab, generator=g)
    p = torch.softmax(logits, -1).to(TYPES[kind])
    q = torch.softmax(logits + near * torch.randn(n, vocab, generator=g), -1).to(TYPES[kind])
    target, draft = torch.zeros(n, 1 + t, vocab, dtype=p.dtype), torch.zeros(n, t, vocab, dtype=p.dtype)
    target[:, 0], draft[:, 0] = p, q
    ratio = q.float() / p.float().clamp(min=1e-30)
    tokens = ratio.argmax(-1, keepdim=True).expand(n, t).clone()            # refused
    accept = torch.full((n, t), 1 - 2.0 ** -24)
    for i in range(n):
        if i % (t + 1):   # behind one refusal or more the token that is left longest
            tokens[i, i % (t + 1):] = ratio[i].argmin()
            accept[i, i % (t + 1):] = torch.rand(t - i % (t + 1), generator=g)
    tokens = tokens.int()
    sample = torch.rand(n, generator=g)
    path, size, token = pool.verify_draft(tokens.cuda(), target.cuda(), [-1] * t, accept.cuda(), sample.cuda(), draft=draft.cuda())
    pool.sync()
    checked = 0
    for i in range(n):
        (want, nxt), clear = _outcome(p[i].tolist(), q[i].tolist(), tokens[i].tolist(), accept[i].tolist(), sample[i].item())
        if not clear:
            continue
        checked += 1
        assert path[i].tolist()[:size[i]] == want, i
        assert nxt is None or token[i].item() == nxt, i
    assert checked > 20
