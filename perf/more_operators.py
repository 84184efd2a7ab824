"""Operators for sequences whose cached rows do not stand at their own positions, with their plain forms.

Four kinds of case, each named by ``kind``:

``verify``  drafted tokens (a tree for every branch) verified against the target's probabilities, and the next token
``axes``    rows appended with rotary positions of several axes, given with the rows (Q rotated beside them), read back
``rows``    branches forked onto selected rows (a cache that is thinned out), read back
``cross``   attention of q_len queries to all rows of another sequence (an encoder's states), of another length

Verification.  Node j hangs on node parents[j] (-1: the last accepted token); row 0 of the target's probabilities p
belongs to the last accepted token, row 1 + j to node j; the draft's q has row 0 and rows 1 + j of the nodes before the
last one, which has no children.  From the last accepted token on, the children x of the current node are tried in
order.  With weights w = p, and S = 1, c = 0 at first, child x with the number u is accepted where w(x) > 0 and
u q(x) S < w(x); it is then the current node.  Where it is not, c becomes c + S, w = max(p - c q, 0) and S = sum w, which
is the residual distribution times a number.  Drafts without probabilities are taken as certain: u S < w(x), and a
refused token leaves w.  The next token is the least one at which the running sum of the last node's w passes u' S
(of p, where no w is left).  A token outside the vocabulary is a padding node: skipped.
"""
import math
import random

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one request, 5 drafted tokens in a row, a small vocabulary: latency
        dict(name="verify_chain", kind="verify", type="fp32", branches=1, new=5, vocab=32000, draft=True, tree=False, pad=0),
        # the spec-verify configuration's 32 requests, 24 drafted tokens each as one tree
        dict(name="verify_tree", kind="verify", type="fp32", branches=32, new=24, vocab=128256, draft=True, tree=True, pad=3),
        # a large batch, 7 proposals each from a table of earlier text (no draft probabilities), rows of an odd length
        dict(name="verify_batch", kind="verify", type="bf16", branches=256, new=7, vocab=50257, draft=False, tree=True, pad=1),
        # one decode step of 33 requests behind images: position and row number differ
        dict(name="axes_decode", kind="axes", cache="bf16", branches=33, base=1500, spread=111, new=1, kv=8, heads=32, dim=128, rot=128,
             interleaved=False, scaling="none", axes=3, woven=False),
        # prompts of 4 requests, text and images: one pass over 130 MB of queries
        dict(name="axes_image", kind="axes", cache="bf16", branches=4, base=5, spread=3, new=4099, kv=8, heads=32, dim=128, rot=128,
             interleaved=False, scaling="none", axes=3, woven=False),
        # clips of 16 requests into the 8-bit cache, neighbouring pairs, axes in turn
        dict(name="axes_video", kind="axes", cache="fp8", branches=16, base=70, spread=19, new=777, kv=4, heads=28, dim=128, rot=96,
             interleaved=True, scaling="bands", axes=4, woven=True),
        # one request thinned from 777 rows to its first 4 and 100 others: latency
        dict(name="rows_single", kind="rows", cache="bf16", branches=1, length=777, spread=1, start=4, keep=100, per_head=False, kv=8, dim=128),
        # 16 contexts of 16,384 tokens thinned to 2,048 rows, each head its own
        dict(name="rows_heads", kind="rows", cache="bf16", branches=16, length=16384, spread=901, start=4, keep=2048, per_head=True, kv=8, dim=128),
        # the 8-bit cache of 32 contexts halved, a shared system prompt of 1,000 tokens kept whole
        dict(name="rows_cache8", kind="rows", cache="fp8", branches=32, length=9000, spread=1501, start=1000, keep=4000, per_head=False, kv=8, dim=128),
        # 4 tokens of 9 requests to an 8-bit cache of 1,500 encoder states: latency
        dict(name="cross_decode", kind="cross", cache="fp8", branches=9, length=1500, spread=301, q_len=4, kv=16, heads=16, dim=128),
        # 16 decoder prompts of 448 tokens to 1,500 encoder states
        dict(name="cross_prompt", kind="cross", cache="bf16", branches=16, length=1500, spread=77, q_len=448, kv=16, heads=16, dim=128),
        # 4 prompts of 515 tokens to the states of several image tiles, 4 query heads for a kv head
        dict(name="cross_image", kind="cross", cache="bf16", branches=4, length=6404, spread=1601, q_len=515, kv=8, heads=32, dim=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["verify", "axes", "rows", "cross"])
    if kind == "verify":
        c = dict(kind=kind, type=rng.choice(["fp32", "fp32", "bf16"]), draft=rng.random() < 0.6, tree=rng.random() < 0.6)
        c["new"] = rng.randint(1, 64) if rng.random() < 0.3 else rng.randint(1, 12)
        c["vocab"] = _log(rng, 50, 160000)
        c["branches"] = _log(rng, 1, max(1, min(300, 80_000_000 // (c["vocab"] * c["new"]))))
        c["pad"] = rng.choice([0, 0, 1, 2]) if c["new"] > 4 else 0
        return c
    kv, group = rng.choice([(8, 4), (4, 7), (8, 1), (2, 5), (1, 7), (16, 1)])
    c = dict(kind=kind, kv=kv, dim=128, cache=rng.choice(["bf16", "bf16", "fp8", "fp32"]), spread=rng.randint(1, 19))
    if c["cache"] == "fp32":
        c["dim"] = rng.choice([64, 96, 128, 256])
    if kind == "axes":
        c["heads"] = kv * group
        c["rot"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, 32])
        c["interleaved"] = rng.random() < 0.5
        c["scaling"] = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
        c["axes"] = rng.randint(1, 4)
        c["woven"] = rng.random() < 0.5
        c["new"] = _log(rng, 1, 3000)
        c["branches"] = _log(rng, 1, max(1, min(64, 8000 // c["new"])))
        c["base"] = _log(rng, 20, min(20000, 200000 // c["branches"]))
    elif kind == "rows":
        c["length"] = _log(rng, 64, 20000)
        c["branches"] = _log(rng, 1, max(1, min(64, 80000 // c["length"])))
        c["start"] = rng.choice([0, 4, 16, rng.randint(0, c["length"] // 3)])
        c["keep"] = _log(rng, 7, c["length"] // 2 - 10)
        c["per_head"] = rng.random() < 0.5
    else:
        c["heads"] = kv * group
        c["length"] = _log(rng, 20, 8000)
        c["q_len"] = rng.choice([1, 2, 5, 16]) if rng.random() < 0.4 else _log(rng, 1, 600)
        most = 4e10 / (512 * c["heads"] * c["length"] * c["q_len"])
        c["branches"] = _log(rng, 1, max(1, min(64, int(most), 80000 // c["length"])))
        c["empty"] = rng.random() < 0.3   # the first sequence has no states: its outputs are zero
        if most < 1:
            c["q_len"] = max(1, int(c["q_len"] * most))
    return c


def _bases(case, n, top):
    """Ragged lengths: `top` and down from it by up to spread - 1."""
    return [top - (37 * i) % case["spread"] for i in range(n)]


def _row_bytes(cache, dim):
    return dim + 1 if cache == "fp8" else dim * (4 if cache == "fp32" else 2)


def _thinned(case):
    """Per branch: its length, the first rows that stay, and how many others do."""
    n = case["branches"]
    lens = _bases(case, n, case["length"])
    return lens, [min(case["start"] + i % 3, x) for i, x in enumerate(lens)], [case["keep"] - (5 * i) % 7 for i in range(n)]


def work(case):
    kind, n = case["kind"], case["branches"]
    if kind == "verify":   # the rows of one node: the target's, and the draft's
        rows = 2 if case["draft"] else 1
        return {"bytes": n * case["vocab"] * rows * (4 if case["type"] == "fp32" else 2) + 8 * n * (2 * case["new"] + 2),
                "flops": 3 * n * case["vocab"] * rows}
    cache, kv, d = case["cache"], case["kv"], case["dim"]
    e, row = (4 if cache == "fp32" else 2), _row_bytes(cache, d)
    if kind == "axes":   # rows in, rows kept, rows out; the queries in and out
        new = case["new"]
        return {"bytes": 2 * n * new * kv * (2 * d * e + row) + 2 * n * new * case["heads"] * d * e + 4 * n * new * case["axes"],
                "flops": 3 * n * new * case["rot"] * (case["heads"] + kv)}
    if kind == "rows":   # rows in, rows kept, rows out
        _, starts, counts = _thinned(case)
        kept, total = sum(counts), sum(starts) + sum(counts)
        return {"bytes": 2 * kv * (2 * kept * row + total * d * e) + 4 * kept * (kv if case["per_head"] else 1), "flops": 0}
    states, rows = sum(_states(case)), case["heads"] * case["q_len"]
    return {"bytes": 2 * states * kv * row + 2 * n * rows * d * e, "flops": 4 * d * rows * states}


def _states(case):
    lens = _bases(case, case["branches"], case["length"])
    return [0] + lens[1:] if case.get("empty") else lens


# ---------------------------------------------------------------- the inputs
# How the rotary frequencies are stretched in a case (factor 4 from 8,192 positions).
ROPE_BASE, ROPE_FACTOR, ROPE_LEN = 500000.0, 4.0, 8192


def _frequencies(rot, scaling):
    """Radians per position of each pair, and the factor on the rotated part, in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        return (ROPE_BASE * ROPE_FACTOR ** (rot / (rot - 2))) ** (-2 * i / rot), 1.0
    f = ROPE_BASE ** (-2 * i / rot)
    if scaling == "linear":
        return f / ROPE_FACTOR, 1.0
    if scaling == "bands":   # wavelengths over the trained length are stretched, those under a quarter of it are not
        s = ((ROPE_LEN * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return (1 - s) * f / ROPE_FACTOR + s * f, 1.0
    if scaling == "yarn":
        at = lambda turns: rot * math.log(ROPE_LEN / (turns * 2 * math.pi)) / (2 * math.log(ROPE_BASE))  # noqa: E731
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        s = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return s * f / ROPE_FACTOR + (1 - s) * f, 0.1 * math.log(ROPE_FACTOR) + 1.0
    return f, 1.0


def _axis_of_pairs(case):
    """The axis that each pair turns by: a quarter of the pairs by the first, the others shared out; or in turn."""
    pairs, axes = case["rot"] // 2, case["axes"]
    if case["woven"]:
        return [i % axes for i in range(pairs)]
    first = pairs // 4 if axes > 1 else pairs
    return [0 if i < first else 1 + (i - first) * (axes - 1) // (pairs - first) for i in range(pairs)]


def _positions(case, rng):
    """[n][new][axes]: text (every axis the same) and grids (the first axis stands still) in turn, ragged."""
    out = []
    for base in _bases(case, case["branches"], case["base"]):
        at, seq = base + rng.randint(0, 5000), []
        while len(seq) < case["new"]:
            seq += [[at + i] * case["axes"] for i in range(rng.randint(1, 40))]
            at += 40
            width, height = rng.randint(2, 40), rng.randint(2, 30)
            cells = torch.cartesian_prod(torch.arange(height), torch.arange(width)).tolist()
            seq += [([at, at + y, at + x, at + y + x])[:case["axes"]] for y, x in cells]
            at += max(width, height)
        out.append(seq[:case["new"]])
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _tree(rng, n, tree):
    """Parents of n drafted tokens: a chain, or a few children of the last accepted token, the others below earlier ones."""
    if not tree:
        return list(range(-1, n - 1))
    return [-1 if j == 0 or rng.random() < 0.12 else rng.randint(max(0, j - 9), j - 1) for j in range(n)]


def _quantise(x):
    """Codes and exponents of rows x (last dimension), from their values in 32 bits."""
    x = x.float()
    m, at = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0, at - 9 + (m > 0.875).int(), torch.full_like(at, -127)).clamp(min=-127)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), e.to(torch.int8)


def _values(codes, e):
    return torch.ldexp(codes.float(), e[..., None].int())


def _inputs(case, seed):
    """The tensors of a case, all on the GPU, and the trees and lengths on the host."""
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    rng = random.Random(case["branches"] * 1009 + case.get("new", 0))   # the trees and grids go with the sizes
    n, kind = case["branches"], case["kind"]
    s = dict(case=case)
    if kind == "verify":
        t, new, vocab = TYPES[case["type"]], case["new"], case["vocab"]
        trees = [_tree(rng, new, case["tree"]) for _ in range(n)]
        s["parents"] = torch.tensor(trees, dtype=torch.int32)
        logits = torch.randn(n, 1 + new, vocab, generator=g, device="cuda").mul_(4.0)
        p = torch.softmax(logits, -1)
        p[p < 2e-7] = 0   # a sampler that cuts the tail off
        s["target"] = (p / p.sum(-1, keepdim=True)).to(t)
        q = torch.softmax(logits[:, :new] + torch.randn(n, new, vocab, generator=g, device="cuda"), -1)
        row = (s["parents"] + 1).long().cuda()
        # each node's token is drawn from its parent's row: a race of exponentials
        drawn = [torch.argmax(q.gather(1, row[:, j, None, None].expand(n, 1, vocab))[:, 0]
                              / torch.empty(n, vocab, device="cuda").exponential_(generator=g), -1) for j in range(new)]
        s["tokens"] = torch.stack(drawn, 1).int()
        for i in range(n):
            s["tokens"][i, new - i % (case["pad"] + 1):] = -1   # trees of fewer nodes, padded
        s["draft"] = q.to(t) if case["draft"] else None
        s["accept"] = torch.rand(n, new, generator=g, device="cuda")
        s["sample"] = torch.rand(n, generator=g, device="cuda")
        return s
    d, kv, t = case["dim"], case["kv"], TYPES[case["cache"]]

    def rows(*shape):
        # keys and values of a model differ in size by channel and by token
        x = torch.randn(*shape, generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))
        return x.mul_(torch.exp(0.3 * torch.randn(*shape[:-1], 1, generator=g, device="cuda"))).to(t)

    if kind == "axes":
        s["bases"] = _bases(case, n, case["base"])
        s["k"], s["v"] = (rows(n, case["new"], kv, d) for _ in range(2))
        s["q"] = torch.randn(n, case["new"], case["heads"], d, generator=g, device="cuda").to(t)
        s["positions"] = _positions(case, rng)
        return s
    if kind == "rows":
        s["lens"], s["starts"], s["counts"] = _thinned(case)
        # the rows that a score keeps, in order: of each head its own, or the same for all
        heads, picked = (kv if case["per_head"] else 1), []
        for x, a, c in zip(s["lens"], s["starts"], s["counts"]):
            score = torch.rand(heads, x - a, generator=g, device="cuda")
            picked.append(score.topk(c, sorted=False).indices.sort().values.T + a)
        s["rows"] = torch.cat(picked).int().contiguous()
        if not case["per_head"]:
            s["rows"] = s["rows"][:, 0].contiguous()
    else:
        s["lens"] = _states(case)
        s["q"] = torch.randn(n, case["q_len"], case["heads"], d, generator=g, device="cuda").to(t)
    s["k"], s["v"] = (rows(n, max(s["lens"] + [1]), kv, d) for _ in range(2))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    kind, n = case["kind"], case["branches"]
    if own:
        from copy_write_forked_gb300.dendrite import Pool, Rope

        if kind == "verify":   # the pool that holds the requests: verification reads none of its rows
            s["pool"] = Pool(16, 16, 1, 128, torch.bfloat16, max_branches=4)
            return s
        kv, d, cache = case["kv"], case["dim"], case["cache"]
        lens = s["bases"] if kind == "axes" else s["lens"]
        extra = case["new"] if kind == "axes" else case["start"] + case["keep"] + 18 if kind == "rows" else 0
        pool = Pool(sum((x + extra) // 16 + 3 for x in lens), 16, kv, d, torch.float8_e4m3fn if cache == "fp8" else TYPES[cache],
                    max_branches=2 * n + 1, max_blocks_per_branch=(max(lens) + extra) // 16 + 2)
        s["branches"] = [pool.new_branch() for _ in lens]
        for i, b in enumerate(s["branches"]):
            if kind == "axes":   # what stands before the appended rows is not read in these cases
                z = torch.zeros(1, lens[i], kv, d, dtype=s["k"].dtype, device="cuda")
                pool.append_kv([b], z, z)
            elif lens[i]:
                pool.append_kv([b], s["k"][i:i + 1, :lens[i]].contiguous(), s["v"][i:i + 1, :lens[i]].contiguous())
        if kind == "axes":
            s["rope"] = Rope(case["rot"], base=ROPE_BASE, interleaved=case["interleaved"], scaling=case["scaling"], factor=ROPE_FACTOR,
                             original_len=ROPE_LEN, axes=_axis_of_pairs(case))
        else:
            del s["k"], s["v"]
        pool.sync()
        s["pool"] = pool
        return s
    # the plain form's cache: dense rows, padded to the longest, in the cache's type
    pack = _quantise if case.get("cache") == "fp8" else (lambda x: (x,))
    if kind == "verify":
        s["parents"] = s["parents"].cuda()
    elif kind == "axes":
        f, s["m"] = _frequencies(case["rot"], case["scaling"])
        s["freq"], s["axis"] = f.cuda(), torch.tensor(_axis_of_pairs(case), device="cuda")
    else:
        s["k"], s["v"] = pack(s["k"]), pack(s["v"])
    if kind == "cross":
        s["lens"] = torch.tensor(s["lens"], device="cuda")
    elif kind == "rows":   # of each row that is read back: its branch, its number there, where its list says what it was
        total = [a + c for a, c in zip(s["starts"], s["counts"])]
        s["of"] = torch.repeat_interleave(torch.arange(n), torch.tensor(total)).cuda()
        s["at"] = torch.cat([torch.arange(x) for x in total]).cuda()
        listed_from = torch.tensor([sum(s["counts"][:i]) - a for i, a in enumerate(s["starts"])], device="cuda")
        s["starts"] = torch.tensor(s["starts"], device="cuda")
        s["list"] = (listed_from[s["of"]] + s["at"]).clamp(min=0)
    return s


# ------------------------------------------------------------- the plain forms
def _plain_verify(s):
    p, q, x, up = s["target"], s["draft"], s["tokens"], s["parents"]
    n, new = x.shape
    vocab = p.shape[-1]
    i = torch.arange(n, device=x.device)
    cur, kept = torch.full_like(i, -1), torch.zeros_like(i)
    path = torch.full((n, new), -1, dtype=torch.int64, device=x.device)
    w, S, c = p[:, 0].double(), torch.ones(n, dtype=torch.float64, device=x.device), torch.zeros(n, dtype=torch.float64, device=x.device)
    for j in range(new):
        t = x[:, j].long()
        tried = (up[:, j] == cur) & (t >= 0) & (t < vocab)
        t = t.clamp(0, vocab - 1)
        size = S if q is None else q[i, (cur + 1).clamp(max=new - 1), t].double() * S
        ok = tried & (w[i, t] > 0) & (s["accept"][:, j].double() * size < w[i, t])
        no = tried & ~ok
        # accepted: the node's own row; refused: what the residual leaves
        path[i, kept.clamp(max=new - 1)] = torch.where(ok, j, path[i, kept.clamp(max=new - 1)])
        kept = kept + ok
        c = torch.where(ok, 0.0, torch.where(no, c + S, c))
        if q is None:
            left = torch.where(no[:, None] & (torch.arange(vocab, device=x.device) == t[:, None]), 0.0, w)
        else:
            left = torch.where(no[:, None], (p[i, cur + 1].double() - c[:, None] * q[i, (cur + 1).clamp(max=new - 1)].double()).clamp(min=0), w)
        w = torch.where(ok[:, None], p[:, j + 1].double(), left)
        S = torch.where(ok, 1.0, torch.where(no, w.sum(-1), S))
        cur = torch.where(ok, j, cur)
    w = torch.where((w > 0).any(-1, keepdim=True), w, p[i, cur + 1].double())
    run_sum = w.cumsum(-1)
    nxt = torch.searchsorted(run_sum, (s["sample"].double() * run_sum[:, -1])[:, None], right=True)[:, 0].clamp(max=vocab - 1)
    return path.int(), kept.int(), nxt.int()


def _rotate(x, a, m, rot, interleaved):
    """x [n][T][heads][d] rotated by angles a [n][T][rot / 2] (64 bits), products in 32."""
    c, s = (torch.cos(a) * m).float()[:, :, None], (torch.sin(a) * m).float()[:, :, None]
    y = x.float()
    r = y[..., :rot]
    if interleaved:
        u, v = r[..., 0::2], r[..., 1::2]
        z = torch.stack((u * c - v * s, v * c + u * s), -1).flatten(-2)
    else:
        u, v = r[..., :rot // 2], r[..., rot // 2:]
        z = torch.cat((u * c - v * s, v * c + u * s), -1)
    return torch.cat((z, y[..., rot:]), -1)


def _run_plain(s):
    case = s["case"]
    if case["kind"] == "verify":
        return _plain_verify(s)
    cache, t = case["cache"], TYPES[case["cache"]]
    if case["kind"] == "axes":
        a = s["positions"].double()[..., s["axis"]] * s["freq"]
        q, k = (_rotate(s[name], a, s["m"], case["rot"], case["interleaved"]) for name in ("q", "k"))
        v = s["v"].float()
        if cache == "fp8":
            k, v = _values(*_quantise(k)), _values(*_quantise(v))
        return q.to(t), k.to(t), v.to(t)
    if case["kind"] == "rows":
        of, at = s["of"], s["at"]
        rows = (s["rows"] if case["per_head"] else s["rows"][:, None].expand(-1, case["kv"])).long()
        rows = torch.where((at < s["starts"][of])[:, None], at[:, None], rows[s["list"].clamp(max=len(rows) - 1)])
        h = torch.arange(case["kv"], device=of.device)
        out = [tuple(y[of[:, None], rows, h] for y in s[name]) for name in ("k", "v")]
        return tuple((_values(*y) if cache == "fp8" else y[0]).to(t) for y in out)
    n, kv, d = case["branches"], case["kv"], case["dim"]
    k, v = (_values(*s[name]) if cache == "fp8" else s[name][0].float() for name in ("k", "v"))
    q = s["q"].float().view(n, case["q_len"], kv, -1, d) * d ** -0.5
    x = torch.einsum("nthgd,nlhd->nhtgl", q, k)
    x.masked_fill_((torch.arange(k.shape[1], device=k.device) >= s["lens"][:, None])[:, None, None, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    x = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
    return torch.einsum("nhtgl,nlhd->nthgd", x, v).reshape(s["q"].shape).to(t)


# ------------------------------------------------------------ the framework's
def _run_own(s):
    case, pool = s["case"], s["pool"]
    kind = case["kind"]
    if kind == "verify":
        return pool.verify_draft(s["tokens"], s["target"], s["parents"], s["accept"], s["sample"], draft=s["draft"])
    br = s["branches"]
    if kind == "axes":
        q = pool.append_rope(br, s["k"], s["v"], s["rope"], Q=s["q"], positions=s["positions"])
        k, v = pool.read_kv(br, s["bases"], [case["new"]] * len(br))
        pool.truncate(br, s["bases"])
        return q, k.view_as(s["k"]), v.view_as(s["v"])
    if kind == "rows":
        kids = pool.fork_rows(br, s["starts"], s["counts"], s["rows"])
        k, v = pool.read_kv(kids, [0] * len(kids), [a + c for a, c in zip(s["starts"], s["counts"])])
        pool.free(kids)
        return k, v
    return pool.tree_attn_cross(s["q"], br)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------- the definition, in 64 bits
def _exact_cached(x, cache):
    """What the cache stands for after rows x are written."""
    x = x.double()
    if cache == "fp32":
        return x.float().double()
    if cache == "bf16":
        return x.to(torch.bfloat16).double()
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).clamp(min=-127)
    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e).clamp(min=-127)   # a logarithm rounded up to an integer
    y = x * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)   # three bits behind the point; 2^-9 at the least
    return torch.round(y / step) * step * torch.exp2(e)


def _exact_rotated(x, positions, case):
    rot, half, axis = case["rot"], case["rot"] // 2, _axis_of_pairs(case)
    freq, m = _frequencies(rot, case["scaling"])
    y = x.double().clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        w = (positions[..., axis[i]].double() * freq[i].item())[..., None]
        u, v = x[..., a].double(), x[..., b].double()
        y[..., a] = m * (u * torch.cos(w) - v * torch.sin(w))
        y[..., b] = m * (u * torch.sin(w) + v * torch.cos(w))
    return y


def _exact_verified(p, q, tokens, parents, accept, sample):
    """One branch: the accepted path and the next token, with each residual a distribution of its own."""
    path, cur, vocab = [], -1, p.shape[-1]
    r = p[0].double()
    for j, x in enumerate(tokens):
        if parents[j] != cur or not 0 <= x < vocab:
            continue
        have, asked = r[x].item(), accept[j]
        if q is not None:
            asked *= q[cur + 1, x].item()
        if have > 0 and asked < have:
            cur = j
            path.append(j)
            r = p[1 + j].double()
            continue
        if q is None:
            r[x] = 0
        else:
            r = torch.relu(r - q[cur + 1].double())
        if r.sum() > 0:
            r = r / r.sum()
    if not r.sum() > 0:
        r = p[cur + 1].double()
    passed = torch.cumsum(r, 0) > sample * r.sum()
    return path, int(torch.nonzero(passed)[0])


def exact(case, seed):
    if case["kind"] == "cross" and work(case)["flops"] > 4e12:
        return None
    s = _inputs(case, seed)
    kind, n = case["kind"], case["branches"]
    if kind == "verify":
        new = case["new"]
        path, kept, nxt = torch.full((n, new), -1, dtype=torch.int32), [], []
        tokens, parents, accept, sample = (s[x].tolist() for x in ("tokens", "parents", "accept", "sample"))
        for i in range(n):
            got, x = _exact_verified(s["target"][i], None if s["draft"] is None else s["draft"][i], tokens[i], parents[i], accept[i], sample[i])
            path[i, :len(got)] = torch.tensor(got, dtype=torch.int32)
            kept.append(len(got))
            nxt.append(x)
        return path, torch.tensor(kept, dtype=torch.int32), torch.tensor(nxt, dtype=torch.int32)
    cache = case["cache"]
    if kind == "axes":
        q, k = (_exact_rotated(s[x], s["positions"], case) for x in ("q", "k"))
        return q, _exact_cached(k, cache), _exact_cached(s["v"], cache)
    if kind == "rows":
        out, at = ([], []), 0
        for i, (a, c) in enumerate(zip(s["starts"], s["counts"])):
            rows = s["rows"][at:at + c].long()
            at += c
            for x, to in zip((s["k"], s["v"]), out):
                to.append(x[i, :a])
                to.append(x[i, rows] if rows.dim() == 1 else torch.stack([x[i, rows[:, h], h] for h in range(case["kv"])], 1))
        return tuple(_exact_cached(torch.cat(x), cache) for x in out)
    group, outs = case["heads"] // case["kv"], []
    for i, length in enumerate(s["lens"]):
        k, v = (_exact_cached(s[x][i, :length], cache) for x in ("k", "v"))
        o = torch.zeros(s["q"].shape[1:], dtype=torch.float64, device="cuda")
        for h in range(case["heads"] if length else 0):
            z = s["q"][i, :, h].double() @ k[:, h // group].T / math.sqrt(case["dim"])
            o[:, h] = torch.softmax(z, -1) @ v[:, h // group]
        outs.append(o)
    return torch.stack(outs)
