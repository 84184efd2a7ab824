"""Operators of a speculative decoding step on the tree cache, with their plain forms.

Five kinds of case, each named by ``kind``:

``rope``   rows appended with rotary positions (Q rotated beside them), read back, rolled back
``cache``  rows quantised into an 8-bit cache as they are appended, read back, rolled back
``attn8``  tree decode attention over an 8-bit cache
``draft``  attention of a tree of drafted tokens over a cache of any type
``step``   a whole step: rotary append of the drafted tokens, their attention, acceptance of one path, its rows
           read back, roll-back

Every cached row is a (token, kv head) vector.  An 8-bit cache holds it as e4m3 codes with one power-of-two scale:
e is the least integer with max|x| <= 448 * 2^e and the code is x * 2^-e rounded to nearest even.
"""
import math
import random

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of 16 branches 4,096 tokens in: the smallest append, where latency counts
        dict(name="rope_decode", kind="rope", cache="bf16", branches=16, base=4096, spread=200, new=1, kv=8, heads=32, dim=128,
             rot=128, interleaved=False, scaling="none", draft=False),
        # prompts of 4 requests: one pass over 130 MB of queries; half of each head rotated, stretched for long contexts
        dict(name="rope_prefill", kind="rope", cache="bf16", branches=4, base=5, spread=3, new=4099, kv=8, heads=32, dim=128,
             rot=64, interleaved=True, scaling="yarn", draft=False),
        # a decode step of 33 beams into the 8-bit cache
        dict(name="cache_decode", kind="cache", branches=33, base=1000, spread=61, new=1, kv=8, dim=128),
        # 8 prompts of the beam configuration's 4,096 tokens, begun inside a block
        dict(name="cache_prefill", kind="cache", branches=8, base=7, spread=5, new=4096, kv=8, dim=128),
        # one request's token, 777 tokens in: latency
        dict(name="attn8_single", kind="attn8", requests=1, prefix=777, spread=1, width=1, leaf=1, q_len=1, kv=8, heads=32, dim=128),
        # the beam configuration: 8 prompts of 4,096 tokens, forked 4 ways, 256 tokens of their own each
        dict(name="attn8_beam", kind="attn8", requests=8, prefix=4096, spread=1, width=4, leaf=256, q_len=1, kv=8, heads=32, dim=128),
        # 8 long contexts of the stress configuration's 32,768 tokens, ragged, one token each
        dict(name="attn8_long", kind="attn8", requests=8, prefix=32768, spread=700, width=1, leaf=3, q_len=1, kv=8, heads=32, dim=128),
        # one request, 8 drafted tokens behind 500: latency
        dict(name="draft_small", kind="draft", cache="bf16", branches=1, base=500, spread=1, new=8, kv=8, heads=32, dim=128),
        # the spec-verify configuration's 32 requests of 8,192 tokens, 24 drafted tokens each as one tree
        dict(name="draft_verify", kind="draft", cache="bf16", branches=32, base=8192, spread=301, new=24, kv=8, heads=32, dim=128),
        # wide trees (61 nodes) over ragged 8-bit contexts, 8 query heads for a kv head
        dict(name="draft_wide", kind="draft", cache="fp8", branches=12, base=4000, spread=3001, new=61, kv=4, heads=32, dim=128),
        # a whole step of a small batch
        dict(name="step_small", kind="step", cache="bf16", branches=4, base=1024, spread=129, new=9, kv=8, heads=32, dim=128,
             rot=128, interleaved=False, scaling="linear"),
        # a whole step of a large batch on the 8-bit cache
        dict(name="step_large", kind="step", cache="fp8", branches=32, base=6000, spread=2500, new=16, kv=8, heads=32, dim=128,
             rot=128, interleaved=False, scaling="bands"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "cache", "attn8", "draft", "step"])
    kv, group = rng.choice([(8, 4), (4, 8), (8, 1), (2, 5), (1, 7), (8, 4)])
    c = dict(kind=kind, kv=kv, dim=128)
    if kind == "rope":
        c["cache"] = rng.choice(["bf16", "bf16", "fp32", "fp8"])
        c["dim"] = rng.choice([64, 96, 128, 256]) if c["cache"] == "fp32" else 128
        c["heads"] = kv * group
        c["rot"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, 32])
        c["interleaved"] = rng.random() < 0.5
        c["scaling"] = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
        c["draft"] = rng.random() < 0.3
        c["new"] = rng.randint(2, 64) if c["draft"] else _log(rng, 1, 3000)
        c["branches"] = _log(rng, 1, max(1, min(64, 8000 // c["new"])))
        c["base"] = _log(rng, 20, min(20000, 200000 // c["branches"]))
        c["spread"] = rng.randint(1, 19)
    elif kind == "cache":
        c["new"] = _log(rng, 1, 4000)
        c["branches"] = _log(rng, 1, max(1, min(100, 30000 // c["new"])))
        c["base"] = _log(rng, 20, 4000)
        c["spread"] = rng.randint(1, 19)
    elif kind == "attn8":
        c["heads"] = kv * group
        c["requests"] = _log(rng, 1, 12)
        c["width"] = rng.choice([1, 1, 2, 3, 4, 7])
        c["q_len"] = rng.choice([1, 1, 1, 2, 5])
        c["prefix"] = _log(rng, 20, 150000 // (c["requests"] * max(1, c["width"] * c["q_len"] // 4)))
        c["spread"] = rng.randint(1, 19)
        c["leaf"] = _log(rng, 5, 300)
    else:
        c["heads"] = kv * group
        c["cache"] = rng.choice(["bf16", "fp8"])
        c["new"] = rng.randint(1, 64)
        c["branches"] = _log(rng, 1, 20)
        c["base"] = _log(rng, 20, 60000 // c["branches"])
        c["spread"] = rng.randint(1, 19)
        if kind == "step":
            c["rot"] = rng.choice([128, 128, 64])
            c["interleaved"] = rng.random() < 0.5
            c["scaling"] = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
    return c


def _bases(case, n, top):
    """Ragged lengths: `top` and down from it by up to spread - 1."""
    return [top - (37 * i) % case["spread"] for i in range(n)]


def _row_bytes(cache, dim):
    return dim + 1 if cache == "fp8" else dim * (4 if cache == "fp32" else 2)


def work(case):
    kv, d, kind = case["kv"], case["dim"], case["kind"]
    if kind == "attn8":
        n = case["requests"] * case["width"]
        lens = _bases(case, case["requests"], case["prefix"])
        rows = case["heads"] * case["q_len"]
        tokens = sum(lens) + n * case["leaf"]
        seen = case["width"] * sum(lens) + n * case["leaf"]
        return {"bytes": 2 * tokens * kv * (d + 1) + 2 * n * rows * d * 2, "flops": 4 * d * rows * seen}
    n, new, cache = case["branches"], case["new"], case.get("cache", "fp8")
    e, row = (4 if cache == "fp32" else 2), _row_bytes(cache, d)
    rows_in, rows_kept = 2 * n * new * kv * d * e, 2 * n * new * kv * row
    if kind in ("rope", "cache"):   # rows in, rows kept, rows out; the queries in and out
        return {"bytes": 2 * rows_in + rows_kept + 2 * n * new * case.get("heads", 0) * d * e,
                "flops": 3 * n * new * case.get("rot", 0) * (case.get("heads", 0) + kv) + 2 * n * new * kv * d}
    bases = _bases(case, n, case["base"])
    att = {"bytes": 2 * kv * row * (sum(bases) + n * new) + 2 * n * new * case["heads"] * d * 2,
           "flops": 4 * d * case["heads"] * new * (sum(bases) + n * (new + 1) // 2)}
    if kind == "step":
        att["bytes"] += rows_in + rows_kept + 2 * n * new * case["heads"] * d * 2
    return att


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


def _tree(rng, n):
    """Parents of n drafted tokens: a few children of the last accepted token, the others below earlier ones."""
    return [-1 if j == 0 or rng.random() < 0.12 else rng.randint(max(0, j - 9), j - 1) for j in range(n)]


def _path(rng, parents):
    """An accepted path: a node and its ancestors, cut at a random length (one node at least)."""
    j, up = rng.randrange(len(parents)), []
    while j >= 0:
        up.append(j)
        j = parents[j]
    up.reverse()
    return up[:rng.randint(1, len(up))]


def _quantise(x):
    """Codes and exponents of rows x (last dimension), from their values in 32 bits."""
    x = x.float()
    m, at = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0, at - 9 + (m > 0.875).int(), torch.full_like(at, -127)).clamp(min=-127)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), e.to(torch.int8)


def _values(codes, e):
    return torch.ldexp(codes.float(), e[..., None].int())


def _inputs(case, seed):
    """The tensors of a case, all on the GPU, and the trees and paths on the host."""
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    rng = random.Random(case.get("new", 0) * 1009 + case.get("branches", 0))   # the trees and accepted paths go with the sizes
    d, kv, kind = case["dim"], case["kv"], case["kind"]
    t = TYPES[case.get("cache", "fp8")]

    def rows(*shape):
        # keys and values of a model differ in size by channel and by token
        x = torch.randn(*shape, generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))
        return x.mul_(torch.exp(0.3 * torch.randn(*shape[:-1], 1, generator=g, device="cuda"))).to(t)

    s = dict(case=case)
    if kind == "attn8":
        r, w = case["requests"], case["width"]
        s["lens"] = _bases(case, r, case["prefix"])
        s["k"], s["v"] = (rows(r, max(s["lens"]), kv, d) for _ in range(2))
        s["leaf_k"], s["leaf_v"] = (rows(r * w, case["leaf"], kv, d) for _ in range(2))
        s["q"] = torch.randn(r * w, case["q_len"], case["heads"], d, generator=g, device="cuda").to(t)
        return s
    n, new = case["branches"], case["new"]
    s["bases"] = _bases(case, n, case["base"])
    s["k"], s["v"] = (rows(n, new, kv, d) for _ in range(2))
    if kind != "cache":
        s["q"] = torch.randn(n, new, case["heads"], d, generator=g, device="cuda").to(t)
    if kind in ("draft", "step"):
        s["past_k"], s["past_v"] = (rows(n, max(s["bases"]), kv, d) for _ in range(2))
    if kind in ("draft", "step") or case.get("draft"):
        trees = [_tree(rng, new) for _ in range(n)]
        s["parents"] = torch.tensor(trees, dtype=torch.int32)
        s["keep"] = [_path(rng, p) for p in trees]
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    kind, cache = case["kind"], case.get("cache", "fp8")
    if own:
        from copy_write_forked_gb300.dendrite import Pool, Rope

        kv, d, dtype = case["kv"], case["dim"], torch.float8_e4m3fn if cache == "fp8" else TYPES[cache]
        if kind == "attn8":
            lens, w, extra = s["lens"], case["width"], case["leaf"]
        else:
            lens, w, extra = s["bases"], 1, case["new"]
        longest = max(lens) + extra
        pool = Pool(sum(n // 16 + 2 + w * (extra // 16 + 3) for n in lens), 16, kv, d, dtype, max_branches=len(lens) * (w + 1) + 1,
                    max_blocks_per_branch=longest // 16 + 2)
        roots = [pool.new_branch() for _ in lens]
        past_k, past_v = (s["k"], s["v"]) if kind == "attn8" else (s.get("past_k"), s.get("past_v"))
        for i, b in enumerate(roots):
            if past_k is None:   # what stands before the appended rows is not read in these cases
                z = torch.zeros(1, lens[i], kv, d, dtype=s["k"].dtype, device="cuda")
                pool.append_kv([b], z, z)
            else:
                pool.append_kv([b], past_k[i:i + 1, :lens[i]].contiguous(), past_v[i:i + 1, :lens[i]].contiguous())
        s["branches"] = roots
        if kind == "attn8":
            s["branches"] = [c for ch in pool.fork_batch(roots, [w] * len(roots)) for c in ch]
            pool.append_kv(s["branches"], s["leaf_k"], s["leaf_v"])
        elif kind == "draft":
            pool.append_kv(roots, s["k"], s["v"])
        if "rot" in case:
            s["rope"] = Rope(case["rot"], base=ROPE_BASE, interleaved=case["interleaved"], scaling=case["scaling"], factor=ROPE_FACTOR,
                             original_len=ROPE_LEN)
        s["counts"] = [len(p) for p in s["keep"]] if kind == "step" else [case.get("new", 0)] * len(roots)
        pool.sync()
        s["pool"] = pool
        for name in ("past_k", "past_v", "leaf_k", "leaf_v") + (("k", "v") if kind in ("attn8", "draft") else ()):
            s.pop(name, None)
        return s
    # the plain form's cache: dense rows, padded to the longest, in the cache's type
    pack = _quantise if cache == "fp8" else (lambda x: (x,))
    if kind == "attn8":
        s["lens"] = torch.tensor(s["lens"], device="cuda")
        for name in ("k", "v", "leaf_k", "leaf_v"):
            s[name] = pack(s[name])
        return s
    s["bases"] = torch.tensor(s["bases"], device="cuda")
    if "parents" in s:
        s["parents"] = s["parents"].cuda()
    if kind in ("draft", "step"):
        for name in ("past_k", "past_v"):
            s[name] = pack(s[name])
    if kind == "draft":
        s["k"], s["v"] = pack(s["k"]), pack(s["v"])
    if "rot" in case:
        f, m = _frequencies(case["rot"], case["scaling"])
        s["freq"], s["m"] = f.cuda(), m
    if kind == "step":
        flat = [(i, j) for i, p in enumerate(s["keep"]) for j in p]
        s["kept"] = torch.tensor(flat, device="cuda").T.contiguous()
    return s


# ------------------------------------------------------------- the plain forms
def _unpack(x):
    return _values(*x) if len(x) == 2 else x[0].float()


def _ancestors(parents):
    """[n][T][T]: node j sees node i (its ancestors and itself); zeros but one for every step down of a path."""
    n = parents.shape[1]
    up = (parents[..., None] == torch.arange(n, device=parents.device)).float()
    return torch.matrix_power(torch.eye(n, device=parents.device) + up, n) > 0


def _rotate(x, positions, freq, m, rot, interleaved):
    """x [n][T][heads][d] rotated by its positions [n][T]: angles in 64 bits, products in 32."""
    a = positions.double()[..., None] * freq
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


def _softmax(s):
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _draft_attention(q, past_k, past_v, k, v, bases, anc):
    """q [n][T][heads][d] over the first bases[i] rows of the past and the drafted rows that anc lets it see."""
    n, t, heads, d = q.shape
    kv = k.shape[2]
    q = q.float().view(n, t, kv, heads // kv, d) * d ** -0.5
    s = torch.einsum("nthgd,nlhd->nhtgl", q, past_k)
    beyond = torch.arange(s.shape[-1], device=q.device) >= bases[:, None]
    s.masked_fill_(beyond[:, None, None, None], -math.inf)
    own_part = torch.einsum("nthgd,nlhd->nhtgl", q, k)
    own_part.masked_fill_(~anc[:, None, :, None], -math.inf)
    p = _softmax(torch.cat((s, own_part), -1))
    out = torch.einsum("nhtgl,nlhd->nthgd", p[..., :s.shape[-1]], past_v) + torch.einsum("nhtgl,nlhd->nthgd", p[..., s.shape[-1]:], v)
    return out.reshape(n, t, heads, d)


def _run_plain(s):
    case = s["case"]
    kind, cache = case["kind"], case.get("cache", "fp8")
    t = TYPES[cache]
    if kind == "cache":
        return tuple(_values(*_quantise(x)).to(t) for x in (s["k"], s["v"]))
    if kind == "attn8":
        r, w, kv, d = case["requests"], case["width"], case["kv"], case["dim"]
        k, v, lk, lv = (_unpack(s[name]) for name in ("k", "v", "leaf_k", "leaf_v"))
        lk, lv = (x.view(r, w, case["leaf"], kv, d) for x in (lk, lv))
        q = s["q"].float().view(r, w, case["q_len"], kv, -1, d) * d ** -0.5
        a = torch.einsum("rwqhgd,rlhd->rhwqgl", q, k)
        a.masked_fill_((torch.arange(k.shape[1], device=k.device) >= s["lens"][:, None])[:, None, None, None, None], -math.inf)
        b = torch.einsum("rwqhgd,rwlhd->rhwqgl", q, lk)
        last = torch.arange(case["leaf"] - case["q_len"], case["leaf"], device=k.device)
        b.masked_fill_((torch.arange(case["leaf"], device=k.device) > last[:, None])[:, None], -math.inf)
        p = _softmax(torch.cat((a, b), -1))
        out = torch.einsum("rhwqgl,rlhd->rwqhgd", p[..., :k.shape[1]], v) + torch.einsum("rhwqgl,rwlhd->rwqhgd", p[..., k.shape[1]:], lv)
        return out.reshape(s["q"].shape).to(t)
    if kind == "draft":
        k, v, pk, pv = (_unpack(s[name]) for name in ("k", "v", "past_k", "past_v"))
        return _draft_attention(s["q"], pk, pv, k, v, s["bases"], _ancestors(s["parents"])).to(t)
    new = case["new"]
    if "parents" in s:
        anc = _ancestors(s["parents"])
        positions = s["bases"][:, None] + anc.sum(-1) - 1
    else:
        positions = s["bases"][:, None] + torch.arange(new, device="cuda")
    q, k = (_rotate(s[name], positions, s["freq"], s["m"], case["rot"], case["interleaved"]) for name in ("q", "k"))
    if cache == "fp8":
        k, v = _values(*_quantise(k)), _values(*_quantise(s["v"]))
    else:
        k, v = k.to(t).float(), s["v"].float()
    if kind == "rope":
        return q.to(t), k.to(t), v.to(t)
    out = _draft_attention(q.to(t), _unpack(s["past_k"]), _unpack(s["past_v"]), k, v, s["bases"], anc)
    i, j = s["kept"]
    return out.to(t), k[i, j].to(t), v[i, j].to(t)


# ------------------------------------------------------------ the framework's
def _run_own(s):
    case, pool, br = s["case"], s["pool"], s["branches"]
    kind = case["kind"]
    if kind == "attn8":
        return pool.tree_attn_decode(s["q"], br)
    if kind == "draft":
        return pool.tree_attn_draft(s["q"], br, s["parents"])
    if kind == "step":
        q = pool.append_rope(br, s["k"], s["v"], s["rope"], Q=s["q"], parents=s["parents"])
        out = pool.tree_attn_draft(q, br, s["parents"])
        pool.accept_draft(br, case["new"], s["keep"])
        k, v = pool.read_kv(br, s["bases"], s["counts"])
        pool.truncate(br, s["bases"])
        return out, k, v
    if kind == "rope":
        q = pool.append_rope(br, s["k"], s["v"], s["rope"], Q=s["q"], parents=s.get("parents"))
        k, v = pool.read_kv(br, s["bases"], s["counts"])
        pool.truncate(br, s["bases"])
        return q, k.view_as(s["k"]), v.view_as(s["v"])
    pool.append_kv(br, s["k"], s["v"])
    k, v = pool.read_kv(br, s["bases"], s["counts"])
    pool.truncate(br, s["bases"])
    return k.view_as(s["k"]), v.view_as(s["v"])


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
    rot, half = case["rot"], case["rot"] // 2
    y = x.double().clone()
    for i in range(half):
        f = ROPE_BASE ** (-2.0 * i / rot)
        m = 1.0
        if case["scaling"] == "linear":
            f /= ROPE_FACTOR
        elif case["scaling"] == "ntk":
            f = (ROPE_BASE * ROPE_FACTOR ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
        elif case["scaling"] == "bands":
            turns = ROPE_LEN * f / (2 * math.pi)
            s = min(max((turns - 1.0) / 3.0, 0.0), 1.0)
            f = (1 - s) * f / ROPE_FACTOR + s * f
        elif case["scaling"] == "yarn":
            pair = [rot * math.log(ROPE_LEN / (b * 2 * math.pi)) / (2 * math.log(ROPE_BASE)) for b in (32.0, 1.0)]
            lo, hi = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), rot - 1)
            s = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f * (1 - s) + f / ROPE_FACTOR * s
            m = 1.0 + 0.1 * math.log(ROPE_FACTOR)
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        w = (positions.double() * f)[..., None]
        u, v = x[..., a].double(), x[..., b].double()
        y[..., a] = m * (u * torch.cos(w) - v * torch.sin(w))
        y[..., b] = m * (u * torch.sin(w) + v * torch.cos(w))
    return y


def _exact_attention(q, k, v, seen):
    """q [T][heads][d] over k, v [L][kv][d] where seen [T][L]; one head after the other."""
    t, heads, d = q.shape
    group = heads // k.shape[1]
    out = torch.empty(t, heads, d, dtype=torch.float64, device=q.device)
    for h in range(heads):
        s = (q[:, h].double() @ k[:, h // group].double().T) / math.sqrt(d)
        out[:, h] = torch.softmax(s.masked_fill(~seen, -math.inf), -1) @ v[:, h // group].double()
    return out


def _exact_seen(parents, base):
    n = len(parents)
    seen = torch.zeros(n, base + n, dtype=torch.bool)
    for j in range(n):
        seen[j, :base] = True
        i = j
        while i >= 0:
            seen[j, base + i] = True
            i = parents[i]
    return seen.cuda()


def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    s = _inputs(case, seed)
    kind, cache, new = case["kind"], case.get("cache", "fp8"), case.get("new", 0)
    if kind == "cache":
        return tuple(_exact_cached(s[x], "fp8") for x in ("k", "v"))
    if kind == "attn8":
        out, w, q_len = [], case["width"], case["q_len"]
        for i, length in enumerate(s["lens"]):
            k, v = (_exact_cached(s[x][i, :length], "fp8") for x in ("k", "v"))
            for b in range(i * w, (i + 1) * w):
                kk, vv = torch.cat((k, _exact_cached(s["leaf_k"][b], "fp8"))), torch.cat((v, _exact_cached(s["leaf_v"][b], "fp8")))
                at = torch.arange(len(kk), device="cuda")
                out.append(_exact_attention(s["q"][b], kk, vv, at <= len(kk) - q_len + at[:q_len, None]))
        return torch.stack(out)
    n, q, k, positions = case["branches"], s["q"], s["k"], None
    trees = s["parents"].tolist() if "parents" in s else None
    if "rot" in case:
        depth = [[] for _ in range(n)]
        for i in range(n):
            for j in range(new):
                depth[i].append(j if trees is None else 0 if trees[i][j] < 0 else depth[i][trees[i][j]] + 1)
        positions = torch.tensor([[s["bases"][i] + x for x in depth[i]] for i in range(n)], device="cuda")
        q, k = _exact_rotated(q, positions, case), _exact_rotated(k, positions, case)
    k, v = _exact_cached(k, cache), _exact_cached(s["v"], cache)
    if kind == "rope":
        return q, k, v
    out = []
    for i in range(n):
        base = s["bases"][i]
        kk = torch.cat((_exact_cached(s["past_k"][i, :base], cache), k[i]))
        vv = torch.cat((_exact_cached(s["past_v"][i, :base], cache), v[i]))
        out.append(_exact_attention(q[i], kk, vv, _exact_seen(trees[i], base)))
    if kind == "draft":
        return torch.stack(out)
    return (torch.stack(out), torch.cat([k[i][p] for i, p in enumerate(s["keep"])]), torch.cat([v[i][p] for i, p in enumerate(s["keep"])]))
