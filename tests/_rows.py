"""64-bit references for the row operators: 8-bit rows, rotary positions, draft
trees, and attention with the error its roundings can make."""
from __future__ import annotations

import math
import random

import numpy as np
import torch


# ------------------------------------------------------------------ 8-bit rows
def e4m3_values():
    """The 256 values of a code."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = -v if c & 128 else v
    out[[127, 255]] = np.nan
    return out


E4M3 = e4m3_values()


def quantise(x):
    """x [..., 128] -> (codes uint8, exponents int): nearest code, ties to even, of x * 2^-e; a row
    that is not finite is NaN throughout, with exponent 128."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x).all(-1)
    x = np.where(fine[..., None], x, 0)
    top = np.abs(x).max(-1)
    e = np.full(top.shape, -126)
    for k in range(-125, 121):     # the least e with top <= 448 * 2^e
        e = np.where(top > 448 * 2.0 ** (k - 1), k, e)
    y = np.abs(x) * 2.0 ** -e[..., None].astype(float)
    y = np.where(e[..., None] == 120, np.minimum(y, 240.0), y)   # 256 * 2^120 is past bf16
    pos = E4M3[:127]
    hi = np.clip(np.searchsorted(pos, y), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    up = (pos[hi] - y < y - pos[lo]) | ((pos[hi] - y == y - pos[lo]) & (hi % 2 == 0))
    code = np.where(up | (pos[hi] == y), hi, lo).astype(np.uint8)
    code |= np.signbit(x).astype(np.uint8) << 7
    return np.where(fine[..., None], code, 0x7f).astype(np.uint8), np.where(fine, e, 128)


def dequantise(codes, e):
    return E4M3[codes] * 2.0 ** np.asarray(e, float)[..., None]


def untile(raw):
    """A block's raw tiles [n_kv][2064] -> (codes [n_kv][16][128], exponents [n_kv][16])."""
    raw = np.asarray(raw)
    codes = raw[:, :2048].reshape(-1, 16, 8, 16)
    out = np.empty_like(codes)
    for s in range(16):
        for c in range(8):
            out[:, s, c] = codes[:, s, c ^ (s & 7)]
    return out.reshape(-1, 16, 128), raw[:, 2048:].astype(int) - 127


def same_codes(a, b):
    """Equal codes, any NaN code equal to any other."""
    nan = (a & 0x7f) == 0x7f
    return np.array_equal(nan, (b & 0x7f) == 0x7f) and np.array_equal(a[~nan], b[~nan])


# --------------------------------------------------------------------- rotary
def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=None):
    """(radians per position of each pair, factor on the turned part)."""
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "yarn":
        high = 32.0 if high is None else high
        pair = lambda turns: rot * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
        out = []
        for i, x in enumerate(f):
            r = min(max((i - a) / max(b - a, 0.001), 0), 1)
            out.append(x / factor * r + x * (1 - r))
        return out, 0.1 * math.log(factor) + 1
    if scaling == "bands":
        high = 4.0 if high is None else high
        out = []
        for x in f:
            turns = original_len * x / (2 * math.pi)
            if turns < low:
                out.append(x / factor)
            elif turns > high:
                out.append(x)
            else:
                s = (turns - low) / (high - low)
                out.append((1 - s) * x / factor + s * x)
        return out, 1.0
    return f, 1.0


def rotate(x, pos, freq, rot, interleaved, m=1.0):
    """x [tokens][heads][d] (float64) turned by pos [tokens]; and max(|x1|, |x2|) sums for bounds."""
    y, size = x.copy(), np.zeros_like(x)
    a = np.asarray(pos, float)[:, None] * np.asarray(freq)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    i = np.arange(rot // 2)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    u, v = x[..., p], x[..., q]
    y[..., p], y[..., q] = m * (u * c - v * s), m * (v * c + u * s)
    size[..., p] = size[..., q] = abs(m) * (np.abs(u) + np.abs(v))
    return y, size


# A turned element's error in fp32, relative to m (|x1| + |x2|).  The angle, as a
# float of half a turn: half a step of 2^-24 at most near 1, so pi 2^-25 < 2^-23.3
# radians; sincospif: one step, 2^-23; the factor m, its product, the two
# products and the sum: half a step each, 5 * 2^-24.  Together below 2^-21.
ROPE_ERR = 2.0 ** -21


# ----------------------------------------------------------------- draft trees
def tree(rng: random.Random, n: int, kind: str = "random"):
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] * n
    return [-1 if j == 0 or rng.random() < 0.15 else rng.randint(max(0, j - 8), j - 1) for j in range(n)]


def depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def path_to(parents, j):
    up = []
    while j >= 0:
        up.append(j)
        j = parents[j]
    return up[::-1]


def seen(parents, base):
    """[n][base + n] bool: what each drafted token sees."""
    n = len(parents)
    out = np.zeros((n, base + n), bool)
    for j in range(n):
        out[j, :base] = True
        out[j, [base + i for i in path_to(parents, j)]] = True
    return out


# ------------------------------------------------------------------- attention
def attention(q, k, v, see):
    """q [T][heads][d] over k, v [L][kv][d] where see [T][L], in 64 bits.  Returns the
    output, sum p |v - out|, sum p |v|, the largest sum |q_i k_i| / sqrt(d) of a row,
    and L times the largest p max|v|."""
    t, heads, d = q.shape
    group = heads // k.shape[1]
    out, dev, mag, size = np.empty_like(q), np.empty_like(q), np.empty_like(q), np.empty((t, heads, 1))
    top = np.empty((t, heads, 1))
    for h in range(heads):
        kk, vv = k[:, h // group], v[:, h // group]
        s = q[:, h] @ kk.T / math.sqrt(d)
        s = np.where(see, s, -np.inf)
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        out[:, h] = p @ vv
        mag[:, h] = p @ np.abs(vv)
        dev[:, h] = np.stack([p[i] @ np.abs(vv - out[i, h]) for i in range(t)])
        size[:, h, 0] = np.where(see, np.abs(q[:, h]) @ np.abs(kk).T, 0).max(-1) / math.sqrt(d)
        top[:, h, 0] = len(kk) * (p * np.abs(vv).max(-1)).max(-1)
    return out, dev, mag, size, top


def attention_bound(kind, out, dev, mag, size, top):
    """How far an output of a pool of this kind may be from attention()'s.

    Scores: 128 products summed in fp32, every addition off by a step (2^-23) of a
    partial sum of at most `size`: 128 * 2^-23 = 2^-16 of it.  Scores off by x (in
    nats) move the output by sum p x (v - out), x dev at most; twice that is taken for
    what is not of first order.
    Weights: bf16 rounds them by 2^-8 in numerator and denominator alike: 2^-8 dev
    (and a step more for the products of two roundings).  fp8 pools round the
    numerator's to fp16, 2^-11 mag, or, where a weight times its token's scale is under
    2^-14 of the largest of them, by 2^-25 of that largest: a scale is under
    max|v| / 224 and a code at most 448, so 2 * 2^-25 `top` over all tokens; queries as
    fp16 lose 2^-25 of the row's largest element each, inside the scores' 2^-16.
    Segments of many rows of an fp8 pool run the bf16 kernel's products on the exact
    bf16 values of the codes, its weights rounded to bf16 too: the larger of the two.  The exponentials, the running rescales
    and the merge: a few 2^-22 of mag each, below 2^-18 together.
    The stored output: half a step, 2^-8 of it in bf16, 2^-24 in fp32."""
    scores = 2 * 2.0 ** -16 * size * dev + 2.0 ** -18 * mag
    if kind == "fp32":
        return scores + 2.0 ** -24 * np.abs(out) + 1e-30
    weights = 1.01 * 2.0 ** -8 * dev
    if kind == "fp8":
        weights = np.maximum(weights, 2.0 ** -11 * mag + 2.0 ** -24 * top)
    return scores + weights + 2.0 ** -8 * (np.abs(out) + scores + weights) + 1e-30


def f64(t):
    return t.detach().double().cpu().numpy()


def held(x, kind):
    """What a pool of this kind holds of rows x (numpy, float64 of the append's dtype)."""
    return dequantise(*quantise(x)) if kind == "fp8" else x


POOL_DTYPE = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
ROW_DTYPE = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16}
