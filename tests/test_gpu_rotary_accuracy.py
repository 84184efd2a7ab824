"""Sine and cosine of rotary positions, one at a time: pairs (1, 0) turned in an fp32
pool leave as (scale * cos a, scale * sin a) without another rounding."""
import numpy as np
import pytest
import torch

from copy_write_forked_gb300.dendrite import Pool, Rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()
    torch.cuda.set_device(0)


# How far a result may be off, relative to itself, in units of 2^-24 (fp32's half step).
# x = p + e is the distance to the nearest quarter turn, |x| <= pi/4, z = p^2; results up
# to sin(pi/4) come from its sine, those above from its cosine.
#   sine: p + st, st = p z t + ..., |st| <= 0.115 of the result.  t is off by 1.6 (its last
#     rounding, 1/6 as a float, what comes before it), z by 1, p z by one more, st's sum by
#     1: 4.6 of 0.115, that is 0.53.  What Taylor leaves out: 2^-28.7, that is 0.04.
#   cosine: w + ct, w = 1 - z/2 with its rounding carried in ct, |ct| <= 0.023 of the result
#     and off by some 5: 0.12, and 2^-33.
#   The last rounding: 1.  A scale other than 1 rounds st or ct once more: 0.12 and 0.03.
def _relative(want, scale):
    extra = scale != 1.0
    return np.where(np.abs(want) <= scale * 0.70711, 1.6 + 0.12 * extra, 1.15 + 0.03 * extra) * 2.0 ** -24


def _angle_error(pos, freq):
    """In radians: inv_freq / 2 pi is rounded twice in 64 bits (2^-52 of the angle), kept to 2^-64
    turns per position, and the turns are read to 2^-46 (two floats)."""
    return pos * freq * 2.0 ** -52 + 2 * np.pi * (pos * 2.0 ** -64 + 2.0 ** -46)


@pytest.mark.parametrize("scale", [1.0, 1.2071])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("where", ["anywhere", "near quarter turns", "near eighths", "far"])
def test_cosine_and_sine(where, interleaved, scale):
    rng = np.random.default_rng(7)
    d, n, base = 256, 1500, 50
    pairs = d // 2
    mid = base + n / 2
    if where == "anywhere":
        freq = 10000.0 ** (-np.arange(pairs) / pairs)
    elif where == "far":     # angles of up to 2^22 radians, as at positions of millions
        freq = rng.uniform(1.0, 2000.0, pairs)
    else:                    # turns close to k / 4 (or k / 8: where the quarter changes) at the middle position
        part = 4 if where == "near quarter turns" else 8
        k = 2 * rng.integers(0, 500, pairs) + (part == 8)
        off = rng.choice([-1, 1], pairs) * 2.0 ** rng.uniform(-26, -6, pairs)
        freq = 2 * np.pi * (k / part + off) / np.floor(mid)
    rope = Rope(d, interleaved=interleaved, inv_freq=[float(f) for f in freq], scale=scale)
    i = np.arange(pairs)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    K = torch.zeros(1, n, 1, d, device="cuda")
    K[..., torch.as_tensor(a, device="cuda")] = 1.0
    pool = Pool(120, 16, 1, d, torch.float32, max_branches=4, max_blocks_per_branch=120)
    br = [pool.new_branch()]
    z = torch.zeros(1, base, 1, d, device="cuda")
    pool.append_kv(br, z, z)
    q = pool.append_rope(br, K, torch.zeros_like(K), rope, Q=K.clone())
    k = pool.read_kv(br, [base], [n])[0]
    pool.sync()
    pos = (base + np.arange(n))[:, None]
    angle = pos.astype(np.longdouble) * np.asarray(rope.inv_freq, np.longdouble)
    m, slack = np.longdouble(np.float32(scale)), scale * _angle_error(pos, np.asarray(rope.inv_freq))
    for got in (q[0, :, 0], k[:, 0]):
        got = got.cpu().numpy().astype(np.longdouble)
        for cols, want in ((a, m * np.cos(angle)), (b, m * np.sin(angle))):
            err, bound = np.abs(got[:, cols] - want), _relative(want, scale) * np.abs(want) + slack
            assert (err <= bound).all(), float((err / bound).max())
    pool.close()
