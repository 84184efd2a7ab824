"""Host side of the row operators, without a GPU: rotary frequencies, what the
calls refuse before any device work, and the references the GPU tests use."""
import ctypes
import math
import random

import numpy as np
import pytest
import torch

import _rows as R


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("rot", [16, 32, 64, 96, 128, 256])
@pytest.mark.parametrize("scaling,factor,length", [("none", 1.0, 0.0), ("linear", 4.0, 0.0), ("ntk", 2.5, 0.0),
                                                   ("yarn", 4.0, 4096.0), ("yarn", 1.0, 4096.0), ("bands", 8.0, 8192.0)])
def test_rope_frequencies(rot, scaling, factor, length):
    from copy_write_forked_gb300.dendrite import Rope
    r = Rope(rot, base=500000.0, scaling=scaling, factor=factor, original_len=length)
    f, m = R.frequencies(rot, 500000.0, scaling, factor, length)
    assert len(r.inv_freq) == rot // 2
    # a handful of operations and a pow: 2^-48 is far above their rounding and far below a wrong formula
    assert np.allclose(r.inv_freq, f, rtol=2.0 ** -48, atol=0)
    assert math.isclose(r.scale, m, rel_tol=2.0 ** -50)


def test_rope_custom_frequencies_and_scale():
    from copy_write_forked_gb300.dendrite import DendriteError, Rope
    r = Rope(16, inv_freq=[0.5] * 8, scale=1.25, interleaved=True)
    assert r.inv_freq == [0.5] * 8 and r.scale == 1.25
    with pytest.raises(DendriteError):
        Rope(16, inv_freq=[0.5] * 7)


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=8), dict(rot_dim=24), dict(rot_dim=272), dict(rot_dim=64, base=1.0),
                                dict(rot_dim=64, base=float("nan")), dict(rot_dim=64, scaling="linear", factor=0.5),
                                dict(rot_dim=64, scaling="linear", factor=float("inf")),
                                dict(rot_dim=64, scaling="yarn", factor=2.0),
                                dict(rot_dim=64, scaling="bands", factor=2.0, original_len=100.0, turns_low=4.0, turns_high=4.0),
                                dict(rot_dim=64, scaling="other")])
def test_rope_refusals(kw):
    from copy_write_forked_gb300.dendrite import DendriteError, Rope
    with pytest.raises(DendriteError) as e:
        Rope(**kw)
    assert e.value.name == "EINVAL"


def test_null_pool_is_refused():
    from copy_write_forked_gb300.dendrite import lib
    L, one = lib(), (ctypes.c_int32 * 4)()
    p = ctypes.addressof(one)
    assert L.dendrite_append_rope(None, p, 1, 1, None, 0, p, p, None, 0, None, None, None) == -1
    assert L.dendrite_append_layer_rope(None, 0, None, 0, p, p, None, 0, None, None, None) == -1
    assert L.dendrite_tree_attn_draft(None, 0, p, 1, 1, p, 1, p, 1, p, None) == -1
    assert L.dendrite_accept_draft(None, p, 1, 1, p, p, None) == -1
    assert L.dendrite_read_kv(None, 0, p, p, p, 1, p, p, None) == -1
    assert L.dendrite_rope_init(None, 16, 0, 10000.0, 0, 1.0, 0.0, 1.0, 4.0) == -1


def test_tree_arguments():
    from copy_write_forked_gb300.dendrite import DendriteError, _trees
    assert _trees(None, 3, 4)[1:] == (None, 0)
    assert _trees([-1, 0, 0, 2], 3, 4)[2] == 1
    assert _trees(torch.zeros(3, 4, dtype=torch.int32), 3, 4)[2] == 3
    for bad in (torch.zeros(4, dtype=torch.int64), torch.zeros(3, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32),
                torch.zeros(4, 3, dtype=torch.int32).T):
        with pytest.raises(DendriteError):
            _trees(bad, 3, 4)


def test_quantise_reference_against_the_cast():
    # the reference's codes against torch's cast of the scaled rows, and its scale against its definition
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((200, 128)) * np.exp2(rng.integers(-40, 40, (200, 1)))).to(torch.bfloat16)
    codes, e = R.quantise(x.double().numpy())
    y = torch.ldexp(x.float(), -torch.from_numpy(e).int()[:, None])
    assert y.abs().max() <= 448
    assert (y.abs().amax(1) > 224).all()
    assert np.array_equal(codes, y.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_quantise_reference_at_the_edges():
    x = np.zeros((6, 128))
    x[1, 0], x[1, 1] = 448.0, 2.0 ** -10            # the largest code; half the smallest: a tie, to even (zero)
    x[2, 0], x[2, 1] = 449.0, -1.0                  # one scale up
    x[3, 0], x[3, 1] = np.inf, 1.0
    x[4, 0] = 2.0 ** -133                           # the smallest bf16: the lowest scale
    x[5, 0] = 255 * 2.0 ** 120                      # the largest bf16: 256 * 2^120 would be past it
    codes, e = R.quantise(x)
    assert e.tolist() == [-126, 0, 1, 128, -126, 120] and R.E4M3[codes[5, 0]] == 240.0
    assert codes[1, 0] == 0x7e and codes[1, 1] == 0
    assert R.E4M3[codes[2, 0]] * 2 == 448.0 and R.E4M3[codes[2, 1]] * 2 == -1.0
    assert (codes[3] == 0x7f).all()                 # a row that is not finite is NaN throughout
    assert R.E4M3[codes[4, 0]] * 2.0 ** -126 == 2.0 ** -133


def test_trees_and_masks():
    rng = random.Random(1)
    for kind in ("random", "chain", "star"):
        p = R.tree(rng, 23, kind)
        see = R.seen(p, 5)
        assert see[:, :5].all()
        assert [int(r[5:].sum()) - 1 for r in see] == R.depths(p)
