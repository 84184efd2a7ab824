"""Host-side refusals of the calls for rows that do not stand at their own positions, without a GPU."""
import ctypes
import struct

import pytest

from copy_write_forked_gb300 import dendrite as D


@pytest.fixture(scope="module")
def L():
    import __graft_entry__ as g
    g.build()
    return D.lib()


def test_calls_reject_a_null_pool(L):
    assert L.dendrite_fork_rows(None, None, None, None, 0, None, 0, None, None) == -1
    assert L.dendrite_append_rope_at(None, None, 0, 0, None, None, None, None, 0, None, None, None) == -1
    assert L.dendrite_append_layer_rope_at(None, 0, None, None, None, None, 0, None, None, None) == -1
    assert L.dendrite_tree_attn_cross(None, 0, None, 1, 1, None, 1, None, None) == -1
    assert L.dendrite_verify_draft(None, 1, 1, None, 1, None, 1, 0, None, 1, None, 1, None, None, None, None, None, None) == -1


def test_axes_of_a_rope(L):
    assert D.Rope(128).n_axes == 1
    assert D.Rope(128, axes=[0] * 16 + [1] * 24 + [2] * 24).n_axes == 3
    assert D.Rope(32, axes=[3] * 16).n_axes == 4
    for axes in ([], [0] * 63, [0] * 65, [4] + [0] * 63, [-1] + [0] * 63):
        with pytest.raises(D.DendriteError):
            D.Rope(128, axes=axes)


def test_positions_are_laid_out_as_the_header_has_them():
    """Pointer, three strides, two int32 and 128 axis bytes: what the binding packs is the C struct."""

    class Positions(ctypes.Structure):
        _fields_ = [("at", ctypes.c_void_p), ("branch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                    ("axis_stride", ctypes.c_int64), ("n_axes", ctypes.c_int32), ("reserved", ctypes.c_int32),
                    ("axis", ctypes.c_uint8 * 128)]

    assert D._POSITIONS.size == ctypes.sizeof(Positions) == 168
    p = Positions.from_buffer_copy(D._POSITIONS.pack(16, 3, 2, 1, 3, 0, bytes(range(128))))
    assert (p.at, p.branch_stride, p.token_stride, p.axis_stride, p.n_axes, p.reserved) == (16, 3, 2, 1, 3, 0)
    assert list(p.axis) == list(range(128)) and struct.calcsize("P") == 8
