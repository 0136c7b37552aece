"""What the backward pass of the combine refuses about its rows (no GPU: the pointers are stand-ins that
are never read)."""
import ctypes
import os

import pytest

from capacity_routing_expert_amd import binding as B

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from capacity_routing_expert_amd import build
        build.build()
    return B.lib()


def at(i):
    return P((i + 1) << 20)  # 1 MiB apart


def test_rows_are_checked_without_capacity(lib):
    """With capacity 0 there are no rows, but a pointer to them is still held to its alignment."""
    s = B.make_shape(16, 64, 8, 8, 2, 0, B.MOE_BF16)
    call = lambda y: lib.moe_combine_backward(ctypes.byref(s), at(0), at(1), at(2), y, at(4), None, None)
    assert call(P(4104)) == 2 and "y_rows is not 16-byte" in B.last_error()


def rows(lib, n, s=None, **kw):
    a = dict(dout=at(0), gates=at(1), slots=at(2), y=at(3), dgates=at(4), dy=at(40))
    a.update(kw)
    s = B.make_shape(16, 64, 8, 8, 2, 100, B.MOE_BF16) if s is None else s
    return lib.moe_combine_backward_rows(ctypes.byref(s), a["dout"], a["gates"], a["slots"], a["y"], n,
                                         a["dgates"], a["dy"], None)


@pytest.mark.parametrize("kw,text", [
    (dict(dgates=P(at(3).value + 799 * 128)), "dgates overlaps dout or y_rows"),
    (dict(gates=P(at(40).value + 799 * 128)), "dy_rows overlaps topk_gates"),
    (dict(slots=P(at(40).value + 799 * 128)), "dy_rows overlaps topk_gates, slot_of"),
    (dict(dout=P(at(40).value + 799 * 128)), "dy_rows overlaps dout"),
    (dict(dgates=P(at(40).value + 799 * 128)), "dy_rows overlaps topk_gates, slot_of or dgates"),
    (dict(y=P(at(40).value + 799 * 128)), "dy_rows overlaps y_rows"),
])
def test_overlaps_in_the_padded_layouts_last_row(lib, kw, text):
    """16 tokens, top-2, 8 buffers of 100 rows of 128 bytes: 32 rows are kept at most, 800 are there."""
    assert rows(lib, 800, **kw) == 1
    assert text in B.last_error()


def test_counts_of_rows(lib):
    assert rows(lib, -1) == 1 and "n_rows = -1" in B.last_error()
    assert rows(lib, 1 << 31) == 2 and "2^31" in B.last_error()
    assert rows(lib, 5, y=None) == 1 and "y_rows is NULL" in B.last_error()
    assert rows(lib, 5, dgates=None, dy=None) == 1 and "both NULL" in B.last_error()
    assert rows(lib, 5, s=B.make_shape(0, 64, 8, 8, 2, 100, B.MOE_BF16), dout=None) == 0
    assert rows(lib, 5, s=B.make_shape(16, 64, 8, 8, 9, 100, B.MOE_BF16)) == 1
