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
