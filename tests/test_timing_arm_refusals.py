"""moe_set_gemm_timing and moe_set_stage_timing arm the next layer call on the thread, which consumes
the arms even if it is refused (no GPU: the events and pointers are stand-ins that are never used)."""
import ctypes
import os

import pytest

from capacity_routing_expert_amd import binding as B

P = ctypes.c_void_p
HANDLES = (P * 4)(1, 2, 3, 4)
SIX = (P * 6)(1, 2, 3, 4, 5, 6)
NULL_LAST = (P * 6)(1, 2, 3, 4, 5, 0)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from capacity_routing_expert_amd import build
        build.build()
    L = B.lib()
    yield L
    L.moe_set_gemm_timing(None)
    L.moe_set_stage_timing(None)


def refused(lib, name, case):
    """Status of a call that is refused for the case's reason."""
    at = [P((i + 1) << 24) for i in range(24)]
    s = B.make_shape(16, 64, 96, 8, 99 if case == "shape" else 2, 4, B.MOE_BF16)
    if case == "scratch":
        s = B.make_shape(1 << 20, 64, 96, 8, 2, 1 << 20, B.MOE_BF16)
    sp = ctypes.byref(s)
    events = NULL_LAST if case == "event 5" else None
    x, wr, br, w1, b1, w2, b2 = (None if case == "x" else at[0]), at[1], None, *at[2:6]
    out, outs, ws, n = at[6], [None] * 5, at[7], (16 if case == "workspace" else 1 << 30)
    q = B.MoeQuantizedExperts(at[8], at[9], at[10], at[11], at[12], at[13], 32, 0)
    if name == "moe_layer_forward":
        return lib.moe_layer_forward(sp, x, wr, br, w1, b1, w2, b2, out, *outs, ws, n, None)
    if name == "moe_layer_forward_profiled":
        return lib.moe_layer_forward_profiled(sp, x, wr, br, w1, b1, w2, b2, out, *outs, ws, n, None,
                                              events if case.startswith("event") else SIX)
    if name == "moe_layer_forward_padded":
        return lib.moe_layer_forward_padded(sp, x, wr, br, w1, b1, w2, b2, out, *outs, None, ws, n,
                                            None, events)
    if name == "moe_layer_forward_gated":
        return lib.moe_layer_forward_gated(sp, x, wr, br, w1, w2, out, *outs, ws, n, None, events)
    if name == "moe_layer_forward_quantized":
        return lib.moe_layer_forward_quantized(sp, x, wr, br,
                                               None if case == "experts" else ctypes.byref(q), out,
                                               *outs, ws, n, None, events)
    assert name == "moe_layer_forward_noalloc"
    return lib.moe_layer_forward_noalloc(sp, x, wr, br, w1, b1, w2, b2, out, *outs, None)


CASES = [(n, c) for n in ("moe_layer_forward", "moe_layer_forward_profiled",
                          "moe_layer_forward_padded", "moe_layer_forward_gated",
                          "moe_layer_forward_quantized")
         for c in ("shape", "x", "workspace")]
CASES += [(n, "event 5") for n in ("moe_layer_forward_profiled", "moe_layer_forward_padded",
                                   "moe_layer_forward_gated", "moe_layer_forward_quantized")]
CASES += [("moe_layer_forward_profiled", "events"), ("moe_layer_forward_quantized", "experts"),
          ("moe_layer_forward_noalloc", "shape"), ("moe_layer_forward_noalloc", "scratch")]


@pytest.mark.parametrize("name,case", CASES)
def test_a_refused_call_disarms(lib, name, case):
    assert lib.moe_set_gemm_timing(HANDLES) == 0
    assert lib.moe_set_stage_timing(HANDLES) == 0
    assert refused(lib, name, case) != 0
    # an empty batch records whatever is still armed, which fails for these handles
    s = B.make_shape(0, 64, 96, 8, 2, 4, B.MOE_BF16)
    assert lib.moe_layer_forward(ctypes.byref(s), *[None] * 14, 0, None) == 0, B.last_error()
