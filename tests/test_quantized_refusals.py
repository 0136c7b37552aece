"""4-bit experts on the host: storage sizes, the references' storage against the header's formula,
and refusals before anything is launched (no GPU: the pointers are stand-ins)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import quant_ref as Q
from capacity_routing_expert_amd import binding as B

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from capacity_routing_expert_amd import build
        build.build()
    return B.lib()


def shape(**kw):
    s = dict(T=16, d_model=64, d_ff=96, n_experts=8, top_k=2, capacity=4, dtype=B.MOE_BF16)
    s.update(kw)
    return B.make_shape(**s)


def at(i):
    return P((i + 1) << 24)


def test_reference_storage_is_the_header_formula():
    rng = np.random.default_rng(0)
    E, rows, cols = 2, 24, 200
    codes = rng.integers(0, 16, (E, rows, cols)).astype(np.uint8)
    words = Q.pack(codes).view(np.uint32)
    KC = 2
    for _ in range(500):
        e, r, c = rng.integers(E), rng.integers(rows), rng.integers(cols)
        block = (e * KC + c // 128) * (rows // 8) + r // 8
        cb = c % 128
        word = words[block * 128 + (cb % 32 // 8 * 8 + r % 8) * 4 + cb // 32]
        assert word >> (4 * (cb % 8)) & 15 == codes[e, r, c]


def test_sizes(lib):
    s = shape()
    assert B.quantized_codes_bytes(s, 96, 64) == 8 * 12 * 1 * 512
    assert B.quantized_codes_bytes(s, 64, 1408) == 8 * 8 * 11 * 512
    assert B.quantized_scales_bytes(s, 96, 136, 32) == 8 * 96 * 2 * 4 * 2
    assert B.quantized_scales_bytes(s, 96, 136, 128) == 8 * 96 * 2 * 2
    for rows, cols, group in ((12, 64, 32), (16, 12, 32), (16, 64, 48), (0, 64, 32)):
        assert B.quantized_scales_bytes(s, rows, cols, group) == 0
    assert B.quantized_codes_bytes(shape(top_k=9), 16, 64) == 0


@pytest.mark.parametrize("kw,status,text", [
    (dict(w=None), 1, "w is NULL"), (dict(codes=None), 1, "codes is NULL"),
    (dict(scales=P(4104)), 2, "16-byte"), (dict(rows=12), 2, "multiples of 8"),
    (dict(cols=20), 2, "multiples of 8"), (dict(cols=0), 1, ">= 1"), (dict(group=16), 1, "group"),
    (dict(codes=P((1 << 24) + 64)), 1, "overlap"), (dict(scales=at(1)), 1, "overlap"),
])
def test_quantize_refusals(lib, kw, status, text):
    a = dict(w=at(0), rows=96, cols=64, group=32, codes=at(1), scales=at(2))
    a.update(kw)
    s = shape()
    assert lib.moe_quantize_weights(ctypes.byref(s), a["w"], a["rows"], a["cols"], a["group"],
                                    a["codes"], a["scales"], None) == status
    assert text in B.last_error()


@pytest.mark.parametrize("kw,status,text", [
    (dict(w=None), 1, "w is NULL"), (dict(codes=None), 1, "codes is NULL"),
    (dict(scales=P(4104)), 2, "16-byte"), (dict(rows=12), 2, "multiples of 8"),
    (dict(cols=20), 2, "multiples of 8"), (dict(group=16), 1, "group"),
    (dict(w=at(1)), 1, "overlaps"), (dict(w=P(at(2).value + 64)), 1, "overlaps"),
])
def test_dequantize_refusals(lib, kw, status, text):
    a = dict(w=at(0), rows=96, cols=64, group=32, codes=at(1), scales=at(2))
    a.update(kw)
    s = shape()
    assert lib.moe_dequantize_weights(ctypes.byref(s), a["codes"], a["scales"], a["rows"],
                                      a["cols"], a["group"], a["w"], None) == status
    assert text in B.last_error()


def experts(**kw):
    a = dict(w1_codes=at(0), w1_scales=at(1), b1=at(2), w2_codes=at(3), w2_scales=at(4), b2=at(5),
             group=32, gated=0)
    a.update(kw)
    return B.MoeQuantizedExperts(**a)


GATED = dict(gated=1, b1=None, b2=None)


@pytest.mark.parametrize("shape_kw,kw,status,text", [
    ({}, dict(w1_codes=None), 1, "w1_codes is NULL"), ({}, dict(w2_scales=P(8)), 2, "aligned"),
    ({}, dict(b1=None), 1, "b1 is NULL"), ({}, dict(group=0), 1, "group"),
    ({}, dict(gated=2), 1, "gated"), ({}, dict(gated=1), 1, "no biases"),
    (dict(dtype=B.MOE_F32), {}, 2, "bf16 only"),
    (dict(weight_layout=B.MOE_WEIGHTS_PACKED), {}, 1, "own storage"),
    ({}, dict(GATED, w2_codes=P(4)), 2, "w2_codes"), (dict(top_k=99), {}, 1, "top_k"),
    (dict(d_model=1 << 16, d_ff=1 << 16), {}, 2, "2 GiB"),
    (dict(d_model=1 << 16, d_ff=1 << 15), GATED, 2, "2 GiB"),
])
def test_expert_refusals(lib, shape_kw, kw, status, text):
    s, q = shape(**shape_kw), experts(**kw)
    assert lib.moe_expert_ffn_quantized(ctypes.byref(s), at(6), at(7), at(8), ctypes.byref(q),
                                        at(9), at(10), 1 << 30, None) == status
    assert text in B.last_error()
    assert lib.moe_layer_forward_quantized(ctypes.byref(s), at(6), at(7), None, ctypes.byref(q),
                                           at(9), None, None, None, None, None, at(10), 1 << 30,
                                           None, None) == status
    assert text in B.last_error()


def test_call_refusals(lib):
    s, q = shape(), experts()
    call = lambda x=at(6), rt=at(7), off=at(8), qq=ctypes.byref(q), y=at(9), ws=at(10), n=1 << 30: \
        lib.moe_expert_ffn_quantized(ctypes.byref(s), x, rt, off, qq, y, ws, n, None)
    assert call(x=None) == 1 and call(rt=None) == 1 and call(off=None) == 1 and call(y=None) == 1
    assert call(qq=None) == 1 and call(ws=None) == 1 and call(n=100) == 3 and call(x=P(8)) == 2
    layer = lambda out, ev=None: lib.moe_layer_forward_quantized(
        ctypes.byref(s), at(6), at(7), None, ctypes.byref(q), out, None, None, None, None, None,
        at(10), 1 << 30, None, ev)
    assert layer(at(6)) == 1 and "aliases" in B.last_error()
    assert layer(at(9), (P * 6)(1, 2, 3, 4, 5, 0)) == 1 and "events[5]" in B.last_error()
    empty = shape(T=0)
    assert lib.moe_expert_ffn_quantized(ctypes.byref(empty), None, None, None, ctypes.byref(q),
                                        None, None, 0, None) == 0


def test_binding_checks(lib):
    u8, bf = torch.uint8, torch.bfloat16
    z = lambda n, t: torch.zeros(n, dtype=t)
    args = dict(w1_codes=z(8 * 12 * 512, u8), w1_scales=z(8 * 96 * 4, bf), b1=z(8 * 96, bf),
                w2_codes=z(8 * 8 * 512, u8), w2_scales=z(8 * 64 * 4, bf), b2=z(8 * 64, bf))
    for name in args:
        short = dict(args)
        for other in args:
            if other != name:
                short[other] = None
        short[name] = args[name][:-1]
        with pytest.raises(ValueError, match=f"{name} holds"):
            B.QuantizedExperts(8, 64, 96, 32, False, **short)
    with pytest.raises(ValueError, match="must be on the GPU"):
        B.QuantizedExperts(8, 64, 96, 32, False, **args)
    with pytest.raises(ValueError, match="no biases"):
        B.QuantizedExperts(8, 64, 96, 32, True, **args)
    with pytest.raises(B.MoeError):
        B.QuantizedExperts(8, 64, 96, 48, False, **args)
    with pytest.raises(B.MoeError):
        B.QuantizedExperts(8, 60, 96, 32, False, **args)
    with pytest.raises(ValueError, match="experts"):
        B.moe_quantize_weights(shape(), torch.zeros(3, 8, 8, dtype=bf), 32, None, None)


def test_matrices_of_2_gib_are_refused(lib):
    """Also where E x rows x cols would leave 64 bits."""
    s = shape(n_experts=256)
    assert B.quantized_codes_bytes(s, 1 << 16, (1 << 16) - 128) == 256 * (2 ** 31 - 2 ** 22)
    for rows, cols in ((1 << 16, 1 << 16), (1 << 30, 1 << 30), (8, (1 << 31) - 8), ((1 << 31) - 8, 8)):
        big = -(-cols // 128) * 64 * rows >= 1 << 31
        assert big == (B.quantized_codes_bytes(s, rows, cols) == 0)
        assert big == (B.quantized_scales_bytes(s, rows, cols, 32) == 0)
        if big:
            assert lib.moe_quantize_weights(ctypes.byref(s), at(0), rows, cols, 32, at(1), at(2),
                                            None) == 2
            assert "2 GiB" in B.last_error()


def test_experts_have_to_fit_together(lib):
    from capacity_routing_expert_amd import layer as L
    w = lambda *n: torch.zeros(n, dtype=torch.bfloat16)
    for w1, w2, gated in ((w(2, 64, 96), w(2, 64, 96), False),   # W1 as [E, d, f]
                          (w(2, 96, 64), w(2, 64, 96), True),    # W1 for a W13
                          (w(2, 192, 64), w(2, 64, 96), False), (w(3, 96, 64), w(2, 64, 96), False)):
        with pytest.raises(ValueError, match="w1 has to be"):
            L.quantize_experts(w1, None, w2, None, 32, gated)
    with pytest.raises(ValueError, match="different devices"):
        B.QuantizedExperts(1, 8, 8, 32, True, torch.zeros(512, dtype=torch.uint8, device="meta"),
                           w(32), None, torch.zeros(512, dtype=torch.uint8), w(32), None)


def test_a_refused_call_consumes_the_timing_arm(lib):
    """A second set of handles may then be armed and disarmed; the refused call left nothing that
    a later call would record into."""
    events = (ctypes.c_void_p * 4)(1, 2, 3, 4)
    s = shape(T=0)
    assert lib.moe_set_gemm_timing(events) == 0
    assert lib.moe_set_stage_timing(events) == 0
    none = [None] * 7
    assert lib.moe_layer_forward_quantized(ctypes.byref(s), None, None, None, None, *none, 0, None,
                                           None) == 1
    ok = B.MoeQuantizedExperts()
    # an empty batch records what is armed: nothing is
    assert lib.moe_layer_forward_quantized(ctypes.byref(s), None, None, None, ctypes.byref(ok), *none,
                                           0, None, None) == 0
