"""Refusals of routing by scores, its backward pass, the bias update and AdamW, checked on the host
before anything is launched (no GPU: the pointers are stand-ins that are never read)."""
import ctypes
import os

import pytest
import torch

from capacity_routing_expert_amd import binding as B

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from capacity_routing_expert_amd import build
        build.build()
    return B.lib()


def shape(**kw):
    s = dict(T=16, d_model=64, d_ff=8, n_experts=8, top_k=2, capacity=0, dtype=B.MOE_BF16)
    s.update(kw)
    return B.make_shape(**s)


def at(i):
    return P((i + 1) << 20)  # 1 MiB apart


def raw_routing(**kw):
    r = dict(score=0, n_groups=1, topk_groups=1, group_score=0, renormalize=0, scale=1.0)
    r.update(kw)
    return B.MoeRouting(*r.values())


def route(lib, s=None, r=None, **kw):
    a = dict(x=at(0), w=at(1), b=None, bias=None, mask=None, ids=at(2), gates=at(3), logits=None,
             ws=at(8), ws_bytes=1 << 30)
    a.update(kw)
    s, r = shape() if s is None else s, raw_routing() if r is None else r
    return lib.moe_route_scored(ctypes.byref(s), ctypes.byref(r), *[a[n] for n in (
        "x", "w", "b", "bias", "mask", "ids", "gates", "logits", "ws", "ws_bytes")], None)


def back(lib, s=None, r=None, **kw):
    a = dict(logits=at(0), ids=at(1), dgates=at(2), add=None, mask=None, dlogits=at(4))
    a.update(kw)
    s, r = shape() if s is None else s, raw_routing() if r is None else r
    return lib.moe_route_scored_backward(ctypes.byref(s), ctypes.byref(r), *[a[n] for n in (
        "logits", "ids", "dgates", "add", "mask", "dlogits")], None)


@pytest.mark.parametrize("kw,text", [
    (dict(score=2), "score 2"), (dict(n_groups=0), "n_groups = 0"), (dict(n_groups=3), "n_groups = 3"),
    (dict(topk_groups=0), "topk_groups = 0"), (dict(topk_groups=2), "topk_groups = 2"),
    (dict(group_score=5), "group_score 5"), (dict(renormalize=2), "renormalize = 2"),
    (dict(n_groups=8, topk_groups=1), "top_k = 2 of 1 groups of 1"), (dict(scale=0.0), "scale = 0"),
    (dict(scale=-1.0), "scale"), (dict(scale=float("inf")), "scale"), (dict(scale=float("nan")), "scale"),
])
def test_routing_refusals(lib, kw, text):
    assert route(lib, r=raw_routing(**kw)) == 1
    assert text in B.last_error()
    assert back(lib, r=raw_routing(**kw)) == 1
    assert text in B.last_error()


@pytest.mark.parametrize("kw,status,text", [
    (dict(x=None), 1, "x is NULL"), (dict(w=None), 1, "w_router is NULL"),
    (dict(ids=None), 1, "topk_ids is NULL"), (dict(gates=None), 1, "topk_gates is NULL"),
    (dict(x=P(4104)), 2, "16-byte"), (dict(b=P(4098)), 2, "aligned"), (dict(bias=P(4098)), 2, "aligned"),
    (dict(logits=P(4097)), 2, "aligned"), (dict(ws_bytes=16), 3, "workspace"),
    (dict(ws=None), 1, "workspace is NULL"), (dict(ws=P(4100)), 2, "256-byte"),
])
def test_route_scored_refusals(lib, kw, status, text):
    assert route(lib, **kw) == status
    assert text in B.last_error()


@pytest.mark.parametrize("kw,status,text", [
    (dict(logits=None), 1, "logits is NULL"), (dict(ids=None), 1, "topk_ids is NULL"),
    (dict(dgates=None), 1, "dgates is NULL"), (dict(dlogits=None), 1, "dlogits is NULL"),
    (dict(logits=P(4097)), 2, "aligned"), (dict(add=P(4098)), 2, "aligned"),
    (dict(dlogits=at(0)), 1, "dlogits overlaps logits"),
    (dict(dlogits=P(at(2).value - 4)), 1, "dlogits overlaps topk_ids or dgates"),
    (dict(add=P(at(4).value + 16)), 1, "dlogits_add overlaps dlogits"),
])
def test_route_scored_backward_refusals(lib, kw, status, text):
    assert back(lib, **kw) == status
    assert text in B.last_error()


def test_null_structs_and_bad_shapes(lib):
    s = shape()
    assert lib.moe_route_scored(ctypes.byref(s), None, *[at(0)] * 9, 1 << 20, None) == 1
    assert "routing is NULL" in B.last_error()
    assert lib.moe_route_scored_backward(ctypes.byref(s), None, *[at(0)] * 6, None) == 1
    for bad in (dict(top_k=9), dict(n_experts=300), dict(T=-1), dict(d_model=12), dict(dtype=3)):
        s = shape(**bad)
        assert route(lib, s) != 0 and back(lib, s) != 0 and bias(lib, s) != 0
        assert B.workspace_bytes_route_scored(s) == 0 and B.workspace_bytes_balance_bias(s) == 0
    big = shape(T=1, d_model=1 << 22, d_ff=8, n_experts=256, dtype=B.MOE_F32)  # W_r of 4 GiB
    assert route(lib, big) == 2 and "w_router" in B.last_error()
    assert route(lib, shape(T=0), x=None, ids=None, ws=None, ws_bytes=0) == 0
    assert back(lib, shape(T=0), logits=None, dlogits=None) == 0


def test_workspaces_are_bounded(lib):
    for T in (1, 63, 4095, 4096, 100000, 1 << 24):
        for E in (1, 8, 64, 256):
            s = shape(T=T, n_experts=E, top_k=1, d_model=8)
            assert 0 < B.workspace_bytes_route_scored(s) <= 64 << 20
            assert B.workspace_bytes_route_scored(s) % 256 == 0


@pytest.mark.parametrize("E", [1, 8, 9, 48, 64, 250])
@pytest.mark.parametrize("d", [8, 136, 1000, 2048, 8192])
def test_a_workspace_serves_smaller_batches(lib, E, d):
    last = [0, 0]
    for T in sorted({*range(1, 700, 9), *range(700, 70000, 613), 2047, 2048, 16384, 16385, 16400}):
        now = [B.workspace_bytes_route_scored(shape(T=T, n_experts=E, top_k=1, d_model=d)),
               B.workspace_bytes_balance_bias(shape(T=T, n_experts=E, top_k=1, d_model=d))]
        assert now[0] >= last[0] and now[1] >= last[1], T
        last = now


def comb(lib, s=None, **kw):
    a = dict(dout=at(0), gates=at(1), slots=at(2), y=at(3), dgates=at(4), dy=at(5))
    a.update(kw)
    s = shape(capacity=8) if s is None else s
    return lib.moe_combine_backward(ctypes.byref(s), *[a[n] for n in (
        "dout", "gates", "slots", "y", "dgates", "dy")], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dgates=None, dy=None), 1, "both NULL"), (dict(dout=None), 1, "dout is NULL"),
    (dict(gates=None), 1, "topk_gates is NULL"), (dict(slots=None), 1, "slot_of is NULL"),
    (dict(y=None), 1, "y_rows is NULL"), (dict(dout=P(4104)), 2, "16-byte"),
    (dict(dy=P(4104)), 2, "16-byte"), (dict(dgates=P(4097)), 2, "aligned"),
    (dict(dgates=at(1)), 1, "dgates overlaps"), (dict(dy=at(0)), 1, "dy_rows overlaps dout"),
    (dict(dy=P(at(3).value + 16)), 1, "dy_rows overlaps y_rows"),
    (dict(dgates=at(0)), 1, "dgates overlaps dout"), (dict(dgates=at(3)), 1, "dgates overlaps dout or y"),
    (dict(dy=at(1)), 1, "dy_rows overlaps topk_gates"), (dict(dy=at(2)), 1, "slot_of or dgates"),
    (dict(dgates=at(5)), 1, "slot_of or dgates"),
])
def test_combine_backward_refusals(lib, kw, status, text):
    assert comb(lib, **kw) == status
    assert text in B.last_error()


def test_combine_backward_empty(lib):
    assert comb(lib, shape(T=0), dout=None, slots=None) == 0
    for bad in (dict(top_k=9), dict(T=-1), dict(d_model=12), dict(dtype=3)):
        assert comb(lib, shape(**bad)) != 0


def bias(lib, s=None, **kw):
    a = dict(ids=at(0), mask=None, rate=0.5, bias=at(1), counts=at(2), ws=at(3), ws_bytes=1 << 20)
    a.update(kw)
    s = shape() if s is None else s
    return lib.moe_balance_bias(ctypes.byref(s), *[a[n] for n in (
        "ids", "mask", "rate", "bias", "counts", "ws", "ws_bytes")], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(bias=None), 1, "score_bias is NULL"), (dict(ids=None, counts=None), 1, "both NULL"),
    (dict(rate=float("nan")), 1, "rate"), (dict(rate=-1.0), 1, "rate"),
    (dict(bias=P(4097)), 2, "aligned"), (dict(counts=P(4097)), 2, "aligned"),
    (dict(ids=P(4097)), 2, "aligned"), (dict(counts=P(at(1).value + 16)), 1, "overlaps"),
])
def test_balance_bias_refusals(lib, kw, status, text):
    assert bias(lib, **kw) == status
    assert text in B.last_error()


def test_balance_bias_workspace(lib):
    long = shape(T=100000)
    assert B.workspace_bytes_balance_bias(long) > 0 and B.workspace_bytes_balance_bias(shape()) == 0
    assert bias(lib, long, ws_bytes=16) == 3 and bias(lib, long, ws=None) == 1
    assert bias(lib, long, ws=P(4100)) == 2


# ---------------------------------------------------------------- AdamW
def config(**kw):
    c = dict(param_dtype=0, grad_dtype=0, state_bits=32, lr=0.1, beta1=0.9, beta2=0.99, eps=1e-8,
             grad_scale=1.0, step=1, dynamic=None)
    c.update(kw)
    return B.MoeAdamWConfig(*c.values())


def tensors(count=1, **kw):
    arr = (B.MoeAdamWTensor * count)()
    for i in range(count):
        t = dict(param=at(10 * i), grad=at(10 * i + 1), m=at(10 * i + 2), v=at(10 * i + 3),
                 m_steps=None, v_steps=None, copy=None, n=1000, weight_decay=0.0)
        t.update(kw)
        arr[i] = B.MoeAdamWTensor(*t.values())
    return arr


def step(lib, c=None, ts=None, n=1):
    c, ts = config() if c is None else c, tensors() if ts is None else ts
    return lib.moe_adamw_step(ctypes.byref(c), ts, n, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(state_bits=16), 1, "state_bits"), (dict(param_dtype=3), 2, "param_dtype"),
    (dict(grad_dtype=-1), 2, "grad_dtype"), (dict(beta1=1.0), 1, "beta1"), (dict(beta2=-0.1), 1, "beta2"),
    (dict(beta1=float("nan")), 1, "beta1"), (dict(eps=0.0), 1, "eps"), (dict(eps=float("inf")), 1, "eps"), (dict(eps=1e-39), 1, "eps"),
    (dict(lr=-1.0), 1, "lr"), (dict(lr=float("nan")), 1, "lr"), (dict(grad_scale=float("inf")), 1, "grad"),
    (dict(step=0), 1, "step = 0"), (dict(dynamic=4098), 2, "dynamic"),
])
def test_adamw_config_refusals(lib, kw, status, text):
    assert step(lib, config(**kw)) == status
    assert text in B.last_error()
    assert lib.moe_adamw_check(ctypes.byref(config(**kw)), tensors(), 1) == status


@pytest.mark.parametrize("kw,bits,status,text", [
    (dict(param=None), 32, 1, "tensors[0].param is NULL"), (dict(grad=None), 32, 1, "grad is NULL"),
    (dict(m=None), 32, 1, "m is NULL"), (dict(v=None), 8, 1, "v is NULL"),
    (dict(m_steps=at(5)), 32, 1, "steps with 32-bit"), (dict(m_steps=at(5)), 8, 1, "v_steps is NULL"),
    (dict(param=P(4098)), 32, 2, "4-byte"), (dict(m=P(4098)), 32, 2, "4-byte"),
    (dict(copy=P(4097)), 32, 2, "2-byte"), (dict(n=-1), 32, 1, "n = -1"),
    (dict(n=(1 << 33) + 1), 32, 2, "2^33"), (dict(weight_decay=-0.1), 32, 1, "weight_decay"),
    (dict(weight_decay=float("nan")), 32, 1, "weight_decay"),
])
def test_adamw_tensor_refusals(lib, kw, bits, status, text):
    assert step(lib, config(state_bits=bits), tensors(**kw)) == status
    assert text in B.last_error()


def test_adamw_lists(lib):
    c = config()
    assert lib.moe_adamw_step(None, tensors(), 1, None) == 1
    assert lib.moe_adamw_step(ctypes.byref(c), None, 1, None) == 1
    assert lib.moe_adamw_step(ctypes.byref(c), tensors(), -1, None) == 1
    assert lib.moe_adamw_step(ctypes.byref(c), None, 0, None) == 0  # nothing to do
    assert step(lib, ts=tensors(n=0, param=None, grad=None)) == 0
    assert step(lib, config(param_dtype=1), tensors(copy=at(8))) == 1
    assert "copy of a bf16 param" in B.last_error()


def test_adamw_check_finds_overlaps(lib):
    check = lambda ts, n, **kw: lib.moe_adamw_check(ctypes.byref(config(**kw)), ts, n)
    ts = tensors(3)
    assert check(ts, 3) == 0
    ts[2].grad = ts[1].grad  # gradients are only read
    assert check(ts, 3) == 0
    ts[2].param = ts[0].param  # the same param twice
    assert check(ts, 3) == 1 and "overlaps" in B.last_error()
    ts = tensors(2)
    ts[1].grad = at(0).value + 3996  # the last element of the first param
    assert check(ts, 2) == 1
    ts[1].grad = at(0).value + 4000
    assert check(ts, 2) == 0
    ts = tensors(2)
    ts[0].copy = ts[1].v
    assert check(ts, 2) == 1
    q = dict(m_steps=at(5), v_steps=P(at(5).value + 12))  # 4 blocks of 256: 16 bytes each
    assert check(tensors(1, **q), 1, state_bits=8) == 1
    q["v_steps"] = P(at(5).value + 16)
    assert check(tensors(1, **q), 1, state_bits=8) == 0


def test_adamw_moments_refusals(lib):
    out = lambda p: (P * 1)(p)
    call = lambda c, ts, m, v: lib.moe_adamw_moments(ctypes.byref(c), ts, 1, m, v, None)
    assert call(config(state_bits=4), tensors(), None, None) == 1
    assert call(config(), tensors(m=None), None, None) == 1
    assert call(config(), tensors(), out(at(2)), None) == 1 and "overlaps the state" in B.last_error()
    assert call(config(), tensors(), out(at(7)), out(at(7))) == 1 and "m_out overlaps" in B.last_error()
    assert call(config(), tensors(), out(4098), None) == 2


def test_binding_checks(lib):
    f = torch.zeros
    with pytest.raises(ValueError, match="score 'tanh'"):
        B.make_routing("tanh")
    with pytest.raises(ValueError, match="group_score"):
        B.make_routing(group_score="mean")
    s, r = shape(), B.make_routing()
    with pytest.raises(TypeError, match="x has dtype"):
        B.moe_route_scored(s, r, f(16, 64), None, None, None, None, None)
    with pytest.raises(ValueError, match="score_bias holds 7 elements, the shape needs 8"):
        B.moe_route_scored(s, r, None, None, None, f(7), None, None)
    with pytest.raises(ValueError, match="must be on the GPU"):
        B.moe_route_scored_backward(s, r, f(16, 8), None, None, None)
    with pytest.raises(TypeError, match="token_mask has dtype"):
        B.moe_balance_bias(s, 0.1, None, token_mask=f(16, dtype=torch.bool))
    with pytest.raises(ValueError, match="grads has 1 entries, params 2"):
        B.AdamWTensors([f(4), f(4)], [f(4)], [f(4)] * 2, [f(4)] * 2)
    with pytest.raises(TypeError, match="params: one dtype"):
        B.AdamWTensors([f(4), f(4).bfloat16()], [f(4)] * 2, [f(4)] * 2, [f(4)] * 2)
    with pytest.raises(ValueError, match="must be on the GPU"):
        B.AdamWTensors([f(4)], [f(4)], [f(4)], [f(4)])
