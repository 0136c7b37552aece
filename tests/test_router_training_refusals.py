"""Refusals of moe_balance_loss and moe_route_backward, checked on the host before anything is
launched (no GPU: the pointers are stand-ins that are never read)."""
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


def balance(lib, s=None, **kw):
    a = dict(logits=at(0), ids=at(1), mask=None, coef=0.01, scale=1.0, loss=at(2), counts=None,
             probs=None, dlogits=None, ws=at(8), ws_bytes=1 << 30)
    a.update(kw)
    s = shape() if s is None else s
    return lib.moe_balance_loss(ctypes.byref(s), a["logits"], a["ids"], a["mask"], a["coef"],
                                a["scale"], a["loss"], a["counts"], a["probs"], a["dlogits"],
                                a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(logits=None), 1, "logits is NULL"), (dict(ids=None), 1, "topk_ids is NULL"),
    (dict(loss=None), 1, "loss is NULL"), (dict(logits=P(4097)), 2, "aligned"),
    (dict(dlogits=P(4098)), 2, "aligned"), (dict(counts=P(4097)), 2, "aligned"),
    (dict(coef=float("nan")), 1, "finite"), (dict(scale=float("inf")), 1, "finite"),
    (dict(ws_bytes=16), 3, "workspace"), (dict(ws=None), 1, "workspace is NULL"),
    (dict(ws=P(4100)), 2, "256-byte"), (dict(dlogits=P((1 << 20) + 64)), 1, "overlaps"),
])
def test_balance_loss_refusals(lib, kw, status, text):
    assert balance(lib, **kw) == status
    assert text in B.last_error()


def backward(lib, s=None, **kw):
    a = dict(x=at(0), w=at(1), logits=at(2), ids=at(3), dgates=at(4), dlogits=at(5), mask=None,
             add=None, dx=at(6), dw=at(7), db=at(9), ws=at(10), ws_bytes=1 << 30)
    a.update(kw)
    s = shape() if s is None else s
    return lib.moe_route_backward(ctypes.byref(s), *[a[n] for n in (
        "x", "w", "logits", "ids", "dgates", "dlogits", "mask", "add", "dx", "dw", "db", "ws",
        "ws_bytes")], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dx=None, dw=None, db=None), 1, "all NULL"),
    (dict(dgates=None, dlogits=None), 1, "both NULL"),
    (dict(logits=None), 1, "logits is NULL"), (dict(ids=None), 1, "topk_ids is NULL"),
    (dict(x=None), 1, "x is NULL"), (dict(w=None), 1, "w_router is NULL"),
    (dict(dx=None, add=at(11)), 1, "dx_add without dx"), (dict(dx=at(0)), 1, "dx overlaps x"),
    (dict(add=P(at(6).value + 16)), 1, "dx_add overlaps dx"), (dict(dw=P(4100)), 2, "16-byte"),
    (dict(x=P(4104)), 2, "16-byte"), (dict(dgates=P(4098)), 2, "aligned"),
    (dict(ws_bytes=1000), 3, "workspace"), (dict(ws=P(4100)), 2, "256-byte"),
])
def test_route_backward_refusals(lib, kw, status, text):
    assert backward(lib, **kw) == status
    assert text in B.last_error()


def test_bad_shapes(lib):
    for bad in (dict(top_k=9), dict(n_experts=300), dict(T=-1), dict(d_model=12), dict(dtype=3)):
        s = shape(**bad)
        assert balance(lib, s) != 0 and backward(lib, s) != 0
        assert B.workspace_bytes_balance(s) == 0 and B.workspace_bytes_route_backward(s) == 0


def test_workspace_sizes(lib):
    """dl in both layouts (bf16: 4 and 6 bytes an expert and token) and one partial dW at least."""
    s = shape(T=1000, d_model=128)
    assert B.workspace_bytes_route_backward(s) >= 1000 * 8 * 10 + 8 * 128 * 4
    assert B.workspace_bytes_route_backward(s) % 256 == 0
    assert B.workspace_bytes_balance(s) % 256 == 0


def test_binding_checks_sizes_and_devices(lib):
    s = shape()
    f = torch.zeros(16 * 8)
    ids = torch.zeros(32, dtype=torch.int32)
    with pytest.raises(ValueError, match="logits holds 127 elements, the shape needs 128"):
        B.moe_balance_loss(s, f[:127], ids, f)
    with pytest.raises(ValueError, match="must be on the GPU"):
        B.moe_balance_loss(s, f, ids, f)
    with pytest.raises(TypeError, match="token_mask has dtype"):
        B.moe_balance_loss(s, None, None, None, token_mask=torch.zeros(16, dtype=torch.bool))
    with pytest.raises(ValueError, match="dw_router holds 511 elements, the shape needs 512"):
        B.moe_route_backward(s, None, None, None, None, None, None, dw_router=torch.zeros(511))
    with pytest.raises(TypeError, match="dgates has dtype"):
        B.moe_route_backward(s, None, None, None, None, ids, None)
