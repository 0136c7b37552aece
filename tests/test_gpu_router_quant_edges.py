"""The router-training and 4-bit operators where calls meet: pointers off their usual alignment,
offsets past 32 bits, streams side by side, graphs that share a workspace, timing arms, batches
without tokens or kept rows."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

import oracle.moe_oracle as O
import parity as P
import quant_ref as Q
import router_ref as R
from capacity_routing_expert_amd import binding as B
from capacity_routing_expert_amd import layer as L
from capacity_routing_expert_amd import workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    B.lib()  # loud failure if the library is missing
    yield
    torch.cuda.synchronize()


def shifted(t, n=1):
    """A copy of t whose first element lies n elements past an aligned address."""
    flat = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
    out = flat[n:].view(t.shape)
    out.copy_(t)
    return out


def router_inputs(T, d, E, k, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, d, generator=g, device=DEV).to(dtype)
    w = (torch.randn(E, d, generator=g, device=DEV) / d ** 0.5).to(dtype)
    logits = torch.randn(T, E, generator=g, device=DEV)
    ids = logits.topk(k, dim=1).indices.to(torch.int32).contiguous()
    dg = torch.randn(T, k, generator=g, device=DEV)
    mask = (torch.rand(T, generator=g, device=DEV) < 0.8).to(torch.uint8)
    return x, w, logits, ids, dg, mask


@pytest.mark.parametrize("T,E,k", [(37, 8, 2), (700, 64, 6), (2100, 256, 8), (5000, 12, 3)])
def test_arrays_off_16_bytes(T, E, k):
    """fp32, int32 and mask arrays need 4 bytes (the mask 1): the kernels that take rows in 16-byte
    pieces otherwise give the same values, within two of the bounds on each."""
    x, w, logits, ids, dg, mask = router_inputs(T, 64, E, k)
    lg64, id_np, m = logits.double().cpu().numpy(), ids.cpu().numpy(), mask.cpu().numpy()
    for n in (1, 2, 3):
        a = L.balance_loss(shifted(logits, n), shifted(ids, n), coef=0.5, token_mask=shifted(mask, n))
        loss, c, probs, grad = R.balance(lg64, id_np, m, 0.5, 1.0)
        bl, bp, bg = R.balance_bounds(lg64, id_np, m, 0.5, 1.0)
        assert np.array_equal(a["counts"].cpu().numpy(), c)
        assert abs(float(a["loss"]) - loss) <= bl
        assert np.all(np.abs(a["probs"].double().cpu().numpy() - probs) <= bp)
        assert np.all(np.abs(a["dlogits"].double().cpu().numpy() - grad) <= bg)
        got = L.route_backward(x, w, shifted(logits, n), shifted(ids, n), shifted(dg, n),
                               shifted(a["dlogits"], n), token_mask=shifted(mask, n))
        args = (x.double().cpu().numpy(), w.double().cpu().numpy(), lg64, id_np,
                dg.double().cpu().numpy(), a["dlogits"].double().cpu().numpy(), m, None)
        ref = R.route_backward(*args)[:3]
        for name, r, b in zip(("dx", "dw_router", "db_router"), ref,
                              R.route_backward_bounds(*args, True)):
            assert np.all(np.abs(got[name].double().cpu().numpy() - r) <= b), (name, n)


def test_f32_arrays_on_4_bytes():
    """fp32 x, W_r, dx, dx_add and dW_r need 4 bytes: each off 16 in turn, and all of them, give the
    bits of the aligned call (the sums are the same, only the pieces are not)."""
    T, d, E, k = 300, 64, 20, 3
    x, w, logits, ids, dg, mask = router_inputs(T, d, E, k, torch.float32)
    add = torch.randn(T, d, device=DEV)
    shape = B.make_shape(T, d, 8, E, k, 0, B.MOE_F32)
    ws = torch.empty(B.workspace_bytes_route_backward(shape), dtype=torch.uint8, device=DEV)

    def run(off):
        place = lambda t, name: shifted(t, off[name]) if off.get(name) else t
        dx = place(torch.full((T, d), 7.0, device=DEV), "dx")
        dw = place(torch.full((E, d), 7.0, device=DEV), "dw")
        db = torch.empty(E, device=DEV)
        B.moe_route_backward(shape, place(x, "x"), place(w, "w"), logits, ids, dg, None, dx=dx,
                             dw_router=dw, db_router=db, dx_add=place(add, "add"), token_mask=mask,
                             ws=ws)
        return dx, dw, db

    want = run({})
    for n in (1, 2, 3):
        for off in [{name: n} for name in ("x", "w", "dx", "add", "dw")] + [
                dict(x=n, w=n, dx=n, add=n, dw=n)]:
            assert all(torch.equal(a, b) for a, b in zip(run(off), want)), off


def test_logits_past_32_bit_offsets():
    """T x E past 2^31 elements: one block of tokens repeated.  Every repeat's gradients are the same
    bits, and dx those of the block alone; counts are multiples; the sums over tokens are within
    fp32 chains of at most T / 128 additions (blocks, waves and lanes share the tokens)."""
    Tb, reps, E, k, d = 65537, 129, 256, 2, 8
    T = Tb * reps
    assert T * E > 2 ** 31
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    say(f"[large logits] T={T} E={E}")
    x, w, logits, ids, dg, _ = router_inputs(Tb, d, E, k, torch.float32)
    chain = T / 128 * R.U
    small = L.balance_loss(logits, ids, coef=1.0)
    big_lg, big_ids = logits.repeat(reps, 1), ids.repeat(reps, 1)
    big = L.balance_loss(big_lg, big_ids, coef=1.0)
    assert torch.equal(big["counts"], small["counts"] * reps)
    assert abs(float(big["loss"]) - float(small["loss"])) <= 2 * chain * float(small["loss"])
    blocks = big["dlogits"].view(reps, Tb, E)
    assert all(torch.equal(blocks[i], blocks[0]) for i in range(1, reps))
    assert torch.isfinite(blocks[0]).all() and bool((blocks[0] != 0).any())
    del big, blocks
    say("[large logits] route backward")
    dlg = torch.randn(Tb, E, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV)
    one = L.route_backward(x, w, logits, ids, dg, dlg)
    big_dlg = dlg.repeat(reps, 1)
    many = L.route_backward(x.repeat(reps, 1), w, big_lg, big_ids, dg.repeat(reps, 1), big_dlg)
    dx = many["dx"].view(reps, Tb, d)
    assert all(torch.equal(dx[i], one["dx"]) for i in range(reps))
    del many, big_lg
    sums = L.route_backward(x.repeat(reps, 1), w, None, None, None, big_dlg)
    dw = reps * (dlg.double().T @ x.double())
    db = reps * dlg.double().sum(0)
    assert bool(((sums["dw_router"].double() - dw).abs() <=
                 chain * reps * (dlg.double().abs().T @ x.double().abs())).all())
    assert bool(((sums["db_router"].double() - db).abs() <= chain * reps * dlg.double().abs().sum(0)).all())
    del big_dlg, sums
    torch.cuda.empty_cache()


def test_activation_past_32_bit_offsets():
    """kept rows x d_ff past 2^31 elements: every repeat of a block of tokens gives the same bits,
    within the layer's tolerance of the oracle on the dequantised weights."""
    Tb, reps, d, f, E, k = 64, 2188, 64, 4096, 8, 4
    T = Tb * reps
    assert T * k * f > 2 ** 31
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB of free device memory")
    say(f"[large activation] T={T} rows={T * k} d_ff={f}")
    inp = W.make_shape_inputs(Tb, d, f, E, "bf16", seed=1, router_bias_std=1.0)
    dev = L.upload(inp, DEV)
    experts = L.quantize_experts(dev["w1"], dev["b1"], dev["w2"], dev["b2"], 64)
    dev["x"] = dev["x"].repeat(reps, 1)
    out = L.layer_forward_quantized(dev, experts, k, T)["out"].view(reps, Tb, d)
    assert bool((out == out[0]).all())
    f64 = lambda a: W.to_float64(a, "bf16")
    w1, w2 = (Q.dequantize(*Q.quantize(f64(inp[n]), 64), 64) for n in ("w1", "w2"))
    ref = O.forward(f64(inp["x"]), f64(inp["w_router"]), inp["b_router"], w1, f64(inp["b1"]), w2,
                    f64(inp["b2"]), k, float(E))
    assert P.max_abs_rel(P.to_np(out[0]), ref["out"]) <= P.TOL["bf16"]
    del out
    torch.cuda.empty_cache()


def test_calls_on_two_streams_at_once():
    """Router training on one stream beside the 4-bit products on another, each with its own
    workspace, many times: the bits of the calls one after another."""
    T, d, f, E, k = 3000, 256, 512, 64, 4
    x, w, logits, ids, dg, mask = router_inputs(T, d, E, k)
    inp = W.make_shape_inputs(200, d, f, E, "bf16", seed=3, router_bias_std=1.0)
    dev = L.upload(inp, DEV)
    experts = L.quantize_experts(dev["w1"], dev["b1"], dev["w2"], dev["b2"], 32)

    def train():
        b = L.balance_loss(logits, ids, token_mask=mask)
        g = L.route_backward(x, w, logits, ids, dg, b["dlogits"], token_mask=mask)
        return [b["loss"], b["counts"], b["dlogits"], g["dx"], g["dw_router"], g["db_router"]]

    def serve():
        return [L.layer_forward_quantized(dev, experts, k, 100)["out"]]

    want_t, want_s = train(), serve()
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    one.wait_stream(torch.cuda.current_stream())
    two.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(10):
        with torch.cuda.stream(one):
            got.append((train(), want_t))
        with torch.cuda.stream(two):
            got.append((serve(), want_s))
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("T,E", [(300, 256), (20000, 64)])
def test_graphs_share_a_workspace(T, E):
    """Balance loss and router backward, each in a graph of its own over one workspace, replayed in
    turn with new logits and with eager calls on the same workspace between them."""
    k, d = 2, 128
    x, w, logits, ids, dg, mask = router_inputs(T, d, E, k)
    shape = B.make_shape(T, d, 8, E, k, 0, B.MOE_BF16)
    ws = torch.empty(max(B.workspace_bytes_balance(shape), B.workspace_bytes_route_backward(shape)),
                     dtype=torch.uint8, device=DEV)
    a = L.balance_loss(logits, ids, ws=ws)
    L.route_backward(x, w, logits, ids, dg, a["dlogits"], ws=ws)
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        bal = L.balance_loss(logits, ids, token_mask=mask, ws=ws)
    with torch.cuda.graph(second):
        back = L.route_backward(x, w, logits, ids, dg, bal["dlogits"], token_mask=mask, ws=ws)
    gen = torch.Generator(device=DEV).manual_seed(8)
    for turn in range(4):
        logits.copy_(torch.randn(T, E, generator=gen, device=DEV))
        ids.copy_(logits.topk(k, dim=1).indices)
        first.replay()
        second.replay()
        if turn % 2:
            second.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*bal.values(), *back.values())]
        want_b = L.balance_loss(logits, ids, token_mask=mask, ws=ws)
        want_r = L.route_backward(x, w, logits, ids, dg, want_b["dlogits"], token_mask=mask, ws=ws)
        want = [*want_b.values(), *want_r.values()]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), turn


def test_timing_arms_cover_the_quantized_calls():
    T, d, f, E, k = 64, 256, 512, 8, 2
    dev = L.upload(W.make_shape_inputs(T, d, f, E, "bf16", seed=0, router_bias_std=1.0), DEV)
    experts = L.quantize_experts(dev["w1"], dev["b1"], dev["w2"], dev["b2"], 32)
    plain = L.layer_forward_quantized(dev, experts, k, T)["out"]
    ev = lambda: [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    gemm, stage = ev(), ev()
    for e in gemm + stage:
        e.record()
    B.moe_set_gemm_timing(gemm)
    B.moe_set_stage_timing(stage)
    timed = L.layer_forward_quantized(dev, experts, k, T)["out"]
    torch.cuda.synchronize()
    assert torch.equal(timed, plain)
    assert all(0 < e[i].elapsed_time(e[i + 1]) < 1000 for e in (gemm, stage) for i in (0, 2))
    shape = B.make_shape(T, d, f, E, k, T, B.MOE_BF16)
    r = L.route(dev, k, T)
    disp = L.dispatch(shape, r["ids"], r["gates"])
    B.moe_set_gemm_timing(gemm)
    L.expert_ffn_quantized(shape, dev["x"], experts, disp["row_token"], disp["offsets"])
    torch.cuda.synchronize()
    assert all(0 < gemm[i].elapsed_time(gemm[i + 1]) < 1000 for i in (0, 2))


@pytest.mark.parametrize("T,cap", [(0, 4), (16, 0)])
def test_layer_without_rows(T, cap):
    """No tokens: nothing is written.  No slot: every token drops and is passed on as it is."""
    d, f, E, k = 64, 96, 8, 2
    dev = L.upload(W.make_shape_inputs(16, d, f, E, "bf16", seed=0, router_bias_std=1.0), DEV)
    experts = L.quantize_experts(dev["w1"], dev["b1"], dev["w2"], dev["b2"], 32)
    dev["x"] = dev["x"][:T].contiguous()
    res = L.layer_forward_quantized(dev, experts, k, cap)
    plain = L.layer_forward(dev, k, cap)
    assert res["out"].shape == (T, d)
    assert torch.equal(res["out"], plain["out"])
    if T:
        assert bool(res["drop_mask"].all())
