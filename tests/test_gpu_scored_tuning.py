"""Routing by scores, its gradients, the bias update and AdamW together, as a router is tuned over
frozen experts: one training step's gradients against fp64, captured graphs, streams."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

import scored_ref as S
from capacity_routing_expert_amd import binding as B
from capacity_routing_expert_amd import layer as L

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = S.U


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    B.lib()
    yield
    torch.cuda.synchronize()


def layer(T=96, d=64, f=64, E=16, dtype=torch.float32, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    return dict(x=r(T, d).to(dtype), w_router=(r(E, d) / d ** 0.5).to(dtype), b_router=0.1 * r(E),
                w1=(r(E, f, d) / d ** 0.5).to(dtype), b1=(0.1 * r(E, f)).to(dtype),
                w2=(r(E, d, f) / f ** 0.5).to(dtype), b2=(0.1 * r(E, d)).to(dtype)), r(T, d).to(dtype)


@pytest.mark.parametrize("score,renormalize", [("sigmoid", True), ("sigmoid", False), ("softmax", True),
                                               ("softmax", False)])
def test_gradient_of_a_training_step(score, renormalize):
    """dW_r and db_r of sum(dout * out) through combine, gates and router, in fp32 experts, against
    autograd in fp64 with the choice and the kept slots as constants."""
    k, E = 3, 16
    dev, dout = layer()
    T, d = dev["x"].shape
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)
    mask[-9:] = 0
    routing = B.make_routing(score, n_groups=4, topk_groups=2, group_score="top2", renormalize=renormalize,
                             scale=1.5)
    bias = 0.2 * torch.randn(E, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    fwd = L.layer_forward_scored(dev, k, 20, routing, bias, mask)
    assert bool((fwd["slot_of"][-9:] == -1).all()) and bool((fwd["out"][-9:] == dev["x"][-9:]).all())
    assert bool((fwd["slot_of"][:-9] == -1).any())  # some dropped
    dg = L.combine_backward(fwd["shape"], dout, fwd["gates"], fwd["slot_of"], fwd["y_rows"])["dgates"]
    dl = L.route_scored_backward(fwd["logits"], fwd["ids"], dg, routing, token_mask=mask)
    grad = L.route_backward(dev["x"], dev["w_router"], None, None, dlogits=dl)

    c = lambda t: t.double().cpu()
    w, b = c(dev["w_router"]).requires_grad_(), c(dev["b_router"]).requires_grad_()
    ids, slots = fwd["ids"].cpu().long(), fwd["slot_of"].cpu().long()
    z = c(dev["x"]) @ w.t() + b
    s = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1)
    g = torch.where(ids >= 0, s.gather(1, ids.clamp(min=0)), 0.0)
    if renormalize:
        g = g / g.sum(1, keepdim=True).clamp(min=1e-300)
    g = 1.5 * g
    y = c(fwd["y_rows"])[slots.clamp(min=0)] * (slots >= 0).unsqueeze(2)
    loss = ((g.unsqueeze(2) * y).sum(1) * c(dout)).sum()
    loss.backward()
    # dgates are d / 64 + 14 roundings off, dlogits E + k + 40 (both of terms of their size), the sums
    # over tokens 97; the logits that the kernels take are rounded, which moves a score by U |l| at most
    size_dg = ((y.abs() * c(dout).abs().unsqueeze(1)).sum(2)).numpy()
    lg = fwd["logits"].double().cpu().numpy()
    _, size = S.route_backward(lg, fwd["ids"].cpu().numpy(), size_dg, score, renormalize, 1.5)
    per_logit = size / (E + k + 40) * (E + k + 40 + d / 64 + 14 + T + 4 * np.abs(lg).max())
    # The reference cancels by itself where an entry is zero by the formula (a softmax's experts that
    # were not chosen): it leaves k + E roundings of 2^-53 of the two sums, each at most 1.5 sum |dg|,
    # doubled for the products within them.
    per_logit = per_logit + (k + E) * 2.0 ** -53 * 2 * 2 * 1.5 * size_dg.sum(1, keepdims=True)
    tol_w = per_logit.T @ np.abs(c(dev["x"]).numpy())
    assert np.all(np.abs(c(grad["dw_router"]).numpy() - w.grad.numpy()) <= tol_w)
    assert np.all(np.abs(c(grad["db_router"]).numpy() - b.grad.numpy()) <= per_logit.sum(0))
    assert float(w.grad.abs().max()) > 10 * tol_w.max()


def test_router_tuned_over_quantized_experts():
    """Steps of the whole loop with 4-bit experts, a bf16 copy of the router and 8-bit moments run, stay
    finite, and the bias moves against the load."""
    dev, dout = layer(T=256, d=128, f=128, E=16, dtype=torch.bfloat16, seed=4)
    experts = L.quantize_experts(dev["w1"], dev["b1"], dev["w2"], dev["b2"])
    routing = B.make_routing("sigmoid", n_groups=4, topk_groups=2, group_score="top2", renormalize=True)
    master = [dev["w_router"].float(), dev["b_router"].clone()]
    opt = L.AdamW(master, lr=1e-3, state_bits=8, copies=[dev["w_router"], None], weight_decay=[0.1, 0.0])
    dev["b_router"] = master[1]
    bias = torch.zeros(16, device=DEV)
    for step in range(3):
        before = [bias.clone()] + [p.clone() for p in master]
        fwd = L.layer_forward_scored(dev, 4, 80, routing, bias, experts=experts)
        g = L.combine_backward(fwd["shape"], dout, fwd["gates"], fwd["slot_of"], fwd["y_rows"], want_rows=True)
        bal = L.balance_loss(fwd["logits"], fwd["ids"], coef=0.01)
        dl = L.route_scored_backward(fwd["logits"], fwd["ids"], g["dgates"], routing, dlogits_add=bal["dlogits"])
        grad = L.route_backward(dev["x"], dev["w_router"], None, None, dlogits=dl, dx_add=dout)
        opt.step([grad["dw_router"], grad["db_router"]])
        counts = L.balance_bias(fwd["ids"], bias, 0.01)
        assert torch.equal(counts, bal["counts"])
        mean = counts.double().mean()
        assert torch.equal(torch.sign(bias - before[0]).double(), torch.sign(mean - counts.double()))
        assert torch.equal(dev["w_router"], master[0].to(torch.bfloat16))
        for p, old in zip(master, before[1:]):
            assert bool(torch.isfinite(p).all()) and bool((p != old).any())
        assert bool(torch.isfinite(grad["dx"].float()).all())
        kept = fwd["slot_of"] >= 0
        assert bool((g["dy_rows"][fwd["slot_of"][kept].long()] != 0).any(1).all())
    m, v = opt.moments()
    assert all(bool(torch.isfinite(t).all()) and bool((t != 0).any()) for t in m + v)


class Step:
    """One training step of a router on buffers of its own (a shared workspace, if given)."""

    def __init__(self, seed, ws=None, T=200, d=64, E=64, k=6):
        dev, self.dout = layer(T, d, 8, E, torch.bfloat16, seed)
        self.x, self.b, self.k, self.E = dev["x"], dev["b_router"], k, E
        self.master = [dev["w_router"].float()]
        self.w = dev["w_router"]
        self.routing = B.make_routing("sigmoid", 8, 4, "top2", True, 2.5)
        self.bias = torch.zeros(E, device=DEV)
        self.shape = B.make_shape(T, d, 8, E, k, T, B.MOE_BF16)
        self.ws = torch.empty(self.need(self.shape), dtype=torch.uint8, device=DEV) if ws is None else ws
        e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=DEV)
        self.ids, self.gates, self.logits = e(T, k, dt=torch.int32), e(T, k), e(T, E)
        self.dg, self.dl, self.dw, self.counts = e(T, k), e(T, E), e(E, d), e(E, dt=torch.int32)
        self.y = torch.randn(T * k, d, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).bfloat16()
        self.slots = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k)
        z = lambda dt, n: [torch.zeros(n, dtype=dt, device=DEV)]
        n = E * d
        self.m, self.v, self.ms, self.vs = (z(torch.int8, n), z(torch.uint8, n), z(torch.float32, n // 256),
                                            z(torch.float32, n // 256))
        self.opt = B.AdamWTensors(self.master, [self.dw], self.m, self.v, self.ms, self.vs, copies=[self.w],
                                  weight_decay=0.1)
        self.dyn = torch.tensor([1e-3, 1.0, 0.0, 0.0], device=DEV)

    @staticmethod
    def need(shape):
        return max(B.workspace_bytes_route_scored(shape), B.workspace_bytes_route_backward(shape),
                   B.workspace_bytes_balance_bias(shape), 256)

    def run(self):
        B.moe_route_scored(self.shape, self.routing, self.x, self.w, self.b, self.bias, self.ids, self.gates,
                           logits=self.logits, ws=self.ws)
        B.moe_combine_backward(self.shape, self.dout, None, self.slots, self.y, dgates=self.dg)
        B.moe_route_scored_backward(self.shape, self.routing, self.logits, self.ids, self.dg, self.dl)
        B.moe_route_backward(self.shape, self.x, self.w, None, None, None, self.dl, dw_router=self.dw, ws=self.ws)
        self.dyn[2:3].add_(1.0)
        B.moe_adamw_step(self.opt, 0.0, 0.9, 0.99, 1e-8, 0, dynamic=self.dyn)
        B.moe_balance_bias(self.shape, 0.01, self.bias, self.counts, topk_ids=self.ids, ws=self.ws)

    def state(self):
        return [self.ids, self.gates, self.logits, self.dg, self.dl, self.dw, self.counts, self.bias, self.w,
                *self.master, *self.m, *self.v, *self.ms, *self.vs, self.dyn]


@pytest.mark.parametrize("T", [1, 200, 5000])
def test_captured_training_steps(T):
    """Two graphs that share a workspace, replayed in turn with eager work between, against eager
    steps."""
    say(f"[captured training step] T={T}")
    eager = [Step(1, T=T), Step(2, T=T)]
    ws = torch.empty(Step.need(eager[0].shape), dtype=torch.uint8, device=DEV)
    mine = [Step(1, ws, T=T), Step(2, ws, T=T)]
    graphs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for m in mine:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            g.capture_begin()
            m.run()
            g.capture_end()
        graphs.append(g)
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for e, m, g in zip(eager, mine, graphs):
            ws.fill_(0xA5)  # nothing in the workspace has to survive
            g.replay()
            e.run()
            torch.cuda.synchronize()
            for a, b in zip(e.state(), m.state()):
                assert torch.equal(a, b)


def test_streams_side_by_side():
    """Two steps on two streams with workspaces of their own give what they give alone."""
    alone, both = [Step(3, T=3000), Step(4, T=5000)], [Step(3, T=3000), Step(4, T=5000)]
    for a in alone:
        a.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for b, s in zip(both, streams):
        with torch.cuda.stream(s):
            b.run()
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y)


def test_equal_calls_give_equal_bits():
    for T in (37, 4500):
        a, b = Step(5, T=T), Step(5, T=T)
        a.run()
        b.run()
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y)


def test_empty_batch():
    s = B.make_shape(0, 64, 8, 16, 2, 0, B.MOE_BF16)
    e = lambda *n, dt=torch.float32: torch.empty(*n, dtype=dt, device=DEV)
    B.moe_route_scored(s, B.make_routing(), e(0, 64, dt=torch.bfloat16), e(16, 64, dt=torch.bfloat16), None, None,
                       e(0, 2, dt=torch.int32), e(0, 2))
    B.moe_route_scored_backward(s, B.make_routing(), e(0, 16), e(0, 2, dt=torch.int32), e(0, 2), e(0, 16))
    B.moe_combine_backward(s, e(0, 64, dt=torch.bfloat16), e(0, 2), e(0, 2, dt=torch.int32), None, dgates=e(1))
    bias, counts = torch.ones(16, device=DEV), torch.full((16,), 5, dtype=torch.int32, device=DEV)
    B.moe_balance_bias(s, 0.5, bias, counts, topk_ids=e(0, 2, dt=torch.int32))
    assert bool((counts == 0).all()) and bool((bias == 1).all())
    B.moe_adamw_step(B.AdamWTensors([], [], [], []), 0.1, 0.9, 0.99, 1e-8, 1)


def test_tensors_elsewhere_are_refused():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="must be on the GPU"):
        L.route_scored(x.to(DEV), torch.zeros(8, 64), None, 2, B.make_routing())
    t = B.AdamWTensors([torch.zeros(4, device=DEV)], [torch.zeros(4, device=DEV)], [torch.zeros(4, device=DEV)],
                       [torch.zeros(4, device=DEV)])
    with pytest.raises(ValueError, match="must be on the GPU"):
        B.moe_adamw_step(t, 0.1, 0.9, 0.99, 1e-8, 1, dynamic=torch.zeros(4))
