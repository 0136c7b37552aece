"""Which tensors a step of the AdamW class of layer.py takes, and what it refuses (no GPU: the addresses
are host tensors', and the step itself is recorded instead of launched)."""
import os

import pytest
import torch

from capacity_routing_expert_amd import binding as B
from capacity_routing_expert_amd import layer as L


@pytest.fixture
def steps(monkeypatch):
    """The entries that each step was called with; host tensors pass for the GPU's."""
    if not os.path.exists(B.LIB_PATH):
        from capacity_routing_expert_amd import build
        build.build()
    real, taken = B._ptr, []

    def ptr(t, name, dtype=None, device=None, numel=None):
        try:
            return real(t, name, dtype, device, numel)
        except ValueError as e:
            if "must be on the GPU" not in str(e):
                raise
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def step(tensors, *args, **kw):
        taken.append([dict(param=a.param, grad=a.grad, m=a.m, v=a.v, copy=a.copy, n=a.n, wd=a.weight_decay,
                           params=tensors.param_dtype, grads=tensors.grad_dtype)
                      for a in tensors.array[:tensors.n]])

    monkeypatch.setattr(B, "_ptr", ptr)
    monkeypatch.setattr(B, "moe_adamw_step", step)
    return taken


def make(copies=False, **kw):
    params = [torch.zeros(16, 16), torch.zeros(300)]
    return L.AdamW(params, copies=[torch.zeros(16, 16, dtype=torch.bfloat16), None] if copies else None,
                   **kw), [torch.ones(16, 16), torch.ones(300)]


# ways to look at a tensor's storage from the same address that a step must not take as before
VIEWS = {"transposed": lambda t: t.t(), "shorter": lambda t: t.flatten()[:100],
         "strided": lambda t: t.flatten()[::2],
         "retyped": lambda t: t.view(torch.int32 if t.element_size() == 4 else torch.int16)}


@pytest.mark.parametrize("view", sorted(VIEWS))
@pytest.mark.parametrize("which", ["param", "grad", "copy"])
def test_another_view_at_the_same_address(steps, view, which):
    opt, grads = make(copies=True)
    opt.step(grads)
    t = {"param": opt.params, "grad": grads, "copy": opt.copies}[which][0]
    before, at = t.data, t.data_ptr()
    t.data = VIEWS[view](before)
    assert t.data_ptr() == at
    with pytest.raises((ValueError, TypeError)):
        opt.step(grads)
    assert len(steps) == 1 and opt.steps == 1
    t.data = before
    opt.step(grads)
    assert steps[1] == steps[0] and opt.steps == 2


def test_gradients_of_another_type_at_the_same_address(steps):
    """As many bf16 gradients in the storage of the fp32 ones are taken as what they are."""
    opt, grads = make()
    opt.step(grads)
    for g in grads:
        g.data = g.data.flatten().view(torch.bfloat16)[:g.numel()]
    opt.step(grads)
    assert all(s["grads"] is torch.float32 for s in steps[0])
    assert all(s["grads"] is torch.bfloat16 for s in steps[1])
    assert [s["grad"] for s in steps[0]] == [s["grad"] for s in steps[1]]


def test_storage_that_was_exchanged(steps):
    opt, grads = make(copies=True)
    opt.step(grads)
    for t in (opt.params[1], grads[0], opt.copies[0]):
        t.data = t.data.clone()
    opt.step(grads)
    assert [s["param"] for s in steps[1]] == [p.data_ptr() for p in opt.params]
    assert [s["grad"] for s in steps[1]] == [g.data_ptr() for g in grads]
    assert [s["copy"] for s in steps[1]] == [opt.copies[0].data_ptr(), None]
    new = [g.clone() for g in grads]
    opt.step(new)
    assert [s["grad"] for s in steps[2]] == [g.data_ptr() for g in new]


def test_a_refused_step_leaves_no_address_behind(steps):
    """Gradients in a param's storage are refused; the next step takes those that are there then."""
    opt, grads = make()
    opt.step(grads)
    before = grads[0].data
    grads[0].data = opt.params[0].data
    with pytest.raises(B.MoeError, match="overlaps"):
        opt.step(grads)
    grads[0].data = before
    opt.step(grads)
    assert len(steps) == 2 and steps[1] == steps[0]


def test_refused_gradients_leave_the_list_as_it_was(steps):
    p, m, v = torch.zeros(300), torch.zeros(300), torch.zeros(300)
    g = torch.ones(300, dtype=torch.bfloat16)
    t = B.AdamWTensors([p, torch.zeros(4)], [g, torch.ones(4, dtype=torch.bfloat16)], [m, torch.zeros(4)],
                       [v, torch.zeros(4)])
    held = list(t.grads)
    for bad, error in (([v, torch.ones(4)], B.MoeError), ([torch.ones(300), torch.ones(3)], ValueError),
                       ([torch.ones(300), torch.ones(4).bfloat16()], TypeError), ([g], ValueError)):
        with pytest.raises(error):
            t.set_grads(bad)
        B.moe_adamw_step(t)
        assert [e["grad"] for e in steps[-1]] == [x.data_ptr() for x in held]
        assert steps[-1][0]["grads"] is torch.bfloat16
        assert all(x is y for x, y in zip(t.grads, held))


def test_weight_decay_that_was_changed(steps):
    """It takes effect at the next step, as lr, betas and eps do: a number, a list, an entry of it."""
    opt, grads = make(weight_decay=0.5)
    opt.step(grads)
    opt.weight_decay = 0.25
    opt.step(grads)
    opt.weight_decay = [0.125, 0.0]
    opt.step(grads)
    opt.weight_decay[1] = 1.0
    opt.step(grads)
    assert [[e["wd"] for e in s] for s in steps] == [[0.5, 0.5], [0.25, 0.25], [0.125, 0.0], [0.125, 1.0]]


@pytest.mark.parametrize("bits", [32, 8])
def test_a_state_that_was_put_in_place(steps, monkeypatch, bits):
    """Tensors put into m, v or the steps, one or all, are the state from then on, as before the first
    step; so are copies that are given later."""
    read = []
    monkeypatch.setattr(B, "moe_adamw_moments", lambda t, m, v: read.append([(a.m, a.v) for a in t.array[:t.n]]))
    opt, grads = make(state_bits=bits)
    opt.step(grads)
    opt.m[0] = opt.m[0].clone()
    opt.v = [t.clone() for t in opt.v]
    opt.m[1].data = opt.m[1].data.clone()
    if bits == 8:
        opt.m_steps[1] = opt.m_steps[1].clone()
    opt.moments()
    opt.step(grads)
    want = [(m.data_ptr(), v.data_ptr()) for m, v in zip(opt.m, opt.v)]
    assert read == [want] and [(e["m"], e["v"]) for e in steps[1]] == want
    if bits == 8:
        assert opt.tensors.array[1].m_steps == opt.m_steps[1].data_ptr()
    opt.copies = [torch.zeros(16, 16, dtype=torch.bfloat16), None]
    opt.step(grads)
    opt.copies = None
    opt.step(grads)
    assert [steps[i][0]["copy"] is None for i in range(4)] == [True, True, False, True]


def test_params_and_gradients_of_an_iterator(steps):
    params = [torch.zeros(4), torch.zeros(300)]
    opt = L.AdamW(iter(params), state_bits=8)
    assert [t.numel() for t in opt.v] == [4, 300] and [t.numel() for t in opt.v_steps] == [1, 2]
    for _ in range(2):
        opt.step(torch.ones_like(p) for p in params)
    assert [e["param"] for e in steps[1]] == [p.data_ptr() for p in params]
