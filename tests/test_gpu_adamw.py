"""The AdamW step over many tensors against the formula: moments to the bit, params within their
roundings; 8-bit codes to the code."""
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
HALF16 = 2.0 ** -8  # half a step of bf16, relative


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    B.lib()
    yield
    torch.cuda.synchronize()


HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8)
LENGTHS = [1, 3, 255, 256, 257, 0, 1000, 4096, 4097, 20011, 64]


def place(t, off):
    """A copy of t on the device, `off` elements past an aligned address."""
    flat = torch.zeros(t.numel() + off + 8, dtype=t.dtype, device=DEV)
    out = flat[off:off + t.numel()]
    out.copy_(t.flatten())
    return out


class Case:
    """Tensors of the given lengths with moments of earlier steps."""

    def __init__(self, lengths, bits, param="f32", grad="f32", copy=False, off=0, seed=0, fresh=False):
        rng = np.random.default_rng(seed)
        pdt = torch.bfloat16 if param == "bf16" else torch.float32
        gdt = torch.bfloat16 if grad == "bf16" else torch.float32
        self.bits, self.pdt = bits, pdt
        self.p, self.g, self.m, self.v, self.ms, self.vs, self.copy = ([] for _ in range(7))
        for n in lengths:
            size = np.exp(2 * rng.normal(size=n))
            f = lambda a: torch.from_numpy(np.asarray(a, np.float32))
            self.p.append(place(f(rng.normal(size=n)).to(pdt), off))
            self.g.append(place(f(1e-2 * rng.normal(size=n) * size).to(gdt), off))
            m, r = f(1e-3 * rng.normal(size=n) * size), f(1e-2 * rng.random(n) * size)
            if fresh:
                m, r = torch.zeros(n), torch.zeros(n)
            if bits == 32:
                self.m.append(place(m, off))
                self.v.append(place(r * r, off))
            else:
                for x, top, codes, steps in ((m, 127, self.m, self.ms), (r, 255, self.v, self.vs)):
                    c, s = S.encode(x.numpy(), top)
                    codes.append(place(torch.from_numpy(c), off))
                    steps.append(place(torch.from_numpy(s), off))
            if copy:
                self.copy.append(place(torch.full((n,), 7.0, dtype=torch.bfloat16), off))
        self.wd = [0.1 * (i % 3) for i in range(len(lengths))]
        self.tensors = B.AdamWTensors(self.p, self.g, self.m, self.v, m_steps=self.ms if bits == 8 else None,
                                      v_steps=self.vs if bits == 8 else None,
                                      copies=self.copy if copy else None, weight_decay=self.wd)

    def host(self, i):
        """p, g, m, v of tensor i as fp32 arrays."""
        f = lambda t: t.float().cpu().numpy()
        if self.bits == 32:
            return f(self.p[i]), f(self.g[i]), f(self.m[i]), f(self.v[i])
        r = S.decode(self.v[i].cpu().numpy(), self.vs[i].cpu().numpy())
        with np.errstate(all="ignore"):
            return f(self.p[i]), f(self.g[i]), S.decode(self.m[i].cpu().numpy(), self.ms[i].cpu().numpy()), r * r

    def expect(self, step, grad_scale=1.0, **hyper):
        h = {**HYPER, **hyper}
        return [S.adamw(*self.host(i), h["lr"], h["beta1"], h["beta2"], h["eps"], step, self.wd[i], grad_scale)
                for i in range(len(self.p))]

    def check(self, want):
        for i, (p, bound, m, v) in enumerate(want):
            if len(p) == 0:
                continue
            got = self.p[i].double().cpu().numpy()
            tol = bound + (HALF16 * np.abs(p) if self.pdt == torch.bfloat16 else 0)
            assert np.all(np.abs(got - p) <= tol), i
            if self.copy:
                exact = self.p[i].to(torch.bfloat16)
                assert torch.equal(self.copy[i], exact), i
            if self.bits == 32:
                assert np.array_equal(self.m[i].cpu().numpy(), m) and np.array_equal(self.v[i].cpu().numpy(), v), i
            else:
                for x, top, codes, steps in ((m, 127, self.m[i], self.ms[i]),
                                             (np.sqrt(v), 255, self.v[i], self.vs[i])):
                    c, s = S.encode(x, top)
                    assert np.array_equal(steps.cpu().numpy(), s), i
                    assert np.array_equal(codes.cpu().numpy(), c), i


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,copy", [("f32", "f32", True), ("f32", "bf16", False), ("bf16", "bf16", False),
                                             ("bf16", "f32", False)])
@pytest.mark.parametrize("off", [0, 1])
def test_adamw(bits, param, grad, copy, off):
    """Off their alignment, bf16 arrays lie on 2 bytes, codes on 1, the rest on 4."""
    say(f"[adamw] bits={bits} param={param} grad={grad} off={off}")
    c = Case(LENGTHS, bits, param, grad, copy, off, seed=bits)
    for step in (7, 8):
        want = c.expect(step, grad_scale=0.25)
        B.moe_adamw_step(c.tensors, step=step, grad_scale=0.25, **HYPER)
        c.check(want)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(bits):
    """Over the 48 that one launch takes, empty ones between."""
    c = Case([(37 * i) % 700 for i in range(150)], bits, seed=5)
    want = c.expect(3)
    B.moe_adamw_step(c.tensors, step=3, **HYPER)
    c.check(want)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("hyper", [dict(beta1=0.0, beta2=0.0), dict(beta1=0.0), dict(lr=0.0), dict(eps=1.0),
                                   dict(beta2=0.999)])
def test_first_step_and_ends_of_the_betas(bits, hyper):
    c = Case([5, 256, 1025], bits, seed=2, fresh=True)
    want = c.expect(1, **hyper)
    B.moe_adamw_step(c.tensors, step=1, **{**HYPER, **hyper})
    c.check(want)


@pytest.mark.parametrize("bits", [32, 8])
def test_far_steps(bits):
    c = Case([1025], bits, seed=2)
    for step in (1000, 10 ** 6, 2 ** 40):
        want = c.expect(step)
        B.moe_adamw_step(c.tensors, step=step, **HYPER)
        c.check(want)


def test_blocks_of_zeros_and_single_values():
    """Gradients that leave a block's moments zero, one value in a block, and values whose block step
    is a denormal number or zero."""
    c = Case([256 * 6], 8, seed=3, fresh=True)
    g = torch.zeros(6, 256)
    g[1, 17], g[2, 0], g[2, 1] = 3.0, 1e30, 1e-30  # beside 1e30 the other code is the least
    g[3, 5], g[4, 9], g[5] = 1e-33, 1e-42, 1e-18
    c.g[0].copy_(g.flatten())
    want = c.expect(1)
    B.moe_adamw_step(c.tensors, step=1, **HYPER)
    c.check(want)
    v = c.v[0].view(6, 256).cpu()
    # 1e30 squared is past fp32, so that block has no finite root; 1e-33 and 1e-42 squared are 0
    assert int(v[0].max()) == 0 and v[1, 17] == 255 and int(v[2].max()) <= 1 and int(v[3:5].max()) == 0
    assert bool((v[5] == 255).all())


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_codes_at_their_borders(seed):
    """Values within a few steps of fp32 of the border between two codes, where the kernel's short way
    must not decide: with betas of 0, m is the gradient and v its square."""
    rng = np.random.default_rng(seed)
    blocks = []
    for top in (127, 255):
        for _ in range(400):
            s = np.exp(rng.uniform(-25, 15))  # the squares stay normal numbers
            c = rng.integers(0, top, 256)
            x = ((c + 0.5) ** 2 * s).astype(np.float32)
            x = (x.view(np.int32) + rng.integers(-6, 7, 256).astype(np.int32)).view(np.float32)
            x[rng.integers(256)] = np.float32(top * top * s)
            blocks.append(x * np.where(rng.random(256) < 0.5, -1, 1).astype(np.float32))
    g = torch.from_numpy(np.concatenate(blocks).astype(np.float32))
    c = Case([g.numel()], 8, seed=3, fresh=True)
    c.g[0].copy_(g)
    want = c.expect(1, beta1=0.0, beta2=0.0)
    B.moe_adamw_step(c.tensors, step=1, **{**HYPER, "beta1": 0.0, "beta2": 0.0})
    c.check(want)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite(bits, bad):
    """32 bits: the element alone.  8 bits: its block has no finite moment left, the params of the step
    itself are only off where the gradient was; the other blocks and tensors go on."""
    c = Case([1024, 300], bits, seed=4)
    c.g[0][300] = bad
    want = c.expect(2)
    B.moe_adamw_step(c.tensors, step=2, **HYPER)
    p = c.p[0].cpu()
    assert not np.isfinite(p[300]) and int(torch.isfinite(p).sum()) == 1023
    m, v = [torch.empty(1024, device=DEV), torch.empty(300, device=DEV)], [torch.empty(1024, device=DEV),
                                                                         torch.empty(300, device=DEV)]
    B.moe_adamw_moments(c.tensors, m, v)
    for out in (m, v):
        fine = torch.isfinite(out[0].cpu())
        if bits == 32:
            assert not fine[300] and int(fine.sum()) == 1023
        else:
            assert not fine[256:512].any() and fine[:256].all() and fine[512:].all()
        assert bool(torch.isfinite(out[1]).all())
    keep = np.r_[0:300, 301:1024]
    got = p.double().numpy()
    assert np.all(np.abs(got - want[0][0])[keep] <= want[0][1][keep])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("off", [0, 1])
def test_moments(bits, off):
    c = Case(LENGTHS, bits, off=off, seed=6)
    m, v = ([place(torch.full((n,), 7.0), off) for n in LENGTHS] for _ in range(2))
    B.moe_adamw_moments(c.tensors, m, v)
    for i in range(len(LENGTHS)):
        _, _, want_m, want_v = c.host(i)
        assert np.array_equal(m[i].cpu().numpy(), want_m) and np.array_equal(v[i].cpu().numpy(), want_v)
    only = [None] * len(LENGTHS)
    only[3] = torch.empty(LENGTHS[3], device=DEV)
    B.moe_adamw_moments(c.tensors, None, only)
    assert torch.equal(only[3], v[3])


@pytest.mark.parametrize("bits", [32, 8])
def test_dynamic(bits):
    """lr, grad_scale and step from the device; skip leaves everything as it is."""
    c = Case(LENGTHS, bits, copy=True, seed=7)
    dyn = torch.tensor([1e-3, 0.5, 9.0, 0.0], device=DEV)
    want = c.expect(9, grad_scale=0.5, lr=1e-3)
    B.moe_adamw_step(c.tensors, lr=99.0, beta1=0.9, beta2=0.99, eps=1e-8, step=0, dynamic=dyn)
    c.check(want)
    before = [t.clone() for t in c.p + c.m + c.v + c.ms + c.vs + c.copy]
    dyn[3] = 1.0
    B.moe_adamw_step(c.tensors, lr=99.0, beta1=0.9, beta2=0.99, eps=1e-8, step=0, dynamic=dyn)
    assert all(torch.equal(a, b) for a, b in zip(before, c.p + c.m + c.v + c.ms + c.vs + c.copy))
    dyn[2:] = torch.tensor([-3.0, 0.0])  # counts as the first step
    want = c.expect(1, grad_scale=0.5, lr=1e-3)
    B.moe_adamw_step(c.tensors, lr=99.0, beta1=0.9, beta2=0.99, eps=1e-8, step=0, dynamic=dyn)
    c.check(want)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_go_on_counting(bits):
    """A graph of the step and of its counter, replayed with eager work between, against eager steps."""
    a, b = Case(LENGTHS, bits, copy=True, seed=8), Case(LENGTHS, bits, copy=True, seed=8)
    dyn = torch.tensor([2e-3, 1.0, 0.0, 0.0], device=DEV)
    kw = dict(lr=0.0, beta1=0.9, beta2=0.99, eps=1e-8, step=0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        graph.capture_begin()
        dyn[2:3].add_(1.0)
        B.moe_adamw_step(a.tensors, dynamic=dyn, **kw)
        graph.capture_end()
    torch.cuda.current_stream().wait_stream(s)
    assert float(dyn[2]) == 0.0
    other = torch.zeros(4, device=DEV)
    for step in range(1, 5):
        for x, y in zip(a.g, b.g):  # new gradients in the same buffers
            x.mul_(0.9)
            y.mul_(0.9)
        graph.replay()
        other.copy_(torch.tensor([2e-3, 1.0, float(step), 0.0]))
        B.moe_adamw_step(b.tensors, dynamic=other, **kw)
        torch.cuda.synchronize()
        for x, y in zip(a.p + a.m + a.v + a.ms + a.vs + a.copy, b.p + b.m + b.v + b.ms + b.vs + b.copy):
            assert torch.equal(x, y), step


def test_set_grads_and_refused_lists():
    c = Case([300, 256], 32, seed=9)
    new = [torch.randn(300, device=DEV).bfloat16(), torch.randn(256, device=DEV).bfloat16()]
    c.tensors.set_grads(new)
    c.g = new
    want = c.expect(2)
    B.moe_adamw_step(c.tensors, step=2, **HYPER)
    c.check(want)
    p = torch.zeros(256, device=DEV)
    z = lambda: torch.zeros(256, device=DEV)
    with pytest.raises(B.MoeError, match="overlaps"):
        B.AdamWTensors([p, p], [z(), z()], [z(), z()], [z(), z()])
    with pytest.raises(ValueError, match="holds 255 elements, the shape needs 256"):
        B.AdamWTensors([p], [z()[:255]], [z()], [z()])
    with pytest.raises(ValueError, match="257 elements, 256 are expected"):
        B.AdamWTensors([p], [torch.zeros(257, device=DEV)], [z()], [z()])
    with pytest.raises(ValueError, match="contiguous"):
        B.AdamWTensors([torch.zeros(256, 2, device=DEV)[:, 0]], [z()], [z()], [z()])


def test_gradients_in_other_storage():
    """A gradient tensor whose storage was exchanged is taken where it lies now."""
    p = torch.zeros(512, device=DEV)
    opt = L.AdamW([p], lr=0.5, betas=(0.0, 0.0), weight_decay=0.0)
    g = torch.ones(512, device=DEV)
    opt.step([g])
    assert bool((p + 0.5).abs().max() < 1e-6)
    g.data = torch.full((512,), -1.0, device=DEV)
    opt.step([g])
    assert bool(p.abs().max() < 1e-6)
    m, v = opt.moments()
    assert torch.equal(m[0], g) and torch.equal(v[0], g * g)


def test_params_and_copies_are_taken_where_they_lie():
    """So are a param and a copy; what they held before stays as it was left."""
    p, c = torch.zeros(512, device=DEV), torch.zeros(512, dtype=torch.bfloat16, device=DEV)
    opt = L.AdamW([p], lr=0.5, betas=(0.0, 0.0), weight_decay=0.0, copies=[c])
    g = torch.ones(512, device=DEV)
    opt.step([g])
    old = [p.data, c.data]
    left = [t.clone() for t in old]
    p.data = torch.full((512,), 8.0, device=DEV)
    opt.step([g])
    assert bool((p - 7.5).abs().max() < 1e-5) and bool((c == 7.5).all())
    assert torch.equal(old[0], left[0])
    left[1].copy_(c)
    c.data = torch.zeros_like(c)
    opt.step([g])
    assert bool((p - 7.0).abs().max() < 1e-5) and bool((c == 7.0).all())
    assert torch.equal(old[1], left[1]) and opt.steps == 3


def test_another_stream():
    c, d = Case([100000], 8, seed=10), Case([100000], 8, seed=10)
    B.moe_adamw_step(c.tensors, step=1, **HYPER)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        B.moe_adamw_step(d.tensors, step=1, **HYPER)
    B.moe_adamw_step(d.tensors, step=2, stream=s, **HYPER)
    B.moe_adamw_step(c.tensors, step=2, **HYPER)
    torch.cuda.synchronize()
    for x, y in zip(c.p + c.m + c.v, d.p + d.m + d.v):
        assert torch.equal(x, y)


def test_past_32_bit_offsets():
    """More than 2^31 elements: the last ones are those of a short tensor with the same values."""
    n, tail = 2 ** 31 + 4096 + 300, 4096 + 300
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    say("[adamw] 2^31 elements")
    for bits in (8, 32):
        small = Case([tail], bits, "bf16", "bf16", seed=11)
        big = {}
        for name, src, count in (("p", small.p, n), ("g", small.g, n), ("m", small.m, n), ("v", small.v, n)):
            big[name] = torch.zeros(count, dtype=src[0].dtype, device=DEV)
            big[name][-tail:] = src[0]
        steps = {}
        if bits == 8:
            for name, src in (("m_steps", small.ms), ("v_steps", small.vs)):
                steps[name] = [torch.zeros((n + 255) // 256, device=DEV)]
                steps[name][0][-src[0].numel():] = src[0]
        t = B.AdamWTensors([big["p"]], [big["g"]], [big["m"]], [big["v"]], **steps)
        B.moe_adamw_step(t, step=3, **HYPER)
        B.moe_adamw_step(small.tensors, step=3, **HYPER)
        for name, src in (("p", small.p), ("m", small.m), ("v", small.v)):
            assert torch.equal(big[name][-tail:], src[0]), (bits, name)
            assert not bool(big[name][:4096].any())
        del big, steps, t
