"""Routing by scores, its backward pass, the bias update and the combine's backward pass against fp64
references, on the sizes, masks and values where they can go wrong."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

import scored_ref as S
from capacity_routing_expert_amd import binding as B

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


def dtype_of(name):
    return (torch.bfloat16, B.MOE_BF16) if name == "bf16" else (torch.float32, B.MOE_F32)


def make(T, d, E, dtype, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    dt, _ = dtype_of(dtype)
    x = torch.randn(T, d, generator=g).to(dt)
    w = (spread * torch.randn(E, d, generator=g) / d ** 0.5).to(dt)
    return x, w, 0.5 * torch.randn(E, generator=g), 0.2 * torch.randn(E, generator=g)


def run(x, w, b, k, bias=None, mask=None, want_logits=True, ws=None, **routing):
    T, d = x.shape
    E = w.shape[0]
    shape = B.make_shape(T, d, 8, E, k, 0, B.MOE_BF16 if x.dtype == torch.bfloat16 else B.MOE_F32)
    dev = lambda t: None if t is None else t.to(DEV)
    ids = torch.full((T, k), 77, dtype=torch.int32, device=DEV)
    gates = torch.full((T, k), 77.0, device=DEV)
    logits = torch.full((T, E), 77.0, device=DEV) if want_logits else None
    if ws is None:
        ws = torch.empty(max(B.workspace_bytes_route_scored(shape), 256), dtype=torch.uint8, device=DEV)
    B.moe_route_scored(shape, B.make_routing(**routing), dev(x), dev(w), dev(b), dev(bias), ids, gates,
                       logits=logits, token_mask=dev(mask), ws=ws)
    return ids.cpu().numpy(), gates.double().cpu().numpy(), (
        logits.double().cpu().numpy() if want_logits else None)


def logits_ref(x, w, b):
    """fp64 logits, and how far another order of the sums can be off: d 2^-53 of the sum of the terms'
    sizes, twice."""
    x, w = x.double().numpy(), w.double().numpy()
    z, size = x @ w.T, np.abs(x) @ np.abs(w).T
    if b is not None:
        z, size = z + b.double().numpy(), size + np.abs(b.double().numpy())
    return z, 2 * (x.shape[1] + 2) * 2.0 ** -53 * size


def check_gates(got, ref, noise):
    """One rounding to fp32 and the fp64 noise of the logits (which a gate takes over relatively)."""
    tol = np.abs(ref) * (U + 4 * noise + 1e-14) + 2.0 ** -150
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.all((np.abs(got - ref) <= tol) | np.isnan(ref))


ROUTES = [
    # T, d, E, k, dtype, routing
    (1, 8, 1, 1, "bf16", dict()),
    (1, 2048, 64, 6, "bf16", dict(renormalize=True)),
    (3, 24, 2, 2, "bf16", dict(score="sigmoid", renormalize=True, scale=2.5)),
    (17, 40, 5, 3, "f32", dict(score="sigmoid")),
    (16, 7, 8, 8, "f32", dict(renormalize=True, scale=0.5)),
    (33, 1000, 16, 4, "f32", dict(n_groups=4, topk_groups=2, group_score="top2")),
    (130, 72, 17, 17, "bf16", dict(score="sigmoid", renormalize=True)),
    (63, 264, 33, 2, "bf16", dict(n_groups=11, topk_groups=3)),
    (64, 2048, 256, 8, "bf16", dict(score="sigmoid", n_groups=8, topk_groups=4, group_score="top2",
                                    renormalize=True, scale=2.5)),
    (37, 136, 96, 5, "f32", dict(n_groups=6, topk_groups=2)),
    (50, 64, 130, 30, "bf16", dict(score="sigmoid", n_groups=2, topk_groups=1)),
    (20, 64, 256, 256, "bf16", dict(score="sigmoid", renormalize=True)),
    (20, 64, 256, 200, "f32", dict(n_groups=256, topk_groups=200, group_score="top2")),
    (4096, 64, 8, 2, "bf16", dict(renormalize=True)),
    (4099, 72, 24, 3, "bf16", dict(score="sigmoid", n_groups=8, topk_groups=3, renormalize=True)),
    (4097, 33, 60, 4, "f32", dict(n_groups=3, topk_groups=2, group_score="top2")),
    (4100, 40, 100, 4, "bf16", dict(score="sigmoid")),
    (8200, 16, 64, 6, "bf16", dict(n_groups=8, topk_groups=3, group_score="top2", renormalize=True)),
    (8193, 24, 39, 39, "bf16", dict(score="sigmoid", n_groups=3, topk_groups=3, renormalize=True)),
    # large tiles of 16 and 32 experts, with and without splits, whose last one holds 16 experts or fewer
    (40001, 520, 12, 2, "bf16", dict(renormalize=True)),
    (40003, 136, 15, 3, "f32", dict(score="sigmoid", n_groups=5, topk_groups=2)),
    (40003, 270, 28, 4, "f32", dict(score="sigmoid", renormalize=True)),
    (4300, 1032, 33, 2, "bf16", dict(n_groups=11, topk_groups=4, group_score="top2")),
    (9001, 264, 64, 6, "bf16", dict(score="sigmoid", n_groups=8, topk_groups=4, group_score="top2")),
    (9000, 268, 72, 4, "f32", dict(renormalize=True)),
    (9001, 264, 80, 8, "bf16", dict(score="sigmoid", renormalize=True, scale=2.5)),
    (5000, 801, 100, 4, "f32", dict(n_groups=5, topk_groups=3)),
    # logits of more than 64 MiB: the tokens in two parts
    (34001, 16, 250, 5, "f32", dict(n_groups=10, topk_groups=3)),
]


@pytest.mark.parametrize("T,d,E,k,dtype,routing", ROUTES)
@pytest.mark.parametrize("biased,masked", [(False, False), (True, True)])
def test_route_scored(T, d, E, k, dtype, routing, biased, masked):
    say(f"[route scored] T={T} d={d} E={E} k={k} {dtype} {routing}")
    x, w, b, bias = make(T, d, E, dtype, seed=T + E)
    bias = bias if biased else None
    mask = (torch.rand(T, generator=torch.Generator().manual_seed(T)) < 0.7).to(torch.uint8) if masked else None
    z, noise = logits_ref(x, w, b)
    ids, gates, logits = run(x, w, b, k, bias=bias, mask=mask, **routing)
    m = None if mask is None else mask.numpy()
    want_ids, want = S.route(z, k, score_bias=None if bias is None else bias.numpy(), token_mask=m, **routing)
    assert np.array_equal(ids, want_ids)
    check_gates(gates, want, noise.max())
    if m is not None:
        z[m == 0], noise[m == 0] = 0.0, 0.0
    assert np.all(np.abs(logits - z) <= U * np.abs(z) + noise)
    if T <= 4096:
        again = run(x, w, None if b is None else b, k, bias=bias, mask=mask, want_logits=False, **routing)
        assert np.array_equal(again[0], ids) and np.array_equal(again[1], gates)


@pytest.mark.parametrize("T,d,E,k,dtype", [(1, 64, 8, 2, "bf16"), (300, 200, 5, 3, "f32"),
                                           (515, 128, 64, 6, "bf16"), (4500, 64, 200, 8, "bf16")])
def test_plain_softmax_is_moe_route(T, d, E, k, dtype):
    """Softmax, one group, no bias, no renormalising: moe_route's ids, and its gates and logits but for
    sums whose order differs (a last bit in rare cases)."""
    x, w, b, _ = make(T, d, E, dtype, seed=3)
    ids, gates, logits = run(x, w, b, k)
    shape = B.make_shape(T, d, 8, E, k, 0, dtype_of(dtype)[1])
    i2 = torch.empty(T, k, dtype=torch.int32, device=DEV)
    g2, l2 = torch.empty(T, k, device=DEV), torch.empty(T, E, device=DEV)
    ws = torch.empty(B.workspace_bytes(shape) + 256, dtype=torch.uint8, device=DEV)
    B.moe_route(shape, x.to(DEV), w.to(DEV), b.to(DEV), i2, g2, l2, ws)
    assert np.array_equal(ids, i2.cpu().numpy())
    assert np.all(np.abs(gates - g2.double().cpu().numpy()) <= 2 * U * gates)
    assert np.all(np.abs(logits - l2.double().cpu().numpy()) <= 2 * U * np.abs(logits))


def exact_logits(z):
    """x, W_r of width E whose logits are the values of z [T, E] (representable in bf16 or fp32)."""
    T, E = z.shape
    return z.clone(), torch.eye(E)


def run_logits(z, k, **kw):
    x, w = exact_logits(z)
    return run(x, w, None, k, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [dict(), dict(n_groups=4, topk_groups=2),
                                    dict(n_groups=4, topk_groups=2, group_score="top2"),
                                    dict(n_groups=12, topk_groups=7, group_score="top2")])
def test_ties_go_to_the_lower_group_and_expert(score, groups):
    g = torch.Generator().manual_seed(5)
    z = torch.randint(-1, 2, (40, 12), generator=g).float()  # three values: ties everywhere
    bias = torch.randint(0, 2, (12,), generator=g).float() * 0.25
    ids, gates, _ = run_logits(z, 5, score=score, bias=bias, renormalize=True, **groups)
    want, ref = S.route(z.double().numpy(), 5, score=score, renormalize=True, score_bias=bias.numpy(), **groups)
    assert np.array_equal(ids, want)
    check_gates(gates, ref, 0.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("off", [(0,), (3, 4, 5), (0, 1, 2, 3, 4, 5, 6, 7, 9), tuple(range(12))])
def test_experts_that_are_off(score, group_score, off):
    """-inf in the bias: never chosen, no share of a group's score; -1 where experts run out."""
    z = torch.randn(30, 12, generator=torch.Generator().manual_seed(7))
    bias = torch.zeros(12)
    bias[list(off)] = -float("inf")
    for kw in (dict(), dict(n_groups=4, topk_groups=2, group_score=group_score),
               dict(n_groups=12, topk_groups=6, group_score=group_score)):
        ids, gates, _ = run_logits(z, 6, score=score, bias=bias, renormalize=True, **kw)
        want, ref = S.route(z.double().numpy(), 6, score=score, renormalize=True, score_bias=bias.numpy(), **kw)
        assert np.array_equal(ids, want), kw
        check_gates(gates, ref, 0.0)
        assert not np.isin(ids, off).any() and np.all(gates[ids < 0] == 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_extreme_logits(score, renormalize):
    """Logits past the ends of exp in fp32 and fp64, -inf, and rows of nothing else."""
    low, inf = -3.4028234663852886e38, float("inf")
    z = torch.tensor([[0, -100, -200, -300, -800, low], [-800, -801, -900, -1000, -5000, low],
                      [low] * 6, [-inf] * 6, [-inf, 3, -inf, 2, -inf, -inf], [800, 799, 0, -800, 700, low],
                      [-700, -701, -740, -750, -760, -inf], [-90, -104, -110, -120, -inf, -91]])
    # one term a logit, so that no sum mixes infinities: x is the row itself times 1, through fp32
    # (an infinite x times a zero weight would be NaN, so the logits come in through the bias)
    for t in range(len(z)):
        x, w = torch.zeros(1, 4), torch.zeros(6, 4)
        ids, gates, logits = run(x, w, z[t].clone(), 4, score=score, renormalize=renormalize)
        want, ref = S.route(z[t:t + 1].double().numpy(), 4, score=score, renormalize=renormalize)
        assert np.array_equal(ids, want), t
        check_gates(gates, ref, 1e-13)  # exp of arguments of some hundred, in fp64
        assert np.array_equal(logits[0], z[t].double().numpy())


def test_gates_where_all_chosen_scores_are_lost():
    """A bias that steers a softmax to experts 1000 below the row's largest: the ratios survive."""
    z = torch.tensor([[0.0, -1000.0, -1001.0, -2000.0]])
    bias = torch.tensor([-5.0, 0.0, 0.0, 0.0])
    ids, gates, _ = run_logits(z, 2, bias=bias, renormalize=True)
    r = 1 / (1 + np.exp(-1.0))
    assert ids.tolist() == [[1, 2]] and np.allclose(gates, [[r, 1 - r]], rtol=1e-7)
    bias = torch.tensor([-5.0, -5.0, -5.0, 0.0])
    ids, gates, _ = run_logits(z, 2, bias=bias, renormalize=True)
    assert ids.tolist() == [[3, 0]] and gates.tolist() == [[0.0, 1.0]]  # e^-2000 beside e^0


def test_nan():
    """NaN scores and biases are chosen first and reach the gates of their token alone."""
    z = torch.randn(5, 8, generator=torch.Generator().manual_seed(2))
    x, w = exact_logits(z)
    x[1, 3] = float("nan")  # the whole row of logits
    for score in ("softmax", "sigmoid"):
        ids, gates, _ = run(x, w, None, 3, score=score)
        zn = z.double().numpy().copy()
        zn[1] = np.nan
        want, ref = S.route(zn, 3, score=score)
        assert np.array_equal(ids, want) and np.isnan(gates[1]).all()
        check_gates(gates, ref, 0.0)
    bias = torch.zeros(8)
    bias[6] = float("nan")
    for kw in (dict(), dict(n_groups=4, topk_groups=1, group_score="top2")):
        ids, gates, _ = run(*exact_logits(z), None, 2, bias=bias, score="sigmoid", **kw)
        want, ref = S.route(z.double().numpy(), 2, score="sigmoid", score_bias=bias.numpy(), **kw)
        assert np.array_equal(ids, want) and np.all(ids[:, 0] == 6)
        check_gates(gates, ref, 0.0)
    # one expert's NaN bias in b_router: only sigmoid keeps it to that expert
    b = torch.zeros(8)
    b[2] = float("nan")
    ids, gates, _ = run(*exact_logits(z), b, 3, score="sigmoid")
    assert np.all(ids[:, 0] == 2) and np.isnan(gates[:, 0]).all() and np.isfinite(gates[:, 1:]).all()


def test_masked_tokens_are_not_looked_at():
    x, w, b, bias = make(50, 64, 16, "bf16", seed=9)
    mask = torch.ones(50, dtype=torch.uint8)
    mask[::3] = 0
    clean = run(x, w, b, 4, bias=bias, mask=mask, renormalize=True)
    x[::3] = float("nan")
    dirty = run(x, w, b, 4, bias=bias, mask=mask, renormalize=True)
    for a, c in zip(clean, dirty):
        assert np.array_equal(a, c)
    assert np.all(clean[0][::3] == -1) and np.all(clean[1][::3] == 0) and np.all(clean[2][::3] == 0)
    none = run(x, w, b, 4, mask=torch.zeros(50, dtype=torch.uint8))
    assert np.all(none[0] == -1) and np.all(none[1] == 0)


@pytest.mark.parametrize("T,d,E", [(70, 72, 20), (4200, 36, 40), (33, 35, 9)])
def test_f32_arrays_on_4_bytes(T, d, E):
    """fp32 x, W_r and the other arrays off 16 bytes give the bits of the aligned call."""
    x, w, b, bias = [t.to(DEV) for t in make(T, d, E, "f32", seed=8)]
    shape, r = B.make_shape(T, d, 8, E, 3, 0, B.MOE_F32), B.make_routing("sigmoid", renormalize=True)
    mask = (torch.arange(T, device=DEV) % 5 > 0).to(torch.uint8)
    ws = torch.empty(B.workspace_bytes_route_scored(shape), dtype=torch.uint8, device=DEV)
    outs = []
    for n in range(4):
        o = [shifted(torch.full((T, 3), 7, dtype=torch.int32, device=DEV), n),
             shifted(torch.full((T, 3), 7.0, device=DEV), n), shifted(torch.full((T, E), 7.0, device=DEV), n)]
        B.moe_route_scored(shape, r, shifted(x, n), shifted(w, n), shifted(b, n), shifted(bias, n), o[0], o[1],
                           logits=o[2], token_mask=shifted(mask, n), ws=ws)
        outs.append(o)
    z, noise = logits_ref(x.cpu(), w.cpu(), b.cpu())
    z[mask.cpu().numpy() == 0] = 0.0
    assert np.all(np.abs(outs[0][2].double().cpu().numpy() - z) <= U * np.abs(z) + noise)
    assert all(torch.equal(p, q) for o in outs[1:] for p, q in zip(o, outs[0]))


def test_more_tokens_than_a_chunk():
    """The workspace bounds how many tokens go through at a time; past that, chunks."""
    T, E, d, k = 40000, 256, 8, 8
    x, w, b, bias = make(T, d, E, "bf16", seed=4)
    shape = B.make_shape(T, d, 8, E, k, 0, B.MOE_BF16)
    need = B.workspace_bytes_route_scored(shape)
    assert need < T * E * 8  # several chunks
    ws = torch.full((need + 4096,), 7, dtype=torch.uint8, device=DEV)
    ids, gates, logits = run(x, w, b, k, bias=bias, ws=ws, score="sigmoid", n_groups=8, topk_groups=3)
    assert bool((ws[need:] == 7).all())
    pick = np.r_[0:20, T // 2:T // 2 + 20, 32760:32780, T - 20:T]
    z, noise = logits_ref(x, w, b)
    want, ref = S.route(z[pick], k, score="sigmoid", n_groups=8, topk_groups=3, score_bias=bias.numpy())
    assert np.array_equal(ids[pick], want)
    check_gates(gates[pick], ref, noise.max())
    assert np.all(np.abs(logits - z) <= U * np.abs(z) + noise)


def test_logits_past_32_bit_offsets():
    """T x E past 2^31: one block of tokens repeated gives the same bits everywhere."""
    Tb, reps, E, d, k = 65536, 129, 256, 8, 2
    T = Tb * reps
    assert T * E > 2 ** 31
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    say(f"[route scored, long] T={T}")
    x, w, b, bias = make(Tb, d, E, "bf16", seed=6)
    r = B.make_routing("sigmoid", 8, 4, "top2", True)
    xs, w, b, bias = x.to(DEV).repeat(reps, 1), w.to(DEV), b.to(DEV), bias.to(DEV)
    shape = B.make_shape(T, d, 8, E, k, 0, B.MOE_BF16)
    ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
    gates, logits = torch.empty(T, k, device=DEV), torch.empty(T, E, device=DEV)
    ws = torch.empty(B.workspace_bytes_route_scored(shape), dtype=torch.uint8, device=DEV)
    B.moe_route_scored(shape, r, xs, w, b, bias, ids, gates, logits=logits, ws=ws)
    for t in (ids, gates, logits):
        v = t.view(reps, Tb, -1)
        assert all(torch.equal(v[i], v[0]) for i in range(1, reps))
    z, noise = logits_ref(x[:64], w.cpu(), b.cpu())
    assert np.all(np.abs(logits[:64].double().cpu().numpy() - z) <= U * np.abs(z) + noise)
    say("[route scored backward, long]")
    dg = torch.randn(Tb, k, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).repeat(reps, 1)
    for renormalize in (False, True):
        r = B.make_routing("softmax", renormalize=renormalize)
        dl = torch.full_like(logits, 7.0)
        B.moe_route_scored_backward(shape, r, logits, ids, dg, dl)
        v = dl.view(reps, Tb, E)
        assert all(torch.equal(v[i], v[0]) for i in range(1, reps))
        ref, bound = S.route_backward(logits[:64].double().cpu().numpy(), ids[:64].cpu().numpy(),
                                      dg[:64].double().cpu().numpy(), "softmax", renormalize, 1.0)
        assert np.all(np.abs(v[0, :64].double().cpu().numpy() - ref) <= bound)


# ---------------------------------------------------------------- backward
def back(z, ids, dg, score, renormalize, scale, add=None, mask=None, out=None):
    T, E = z.shape
    shape = B.make_shape(T, 8, 8, E, ids.shape[1], 0, B.MOE_F32)
    out = torch.full((T, E), 77.0, device=DEV) if out is None else out
    B.moe_route_scored_backward(shape, B.make_routing(score, renormalize=renormalize, scale=scale), z, ids,
                                dg, out, dlogits_add=add, token_mask=mask)
    return out


def back_inputs(T, E, k, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    z = 3 * torch.randn(T, E, generator=g, device=DEV)
    ids = torch.topk(torch.rand(T, E, generator=g, device=DEV), k, dim=1).indices.to(torch.int32).contiguous()
    return (z, ids, torch.randn(T, k, generator=g, device=DEV), torch.randn(T, E, generator=g, device=DEV),
            (torch.rand(T, generator=g, device=DEV) < 0.7).to(torch.uint8))


def shifted(t, n=1):
    flat = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
    out = flat[n:].view(t.shape)
    out.copy_(t)
    return out


def compare(got, z, ids, dg, score, renormalize, scale, add=None, mask=None):
    n = lambda t: None if t is None else t.double().cpu().numpy()
    ref, bound = S.route_backward(n(z), ids.cpu().numpy(), n(dg), score, renormalize, scale, n(add),
                                  None if mask is None else mask.cpu().numpy())
    got = got.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= bound), float(np.max(np.abs(got - ref) - bound))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (37, 5, 2), (5, 4, 4), (33, 8, 2), (40, 16, 3), (31, 32, 32),
                                   (65, 64, 6), (30, 66, 20), (20, 128, 17), (18, 130, 8), (17, 256, 8),
                                   (9, 256, 256), (9, 255, 40)])
def test_backward(score, renormalize, T, E, k):
    say(f"[scored backward] {score} renorm={renormalize} T={T} E={E} k={k}")
    z, ids, dg, add, mask = back_inputs(T, E, k, seed=E)
    compare(back(z, ids, dg, score, renormalize, 2.5), z, ids, dg, score, renormalize, 2.5)
    got = back(z, ids, dg, score, renormalize, 0.5, add, mask)
    compare(got, z, ids, dg, score, renormalize, 0.5, add, mask)
    assert bool((got[mask == 0] == 0).all())
    inplace = add.clone()
    assert torch.equal(back(z, ids, dg, score, renormalize, 0.5, inplace, mask, inplace), got)
    # off 16 bytes: other pieces, the same sums in another order for a whole softmax row
    off = back(shifted(z), shifted(ids), shifted(dg), score, renormalize, 0.5, shifted(add), shifted(mask),
               shifted(add))
    compare(off, z, ids, dg, score, renormalize, 0.5, add, mask)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_backward_of_odd_choices(score, renormalize):
    """No choice (-1, E, a large number), a choice twice or all the same, a token without any."""
    z, ids, dg, _, _ = back_inputs(20, 12, 4, seed=1)
    ids[0, 1], ids[1, 2], ids[2, 0] = -1, 12, 2 ** 31 - 1
    ids[3, 1] = ids[3, 0]
    ids[4] = 7
    ids[5] = -1
    dg[0, 1] = float("nan")  # of no choice: not looked at
    got = back(z, ids, dg, score, renormalize, 1.5)
    clean = dg.clone()
    clean[0, 1] = 0.0
    compare(got, z, ids, clean, score, renormalize, 1.5)
    assert bool((got[5] == 0).all())
    assert torch.equal(back(z, ids, dg, score, renormalize, 1.5), got)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("E,k", [(96, 6), (100, 16), (256, 8), (256, 17), (131, 5)])
def test_backward_of_experts_held_twice(score, renormalize, E, k):
    """Among many experts: tokens that hold one twice, three times or only one beside tokens that do not,
    and choices that are none."""
    z, ids, dg, add, _ = back_inputs(70, E, k, seed=E + k)
    for t in range(0, 70, 3):
        ids[t, 1:1 + t % 4] = ids[t, 0]
    ids[6] = ids[6, 0]
    ids[7, 2], ids[8] = -1, -1
    got = back(z, ids, dg, score, renormalize, 1.5, add)
    compare(got, z, ids, dg, score, renormalize, 1.5, add)
    assert torch.equal(back(z, ids, dg, score, renormalize, 1.5, add), got)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_at_the_ends_of_fp32(score):
    """Renormalised gates of scores that fp32 loses still have their gradients; rows whose chosen
    scores are all zero have none."""
    inf = float("inf")
    z = torch.tensor([[-200.0, -201, -203, 5, 0, 0], [-3e38, -3e38, -3e38, 0, 0, 0], [-inf, -inf, -inf, 0, 0, 0],
                      [-inf, 1, 2, 0, 0, 0], [300, 299, -300, 0, 0, 0], [88, -88, 104, 0, 0, 0]], device=DEV)
    ids = torch.tensor([[0, 1, 2]] * 6, dtype=torch.int32, device=DEV)
    dg = torch.tensor([[1.0, -2.0, 0.5]] * 6, device=DEV)
    got = back(z, ids, dg, score, True, 2.0)
    compare(got, z, ids, dg, score, True, 2.0)
    assert bool((got[2] == 0).all()) and bool((got[0, :3] != 0).all() if score == "softmax" else True)
    got = back(z, ids, dg, score, False, 2.0)
    assert bool(torch.isfinite(got).all())
    compare(got[[0, 1, 3, 4, 5]], z[[0, 1, 3, 4, 5]], ids[:5], dg[:5], score, False, 2.0)


def test_backward_nan():
    z, ids, dg, _, _ = back_inputs(6, 8, 2, seed=3)
    z[1, ids[1, 0].long()] = float("nan")
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            got = back(z, ids, dg, score, renormalize, 1.0)
            assert bool(torch.isnan(got[1]).any()) and bool(torch.isfinite(got[[0, 2, 3, 4, 5]]).all())


# ---------------------------------------------------------------- bias
@pytest.mark.parametrize("T,E,k", [(0, 4, 2), (1, 1, 1), (64, 8, 2), (700, 33, 5), (4100, 256, 4), (32771, 256, 8),
                                   (9000, 7, 7)])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_bias(T, E, k, masked):
    say(f"[bias] T={T} E={E} k={k} masked={masked}")
    rng = np.random.default_rng(T + E)
    ids = rng.integers(-1, E + 1, (T, k)).astype(np.int32)
    mask = (rng.random(T) < 0.6).astype(np.uint8) if masked else None
    bias = rng.normal(size=E).astype(np.float32)
    bias[rng.random(E) < 0.1] = -np.inf
    want, counts = S.balance_bias(ids, E, 0.01, bias, mask)
    shape = B.make_shape(T, 8, 8, E, k, 0, B.MOE_F32)
    ws = torch.empty(max(B.workspace_bytes_balance_bias(shape), 256), dtype=torch.uint8, device=DEV)
    b, c = torch.from_numpy(bias).to(DEV), torch.full((E,), 7, dtype=torch.int32, device=DEV)
    m = None if mask is None else torch.from_numpy(mask).to(DEV)
    B.moe_balance_bias(shape, 0.01, b, c, topk_ids=torch.from_numpy(ids).to(DEV), token_mask=m, ws=ws)
    assert np.array_equal(c.cpu().numpy(), counts) and np.array_equal(b.cpu().numpy(), want)
    b2 = torch.from_numpy(bias).to(DEV)  # the same counts given: other batches' may be in them
    B.moe_balance_bias(shape, 0.01, b2, c)
    assert torch.equal(b, b2) and np.array_equal(c.cpu().numpy(), counts)
    b3 = torch.from_numpy(bias).to(DEV)
    B.moe_balance_bias(shape, 0.01, b3, topk_ids=torch.from_numpy(ids).to(DEV), token_mask=m, ws=ws)
    assert torch.equal(b, b3)


def test_balance_bias_large_counts_and_ties():
    shape = B.make_shape(0, 8, 8, 4, 1, 0, B.MOE_F32)
    big = 2 ** 31 - 1
    for counts, signs in (([big] * 4, [0] * 4), ([big, big, big, big - 1], [-1, -1, -1, 1]), ([0] * 4, [0] * 4)):
        b = torch.tensor([0.5, -0.5, float("nan"), 1e30], device=DEV)
        c = torch.tensor(counts, dtype=torch.int32, device=DEV)
        want = b + 0.25 * torch.tensor(signs, device=DEV, dtype=torch.float32)
        B.moe_balance_bias(shape, 0.25, b, c)
        assert torch.equal(b.nan_to_num(9.0), want.nan_to_num(9.0))


# ---------------------------------------------------------------- combine
@pytest.mark.parametrize("T,d,E,k,dtype", [(1, 8, 1, 1, "bf16"), (5, 16, 4, 2, "bf16"), (37, 520, 5, 3, "bf16"),
                                           (64, 2048, 8, 2, "bf16"), (130, 1032, 16, 6, "bf16"),
                                           (9, 64, 64, 33, "bf16"), (7, 1, 3, 2, "f32"), (33, 65, 5, 5, "f32"),
                                           (40, 260, 8, 2, "f32"), (12, 2048, 12, 9, "f32")])
def test_combine_backward(T, d, E, k, dtype):
    say(f"[combine backward] T={T} d={d} E={E} k={k} {dtype}")
    dt, code = dtype_of(dtype)
    g = torch.Generator().manual_seed(d)
    capacity = max(1, T * k // E)
    rows = min(T * k, E * capacity)
    slots = torch.full((T * k,), -1, dtype=torch.int32)
    n = max(1, rows - rows // 8)  # some rows that no slot names
    slots[torch.randperm(T * k, generator=g)[:n]] = torch.randperm(rows, generator=g)[:n].to(torch.int32)
    slots = slots.view(T, k)
    dout, y = torch.randn(T, d, generator=g).to(dt), torch.randn(rows, d, generator=g).to(dt)
    gates = torch.rand(T, k, generator=g)
    gates[slots < 0] = float("nan")  # of no kept choice: not looked at
    shape = B.make_shape(T, d, 8, E, k, capacity, code)
    dev = lambda t: t.to(DEV)
    for off in (0, 1) if dtype == "f32" else (0,):
        place = lambda t: shifted(dev(t), off) if off else dev(t)
        dg = torch.full((T, k), 77.0, device=DEV)
        dy = place(torch.full((rows, d), 77.0).to(dt))
        args = (shape, place(dout), dev(gates), dev(slots), place(y))
        B.moe_combine_backward(*args, dgates=dg, dy_rows=dy)
        D, Y, kept = dout.double(), y.double(), slots >= 0
        at = slots.clamp(min=0).long()
        want = (Y[at] * D.unsqueeze(1)).sum(2) * kept
        # a lane adds d / 64 terms (fused), the wave 6 more times: at most d / 64 + 14 roundings
        size = (Y[at].abs() * D.abs().unsqueeze(1)).sum(2) * kept
        assert bool(((dg.cpu().double() - want).abs() <= (d / 64 + 14) * U * size).all())
        assert bool((dg.cpu()[~kept] == 0).all())
        ref = torch.full((rows, d), 77.0, dtype=torch.float64)
        ref[slots[kept].long()] = (gates.double().unsqueeze(2) * D.unsqueeze(1))[kept]
        half = U if dtype == "f32" else 2.0 ** -8 + U
        assert bool(((dy.cpu().double() - ref).abs() <= half * ref.abs()).all())
        one, two = torch.empty_like(dg), torch.full_like(dy, 77.0)
        B.moe_combine_backward(*args, dgates=one)
        B.moe_combine_backward(args[0], args[1], args[2], args[3], None, dy_rows=two)
        assert torch.equal(one, dg) and torch.equal(two, dy)
        inplace = args[4].clone() if not off else shifted(args[4])
        unnamed = torch.ones(rows, dtype=torch.bool)
        unnamed[slots[kept].long()] = False
        B.moe_combine_backward(args[0], args[1], args[2], args[3], inplace, dgates=one, dy_rows=inplace)
        assert torch.equal(one, dg)
        assert torch.equal(inplace[(~unnamed).to(DEV)], dy[(~unnamed).to(DEV)])
        assert torch.equal(inplace[unnamed.to(DEV)], args[4][unnamed.to(DEV)])


def test_combine_backward_against_differences():
    """The combine itself, moved along each gate: it is linear in them."""
    T, d, E, k = 6, 64, 4, 2
    g = torch.Generator(device=DEV).manual_seed(3)
    x, y = torch.randn(T, d, generator=g, device=DEV), torch.randn(T * k, d, generator=g, device=DEV)
    dout = torch.randn(T, d, generator=g, device=DEV)
    gates = torch.rand(T, k, generator=g, device=DEV)
    slots = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).view(T, k)
    slots[2, 1] = -1
    shape = B.make_shape(T, d, 8, E, k, T * k, B.MOE_F32)
    dg = torch.empty(T, k, device=DEV)
    B.moe_combine_backward(shape, dout, gates, slots, y, dgates=dg)
    for c in range(k):
        up, down, out = gates.clone(), gates.clone(), torch.empty(2, T, d, device=DEV)
        up[:, c] += 0.5
        down[:, c] -= 0.5
        B.moe_combine(shape, x, up, slots, y, out[0])
        B.moe_combine(shape, x, down, slots, y, out[1])
        diff = ((out[0].double() - out[1].double()) * dout.double()).sum(1)
        # each out is three roundings of terms below |x| + 2 |y| off
        tol = 8 * U * ((x.abs() + 2 * y[slots[:, c].clamp(min=0).long()].abs() + 2 * y.abs().max()).double() *
                       dout.abs().double()).sum(1)
        assert bool(((diff - dg[:, c].double()).abs() <= tol).all())
