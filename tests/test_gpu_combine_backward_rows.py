"""Which rows the backward pass of the combine looks at."""
from __future__ import annotations

import pytest
import torch

import scored_ref as S
from capacity_routing_expert_amd import binding as B
from capacity_routing_expert_amd import layer as L

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    B.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_rows_without_capacity(dtype):
    """Capacity 0: no expert rows, so none is looked at, whatever slot_of holds."""
    T, d, E, k = 9, 40, 4, 3
    shape = B.make_shape(T, d, 8, E, k, 0, B.MOE_BF16 if dtype is torch.bfloat16 else B.MOE_F32)
    dout, gates = torch.ones(T, d, dtype=dtype, device=DEV), torch.rand(T, k, device=DEV)
    slots = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k)
    slots[1], slots[2] = -1, 2 ** 31 - 1
    for y in (None, torch.empty(0, d, dtype=dtype, device=DEV)):
        dg = torch.full((T, k), 7.0, device=DEV)
        B.moe_combine_backward(shape, dout, gates, slots, y, dgates=dg)
        assert not bool(dg.any())
    x = torch.randn(T, d, device=DEV).to(dtype)
    g = L.combine_backward(shape, x, gates, torch.full_like(slots, -1), torch.empty(0, d, dtype=dtype, device=DEV),
                           want_rows=True)
    assert not bool(g["dgates"].any()) and g["dy_rows"].numel() == 0


def check(dout, gates, slots, y, dg, dy, left):
    """Against fp64: dgates within the roundings of its sums, named rows within one of the dtype, the
    others as they were left."""
    T, d = dout.shape
    D, Y, at = dout.double(), y.double(), slots.clamp(min=0, max=len(y) - 1).long()
    kept = (slots >= 0) & (slots < len(y))
    want = (Y[at] * D.unsqueeze(1)).sum(2) * kept
    # a lane adds d / 64 terms (fused), the wave 6 more times: at most d / 64 + 14 roundings
    size = (Y[at].abs() * D.abs().unsqueeze(1)).sum(2) * kept
    assert bool(((dg.double() - want).abs() <= (d / 64 + 14) * S.U * size).all())
    ref = left.double()
    ref[slots[kept].long()] = (gates.double().unsqueeze(2) * D.unsqueeze(1))[kept]
    half = S.U if y.dtype is torch.float32 else 2.0 ** -8 + S.U
    assert bool(((dy.double() - ref).abs() <= half * ref.abs()).all())
    named = torch.zeros(len(y), dtype=torch.bool, device=DEV)
    named[slots[kept].long()] = True
    assert torch.equal(dy[~named], left[~named])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d,E,k,capacity", [(5, 64, 4, 2, 40), (64, 2048, 8, 2, 20), (130, 136, 16, 6, 33),
                                              (1, 8, 3, 1, 7)])
def test_padded_rows(dtype, T, d, E, k, capacity):
    """The padded layer's slots and rows: more rows than assignments, and fewer."""
    g = torch.Generator(device=DEV).manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dtype)
    dev = dict(x=r(T, d), w_router=r(E, d), b_router=r(E).float(), w1=r(E, 16, d) / d ** 0.5, b1=r(E, 16),
               w2=r(E, d, 16) / 4, b2=r(E, d))
    fwd = L.layer_forward_padded(dev, k, capacity)
    shape = L.shape_of(dev, k, capacity)
    slots, y, dout = fwd["slot_of"], fwd["y_rows"], r(T, d)
    assert len(y) == E * capacity
    if T * k < E * capacity:
        assert int(slots.max()) >= T * k  # past the compact layout's rows
    dg, dy = torch.full((T, k), 7.0, device=DEV), torch.full_like(y, 7.0)
    B.moe_combine_backward(shape, dout, fwd["gates"], slots, y, dgates=dg, dy_rows=dy)
    check(dout, fwd["gates"], slots, y, dg, dy, torch.full_like(y, 7.0))
    both = L.combine_backward(shape, dout, fwd["gates"], slots, y, want_rows=True)
    assert torch.equal(both["dgates"], dg)
    check(dout, fwd["gates"], slots, y, dg, both["dy_rows"], torch.zeros_like(y))
    inplace = y.clone()
    B.moe_combine_backward(shape, dout, fwd["gates"], slots, inplace, dgates=dg, dy_rows=inplace)
    check(dout, fwd["gates"], slots, y, dg, inplace, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_slots_past_the_rows(dtype):
    """Rows of a larger array: what lies before and behind those that are handed over is not touched,
    whatever slot_of holds; slots past them count as dropped."""
    T, d, E, k, n = 40, 72, 4, 3, 12
    shape = B.make_shape(T, d, 8, E, k, 3, B.MOE_BF16 if dtype is torch.bfloat16 else B.MOE_F32)  # 12 rows
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dtype)
    y, dy, dout, gates = r(3 * n, d), r(3 * n, d), r(T, d), torch.rand(T, k, generator=g, device=DEV)
    y[:n], y[2 * n:] = float("nan"), float("nan")
    before = dy.clone()
    slots = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).view(T, k) - 4
    slots[0, 0], slots[1, 1], slots[2, 2] = 2 ** 31 - 1, -2 ** 31, n + 1000
    slots[(slots == n + 1000) & (torch.arange(T * k, device=DEV).view(T, k) != 8)] = -1
    dg = torch.full((T, k), 7.0, device=DEV)
    B.moe_combine_backward(shape, dout, gates, slots, y[n:2 * n], dgates=dg, dy_rows=dy[n:2 * n])
    check(dout, gates, slots, y[n:2 * n], dg, dy[n:2 * n], before[n:2 * n])
    assert torch.equal(dy[:n], before[:n]) and torch.equal(dy[2 * n:], before[2 * n:])
    assert int(((slots >= 0) & (slots < n)).sum()) > 4


def test_rows_of_fewer_than_the_layout():
    """Buffers below the kept rows are refused; below the padded layout's, they bound the slots."""
    shape = B.make_shape(8, 64, 8, 4, 2, 10, B.MOE_F32)  # 16 rows compact, 40 padded
    z = lambda *s: torch.ones(*s, device=DEV)
    slots = torch.full((8, 2), 39, dtype=torch.int32, device=DEV)
    slots[1:] = -1
    slots[0, 1] = 15
    for n in (16, 39, 40, 50):
        dg = z(8, 2) * 7
        B.moe_combine_backward(shape, z(8, 64), None, slots, z(n, 64), dgates=dg)
        assert dg[0].tolist() == [64.0 if n >= 40 else 0.0, 64.0] and not bool(dg[1:].any())
    with pytest.raises(ValueError, match="y_rows holds"):
        B.moe_combine_backward(shape, z(8, 64), None, slots, z(15, 64), dgates=z(8, 2))
