"""What 8-bit moments keep of a gradient over many steps: the figures that the format's description
states, from the plain reference."""
import numpy as np
import pytest

import scored_ref as S

F = np.float32


@pytest.mark.parametrize("beta1,beta2,m_stays,r_stays", [(0.9, 0.95, 9, 39), (0.9, 0.999, 9, 255), (0.5, 0.5, 1, 3),
                                                         (0.99, 0.9999, 99, 255)])
def test_codes_that_do_not_decay(beta1, beta2, m_stays, r_stays):
    """Without a gradient, beside a largest value that stays, m's codes c with c (1 - sqrt(beta1)) <= 1/2
    and r's with c (1 - beta2^(1/4)) <= 1/2 return to themselves; the others fall."""
    assert m_stays == min(127, int(0.5 / (1 - beta1 ** 0.5))) and r_stays == min(255, int(0.5 / (1 - beta2 ** 0.25)))
    n = 256
    mc = np.arange(n).clip(0, 127).astype(np.int8)
    vc = np.arange(n).astype(np.uint8)
    mc[0] = 127
    vc[0] = 255
    ms, vs = np.array([2e-6], F), np.array([5e-7], F)
    m, r = S.decode(mc, ms), S.decode(vc, vs)
    g = np.zeros(n, F)
    g[0] = m[0]  # its m stays so; its v is put where it was
    _, _, m2, v2 = S.adamw(np.zeros(n, F), g, m, r * r, 1e-3, beta1, beta2, 1e-8, 100, 0.0)
    v2[0] = r[0] * r[0]
    m2c, m2s = S.encode(m2, 127)
    v2c, v2s = S.encode(np.sqrt(v2), 255)
    assert np.allclose(m2s, ms, rtol=1e-5) and np.allclose(v2s, vs, rtol=1e-5)
    stays_m, stays_v = m2c[1:] == mc[1:], v2c[1:] == vc[1:]
    assert np.array_equal(stays_m, mc[1:] <= m_stays) and np.array_equal(stays_v, vc[1:] <= r_stays)
    assert np.all(m2c[1:] <= mc[1:]) and np.all(v2c[1:] <= vc[1:])


def moved(bits, beta2):
    """How far a param goes after its gradient, 0.004 for 200 steps beside 255 of N(0, 1), has ended, in
    2000 further steps of lr 1e-3."""
    rng = np.random.default_rng(0)
    n, stop = 256, 128
    p, m, v = np.zeros(n, F), np.zeros(n, F), np.zeros(n, F)
    for t in range(1, 2201):
        g = rng.normal(size=n).astype(F)
        g[stop] = 0.004 if t <= 200 else 0.0
        new, _, m, v = S.adamw(p, g, m, v, 1e-3, 0.9, beta2, 1e-8, t, 0.0)
        p = new.astype(F)
        if bits == 8:
            m = S.decode(*S.encode(m, 127))
            r = S.decode(*S.encode(np.sqrt(v), 255))
            v = r * r
        if t == 200:
            left = p[stop]
    return abs(float(p[stop]) - float(left))


@pytest.mark.parametrize("beta2,at_32,at_8", [(0.95, 0.012, 0.47), (0.999, 0.009, 0.15)])
def test_params_that_move_without_a_gradient(beta2, at_32, at_8):
    assert moved(32, beta2) == pytest.approx(at_32, rel=0.05)
    assert moved(8, beta2) == pytest.approx(at_8, rel=0.05)


@pytest.mark.parametrize("beta2,mean", [(0.95, 0.011), (0.999, 0.052)])
def test_roots_of_steady_gradients(beta2, mean):
    """|r / r of fp32 - 1|, averaged over the blocks and over steps 201 to 4000."""
    rng = np.random.default_rng(1)
    n = 16 * 256
    size = np.exp(rng.uniform(-1, 1, n)).astype(F)
    v, v32, off = np.zeros(n, F), np.zeros(n, F), []
    b, c = F(beta2), F(1) - F(beta2)
    for t in range(1, 4001):
        g = rng.normal(size=n).astype(F) * size
        v, v32 = v * b + g * g * c, v32 * b + g * g * c
        r = S.decode(*S.encode(np.sqrt(v), 255))
        v = r * r
        if t > 200:
            off.append(np.abs(r / np.sqrt(v32) - 1).mean())
    assert np.mean(off) == pytest.approx(mean, rel=0.05)
