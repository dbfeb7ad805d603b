"""Pins of the fp64 oracle of the gated linear attention operators."""
import itertools
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import gated


def case(seed=0, B=1, N=6, H=2, d=4):
    r = np.random.default_rng(seed)
    q, k, v = (r.standard_normal((B, N, H, d)) for _ in range(3))
    return q, k, v, -r.random((B, N, H)), r.standard_normal((B, H, d, d)), r


def test_single_token_in_closed_form():
    q, k, v, g, s0, _ = case(N=1)
    out, s1, _ = gated.forward(q, k, v, g, 0.5, s0)
    S = math.e ** g[0, 0, 1] * s0[0, 1] + np.outer(v[0, 0, 1], k[0, 0, 1])
    assert np.allclose(s1[0, 1], S, rtol=1e-14) and np.allclose(out[0, 0, 1], 0.5 * S @ q[0, 0, 1], rtol=1e-13)


def test_definition_pair_by_pair():
    q, k, v, g, s0, _ = case(1, N=7)
    out, _, _ = gated.forward(q, k, v, g, 1.0, s0)
    for t, h in itertools.product(range(7), range(2)):
        o = math.exp(g[0, :t + 1, h].sum()) * s0[0, h] @ q[0, t, h]
        for s in range(t + 1):
            o = o + math.exp(g[0, s + 1:t + 1, h].sum()) * (q[0, t, h] @ k[0, s, h]) * v[0, s, h]
        assert np.allclose(out[0, t, h], o, rtol=1e-12, atol=1e-12)


def test_exact_with_dyadic_inputs():
    """Halving gates and small integers: rational arithmetic, digit by digit."""
    r = np.random.default_rng(3)
    q, k, v = (r.integers(-3, 4, (1, 6, 1, 2)).astype(float) for _ in range(3))
    g = np.full((1, 6, 1), -math.log(2.0))
    out, _, _ = gated.forward(q, k, v, g, 1.0)
    S = [[Fraction(0)] * 2 for _ in range(2)]
    for t in range(6):
        S = [[S[c][e] / 2 + Fraction(int(v[0, t, 0, c])) * int(k[0, t, 0, e]) for e in range(2)] for c in range(2)]
        for c in range(2):
            assert abs(float(S[c][0] * int(q[0, t, 0, 0]) + S[c][1] * int(q[0, t, 0, 1])) - out[0, t, 0, c]) < 1e-12


def test_resets_and_streaming():
    q, k, v, g, s0, _ = case(2, N=9)
    g[0, 4] = -math.inf
    out, s1, _ = gated.forward(q, k, v, g, 1.0, s0)
    late, s2, _ = gated.forward(*(x[:, 4:] for x in (q, k, v, g)), 1.0)
    assert np.array_equal(out[:, 4:], late) and np.array_equal(s1, s2)
    _, mid, _ = gated.forward(*(x[:, :3] for x in (q, k, v, g)), 1.0, s0)
    rest, s3, _ = gated.forward(*(x[:, 3:] for x in (q, k, v, g)), 1.0, mid)
    assert np.array_equal(out[:, 3:], rest) and np.array_equal(s1, s3)


def test_gradient_against_differences():
    q, k, v, g, s0, r = case(4, N=5)
    do, ds = r.standard_normal(q.shape), r.standard_normal(s0.shape)
    got = gated.backward(do, q, k, v, g, 0.6, s0, ds)

    def loss(*x):
        out, s, _ = gated.forward(*x[:4], 0.6, x[4])
        return (out * do).sum() + (s * ds).sum()

    args = [q, k, v, g, s0]
    for i, a in enumerate(args):
        for at in np.ndindex(a.shape):
            keep, h = a[at], 1e-6
            a[at] = keep + h
            up = loss(*args)
            a[at] = keep - h
            num = (up - loss(*args)) / (2 * h)
            a[at] = keep
            assert abs(num - got[i][at]) < 1e-7 * (1 + abs(num))


def test_tables():
    pos = [np.array([0, 3, 1 << 20])]
    c, s = gated.tables(pos, [8])
    assert np.allclose(c ** 2 + s ** 2, 1) and np.array_equal(c[0], np.ones(4)) and np.array_equal(s[0], np.zeros(4))
    assert s[1, 1] == math.sin(3 * 10000.0 ** -0.25)
    lin, _ = gated.tables([np.array([12])], [8], scaling="linear", factor=4.0)
    assert np.allclose(lin, gated.tables([np.array([3])], [8])[0])
    # YaRN leaves fast pairs alone, interpolates slow ones and lies between otherwise
    theta = 1e6
    f = theta ** (-np.arange(0, 64, 2) / 64)
    turns = 4096 * f / (2 * math.pi)
    ang = np.arctan2(*gated.tables([np.array([1])], [64], theta=theta, scaling="yarn", factor=4.0)[::-1])[0]
    assert np.allclose(ang[turns > 32], f[turns > 32]) and np.allclose(ang[turns < 1], f[turns < 1] / 4)
    assert ((ang <= f * (1 + 1e-12)) & (ang >= f / 4 * (1 - 1e-12))).all()
    # NTK keeps the fastest pair and slows the slowest by the factor
    n = np.arctan2(*gated.tables([np.array([1])], [64], theta=theta, scaling="ntk", factor=4.0)[::-1])[0]
    assert np.isclose(n[0], 1.0) and np.isclose(n[-1], f[-1] / 4)


@pytest.mark.parametrize("half", [False, True])
def test_norm_rope(half):
    r = np.random.default_rng(5)
    x = r.standard_normal((2, 3, 2, 12))
    c, s = gated.tables([np.arange(3)], [8])
    y = gated.norm_rope(x, None, c, s, half, eps=0.0)
    assert np.allclose((y * y).mean(-1), 1.0)                       # a rotation keeps the norm
    n = x / np.sqrt((x * x).mean(-1, keepdims=True))
    assert np.array_equal(y[:, 0], n[:, 0]) and np.array_equal(y[..., 8:], n[..., 8:])
    i, j = (1, 5) if half else (2, 3)                               # pair 1 as a complex number
    z = (n[1, 2, 1, i] + 1j * n[1, 2, 1, j]) * (c[2, 1] + 1j * s[2, 1])
    assert np.allclose([y[1, 2, 1, i], y[1, 2, 1, j]], [z.real, z.imag])


def test_bf16_bits_are_widened_exactly():
    assert np.array_equal(gated.widen(np.array([0x3f80, 0xc000, 0x7f80], np.uint16)), [1.0, -2.0, np.inf])
