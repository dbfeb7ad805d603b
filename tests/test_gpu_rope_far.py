"""Rotary tables at far positions, against frequencies and angles in 60 digits."""
import math
from decimal import Decimal, getcontext

import pytest
import torch

import block_causal_relu_b200 as lcla

pytestmark = pytest.mark.gpu
getcontext().prec = 60
PI2 = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def turns(D, theta, scaling, factor, L0=4096, fast=32, slow=1):
    """Revolutions per position of each pair."""
    theta, factor = Decimal(theta), Decimal(factor)
    base = theta * (factor.ln() * D / (D - 2)).exp() if scaling == "ntk" else theta
    out = []
    for j in range(D // 2):
        f = (-base.ln() * 2 * j / D).exp()
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            keep = min(Decimal(1), max(Decimal(0), (L0 * f / PI2 - slow) / (fast - slow)))
            f = f * keep + f / factor * (1 - keep)
        out.append(f / PI2)
    return out


def reference(positions, rev, amp):
    cos, sin = [], []
    for p in positions:
        a = [float((p * r) % 1) * 2 * math.pi for r in rev]
        cos.append([math.cos(x) * amp for x in a])
        sin.append([math.sin(x) * amp for x in a])
    return torch.tensor(cos, dtype=torch.float64), torch.tensor(sin, dtype=torch.float64)


@pytest.mark.parametrize("D,theta", [(32, 10000.0), (64, 500000.0), (128, 10000.0), (256, 1.5)])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 3.0), ("ntk", 8.0), ("yarn", 3.5)])
def test_far_positions(D, theta, scaling, factor):
    """Within 2e-7 of amp times each cosine and sine up to 2^36: the angle's 2^-64 of a turn per position (2.4e-8), its
    rounding to 24 bits (4.7e-8), the polynomials (2e-9), and up to three roundings of the value (1.8e-7 amp at most
    together where it is largest, 6e-8 typically)."""
    amp = 0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0
    rev = turns(D, theta, scaling, factor)
    gen = torch.Generator().manual_seed(D)
    pos = torch.cat([torch.randint(0, 1 << b, (20,), generator=gen) for b in (20, 31, 33, 36)] +
                    [torch.tensor([1 << 36, -(1 << 36), -(1 << 33) + 7, (1 << 31) - 1])])
    c, s = lcla.rotary_tables(len(pos), D, positions=pos.cuda(), theta=theta, scaling=scaling, factor=factor)
    rc, rs = reference(pos.tolist(), rev, amp)
    assert float((c.double().cpu() - rc).abs().max()) < 2e-7 * amp
    assert float((s.double().cpu() - rs).abs().max()) < 2e-7 * amp


def test_far_grid_indices():
    """The last grid of the range, one axis and three."""
    n = 300
    first = (1 << 36) - n
    c, s = lcla.rotary_tables(n, 64, first=first)
    rc, rs = reference(range(first, first + n), turns(64, 10000.0, "none", 1.0), 1.0)
    assert float((c.double().cpu() - rc).abs().max()) < 2e-7 and float((s.double().cpu() - rs).abs().max()) < 2e-7
    dims, ext = [8, 12, 12], [44, 80]
    c, s = lcla.rotary_tables(n, dims, extents=ext, first=first)
    at = 0
    for a, D in enumerate(dims):
        pos = [i // math.prod(ext[a:]) for i in range(first, first + n)]
        pos = [p % ext[a - 1] if a else p for p in pos]
        rc, rs = reference(pos, turns(D, 10000.0, "none", 1.0), 1.0)
        assert float((c[:, at:at + D // 2].double().cpu() - rc).abs().max()) < 2e-7
        assert float((s[:, at:at + D // 2].double().cpu() - rs).abs().max()) < 2e-7
        at += D // 2
    with pytest.raises(lcla.LclaError):
        lcla.rotary_tables(n, 64, first=first + 1)
