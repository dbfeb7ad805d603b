"""Refusals of the gated recurrence's entry points, on the host: every call here
fails validation (or has nothing to do), so no kernel is launched."""
import pytest

import block_causal_relu_b200 as lcla

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = range(5)
A = 1 << 26
BASE = dict(q=A, k=2 * A, v=3 * A, g=4 * A, B=2, H=3, N=400, d=32, scale=0.2, s0=5 * A, out=6 * A, s1=7 * A, dtype=0,
            ws=8 * A, wsb=1 << 25, do=9 * A, dq=10 * A, dk=11 * A, dv=12 * A, dg=13 * A, ds1=14 * A, ds0=15 * A, save=1)


def fwd(**kw):
    a = dict(BASE, **kw)
    return lcla.lib.lcla_gated_forward(a["q"], a["k"], a["v"], a["g"], a["B"], a["H"], a["N"], a["d"], a["scale"],
                                       a["s0"], a["out"], a["s1"], a["dtype"], a["ws"], a["wsb"], None)


def stp(**kw):
    a = dict(BASE, **kw)
    return lcla.lib.lcla_gated_step(a["q"], a["k"], a["v"], a["g"], a["B"], a["H"], a["N"], a["d"], a["scale"], a["s0"],
                                    a["save"], a["out"], a["dtype"], a["ws"], a["wsb"], None)


def bwd(**kw):
    a = dict(BASE, **kw)
    return lcla.lib.lcla_gated_backward(a["do"], a["q"], a["k"], a["v"], a["g"], a["B"], a["H"], a["N"], a["d"],
                                        a["scale"], a["s0"], a["ds1"], a["dq"], a["dk"], a["dv"], a["dg"], a["ds0"],
                                        a["dtype"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(N=-1), INVALID), (dict(d=0), INVALID), (dict(d=33), INVALID),
    (dict(d=128), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(N=(1 << 30) + 1), UNSUPPORTED),
    (dict(B=65536), UNSUPPORTED), (dict(H=65536), UNSUPPORTED), (dict(B=60000, H=60000), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=1e-30), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(g=None), INVALID), (dict(q=A + 8), MISALIGNED), (dict(g=4 * A + 2), MISALIGNED), (dict(ws=8 * A + 8), MISALIGNED),
    (dict(s0=5 * A + 4), MISALIGNED),
])
def test_common(kw, code):
    assert fwd(**kw) == code
    assert stp(**kw) == code
    assert bwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(out=None), INVALID), (dict(out=A), INVALID), (dict(out=4 * A), INVALID), (dict(out=5 * A), INVALID),
    (dict(out=7 * A), INVALID), (dict(s1=2 * A), INVALID), (dict(s1=5 * A + 64), INVALID), (dict(s1=7 * A + 4), MISALIGNED),
    (dict(out=6 * A + 2), MISALIGNED),
])
def test_forward(kw, code):
    assert fwd(**kw) == code


def test_forward_workspace():
    need = lcla.gated_forward_workspace_bytes(2, 3, 4000, 32, lcla.BF16)
    assert need > 0 and need % 256 == 0
    assert fwd(N=4000, ws=None) == WORKSPACE and fwd(N=4000, wsb=need - 1) == WORKSPACE
    assert fwd(N=4000, ws=A, wsb=need) == INVALID and fwd(N=4000, out=8 * A, wsb=need) == INVALID
    assert lcla.gated_forward_workspace_bytes(2, 3, 32, 32, lcla.F32) == 0      # one tile needs none
    assert lcla.gated_forward_workspace_bytes(2, 3, 4000, 128, lcla.F32) == 0
    assert lcla.gated_forward_workspace_bytes(0, 3, 4000, 32, lcla.F32) == 0


def test_empty():
    none = dict(N=0, q=None, k=None, v=None, g=None, out=None, ws=None, wsb=0)
    assert fwd(**none, s1=None) == OK
    assert fwd(**none, s0=5 * A, s1=5 * A) == OK
    assert stp(**none) == OK
    assert stp(N=0, s0=None) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(do=None), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID), (dict(dv=None), INVALID),
    (dict(dg=None), INVALID), (dict(dq=A), INVALID), (dict(dk=10 * A), INVALID), (dict(dg=4 * A), INVALID),
    (dict(dv=9 * A), INVALID), (dict(ds0=5 * A), INVALID), (dict(ds0=14 * A + 64), INVALID), (dict(ws=None), WORKSPACE),
    (dict(wsb=64), WORKSPACE), (dict(ws=9 * A), INVALID), (dict(dq=10 * A + 4), MISALIGNED), (dict(dg=13 * A + 2), MISALIGNED), (dict(ds1=14 * A + 4), MISALIGNED),
    (dict(ds0=13 * A), INVALID),
])
def test_backward(kw, code):
    assert bwd(**kw) == code


def test_binding_refuses():
    import torch
    x, g = torch.zeros(1, 2, 2, 32), torch.zeros(1, 2, 2)
    with pytest.raises(TypeError):
        lcla.gated_forward(x, x, x, g)
    with pytest.raises(TypeError):
        lcla.gated_step(x, x, x, g, None, True)


def test_the_unsupported_string_says_what_is_served():
    text = lcla.lib.lcla_status_string(UNSUPPORTED).decode()
    assert "32 and 64" in text and "256" in text and "2^30" in text
