"""Refusals of the rotary and norm entry points, on the host: every call here
fails validation (or has nothing to do), so no kernel is launched."""
import ctypes

import pytest

import block_causal_relu_b200 as lcla

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = range(5)
A = 1 << 24


def tables(**kw):
    a = dict(pos=None, first=0, N=100, dims=(8, 12, 12), ext=(4, 5), theta=1e4, scaling=0, factor=1.0, L0=4096.0,
             fast=32.0, slow=1.0, c=A, s=2 * A)
    a.update(kw)
    n = len(a["dims"])
    dims = (ctypes.c_int * max(n, 1))(*a["dims"])
    ext = None if a["ext"] is None else (ctypes.c_int * max(len(a["ext"]), 1))(*a["ext"])
    return lcla.lib.lcla_rotary_tables(a["pos"], a["first"], a["N"], n, dims, ext, a["theta"], a["scaling"],
                                       a["factor"], a["L0"], a["fast"], a["slow"], a["c"], a["s"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), INVALID), (dict(dims=()), INVALID), (dict(dims=(2, 2, 2, 2)), INVALID), (dict(dims=(3,)), INVALID),
    (dict(dims=(0,)), INVALID), (dict(dims=(258,)), UNSUPPORTED), (dict(ext=None), INVALID), (dict(ext=(0, 5)), INVALID),
    (dict(theta=0.5), INVALID), (dict(theta=float("nan")), INVALID), (dict(scaling=4), INVALID),
    (dict(scaling=1, factor=0.5), INVALID), (dict(scaling=2, dims=(2,), factor=2.0), INVALID),
    (dict(scaling=3, factor=2.0, fast=1.0), INVALID), (dict(scaling=3, factor=2.0, L0=0.0), INVALID),
    (dict(first=-1), UNSUPPORTED), (dict(first=(1 << 60) + 1), UNSUPPORTED), (dict(N=(1 << 30) + 1), UNSUPPORTED),
    (dict(c=None), INVALID), (dict(s=None), INVALID), (dict(c=A + 4), MISALIGNED), (dict(pos=3 * A + 4), MISALIGNED),
    (dict(s=A), INVALID), (dict(pos=A + 8), INVALID), (dict(N=0, c=None, s=None), OK),
])
def test_tables(kw, code):
    assert tables(**kw) == code


BASE = dict(q=A, ldq=256, k=2 * A, ldk=128, B=2, N=10, H=4, Hk=2, d=64, wq=5 * A, wk=6 * A, eps=1e-6, c=7 * A, s=8 * A,
            rows=10, rd=64, half=0, pos=None, qo=9 * A, ldqo=256, ko=10 * A, ldko=128, dtype=0)


def norm(**kw):
    a = dict(BASE, **kw)
    return lcla.lib.lcla_qk_norm_rope(a["q"], a["ldq"], a["k"], a["ldk"], a["B"], a["N"], a["H"], a["Hk"], a["d"],
                                      a["wq"], a["wk"], a["eps"], a["c"], a["s"], a["rows"], a["rd"], a["half"],
                                      a["pos"], a["qo"], a["ldqo"], a["ko"], a["ldko"], a["dtype"], None)


def grad(**kw):
    a = dict(BASE, gq=11 * A, ldgq=256, gk=12 * A, ldgk=128, dwq=13 * A, dwk=14 * A, ws=15 * A, wsb=1 << 20)
    a.update(kw)
    return lcla.lib.lcla_qk_norm_rope_backward(
        a["gq"], a["ldgq"], a["gk"], a["ldgk"], a["q"], a["ldq"], a["k"], a["ldk"], a["B"], a["N"], a["H"], a["Hk"],
        a["d"], a["wq"], a["wk"], a["eps"], a["c"], a["s"], a["rows"], a["rd"], a["half"], a["pos"], a["qo"],
        a["ldqo"], a["ko"], a["ldko"], a["dwq"], a["dwk"], a["dtype"], a["ws"], a["wsb"], None)


COMMON = [
    (dict(B=0), INVALID), (dict(N=-1), INVALID), (dict(H=0), INVALID), (dict(Hk=-1), INVALID), (dict(rd=66), INVALID),
    (dict(rd=7), INVALID), (dict(rd=-2), INVALID), (dict(dtype=2), INVALID), (dict(half=2), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(rows=9), INVALID), (dict(rows=0), INVALID),
    (dict(d=60, rd=32), UNSUPPORTED), (dict(d=264, rd=32), UNSUPPORTED), (dict(half=1, rd=24), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(qo=None), INVALID), (dict(ko=None), INVALID),
    (dict(c=None), INVALID), (dict(ldq=255), INVALID), (dict(ldq=260), MISALIGNED), (dict(ldk=64), INVALID),
    (dict(q=A + 8), MISALIGNED), (dict(c=7 * A + 4), MISALIGNED), (dict(wq=5 * A + 4), MISALIGNED),
    (dict(pos=3 * A + 4), MISALIGNED), (dict(qo=7 * A), INVALID), (dict(ko=9 * A), INVALID),
    (dict(qo=2 * A), INVALID), (dict(qo=A + 512), INVALID), (dict(pos=9 * A), INVALID),
]


@pytest.mark.parametrize("kw,code", COMMON)
def test_norm(kw, code):
    assert norm(**kw) == code
    assert grad(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(qo=A, ldqo=512), INVALID),               # in place needs the same rows
    (dict(N=0, q=None, k=None, qo=None, ko=None, rows=1), OK),
    (dict(N=0, q=None, k=None, qo=None, ko=None, rows=0), OK), (dict(N=0, rows=-1), INVALID),
])
def test_norm_only(kw, code):
    assert norm(**kw) == code


def test_windows_of_one_buffer_are_told_apart():
    # q and k outputs as the two column windows of one buffer: refused only where the columns meet
    assert norm(qo=9 * A, ldqo=384, ko=9 * A + 512, ldko=384, c=None) == INVALID          # tables missing: reached checks
    assert norm(qo=9 * A, ldqo=384, ko=9 * A + 496, ldko=384) == INVALID                  # they share 16 bytes
    assert norm(qo=9 * A + 64, ldqo=384, ko=9 * A, ldko=384) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE), (dict(ws=15 * A + 8), MISALIGNED),
    (dict(wq=None), INVALID), (dict(wk=None), INVALID), (dict(gq=None), INVALID), (dict(gk=None), INVALID),
    (dict(dwq=13 * A + 4), MISALIGNED), (dict(dwk=13 * A), INVALID), (dict(dwq=5 * A), INVALID),
    (dict(qo=A), INVALID),                          # dq in q's place: the forward's input is still needed
    (dict(ws=A), INVALID), (dict(ldgq=128), INVALID), (dict(gk=12 * A + 2), MISALIGNED),
])
def test_gradient(kw, code):
    assert grad(**kw) == code


def test_workspace_query():
    f = lcla.lib.lcla_qk_norm_rope_backward_workspace_bytes
    assert f(64) == 2 * f(32) > 0
    assert f(0) == f(12) == f(264) == 0


def test_binding_refuses():
    import torch
    x = torch.zeros(1, 2, 2, 32)
    with pytest.raises(TypeError):
        lcla.qk_norm_rope(x, None, x[0, 0], x[0, 0])
    with pytest.raises(ValueError):
        lcla.rotary_tables(4, [8, 8], device="cuda")            # no extents
    with pytest.raises(ValueError):
        lcla.rotary_tables(4, 32, scaling="other")
    with pytest.raises(ValueError):
        lcla.rotary_tables(-1, 32)


@pytest.mark.parametrize("first,code", [((1 << 36) - 100, INVALID), ((1 << 36) - 99, UNSUPPORTED), (1 << 50, UNSUPPORTED),
                                        ((1 << 63) - 1, UNSUPPORTED)])
def test_indices_beyond_the_angles_are_refused(first, code):
    """The last grid index is 2^36 - 1, where an angle is still exact enough; the invalid call is refused for its NULL."""
    assert tables(first=first, c=None) == code
