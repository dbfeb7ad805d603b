"""The gradient of the gates, dg_t = e^{g_t} <S_{t-1}, R_t>: a sum over the pairs
(s, u) of tokens s < t <= u, M[u][s] = scale e^{G_u - G_s} (q_u . k_s) (do_u . v_s).

``own`` is the same sum over magnitudes.  A gradient may be off by 2^-17 of it
(the roundings of the recurrence's outputs, 2^-18 at most with both types, and
of up to 64 additions in a row); it has nothing of pairs that a strong gate or a
reset separates from the token.  The kernel takes the pairs around a whole tile
of 32 tokens as a difference, D - sum of B, of two sums over the pairs around
the tile's end: each is within 2^-20 of its magnitudes (two factors at 2^-22,
their product and the additions), hence 2^-19 of ``own`` behind the tile's last
token (behind the sequence: of <|S|, |R|>).
"""
import math

import pytest
import torch

import block_causal_relu_b200 as lcla
from test_gpu_gated import mag, ref_backward, ref_forward

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]


def problem(seed, B, N, H, d, dtype, state=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, do = (r(B, N, H, d).to(dtype) for _ in range(4))
    s0, ds = (r(B, H, d, d), r(B, H, d, d)) if state else (None, None)
    return gen, q, k, v, do, s0, ds


def both(q, k, v, g, do, s0, ds, scale=0.3):
    """(dg, exact dg, own magnitudes, the magnitudes behind each token's tile)"""
    got = lcla.gated_backward(do, q, k, v, g, scale, state_in=s0, dstate_out=ds)[3]
    ref = ref_backward(do, q, k, v, g, s0, ds, scale)[3]
    own = ref_backward(mag(do), mag(q), mag(k), mag(v), g, mag(s0), mag(ds), scale)[3]
    last = torch.zeros_like(own[:, :1])
    if ds is not None:
        _, S, _ = ref_forward(mag(q), mag(k), mag(v), g, mag(s0), scale)
        last = (S * mag(ds)).sum((-1, -2))[:, None]
    N = g.shape[1]
    t = torch.arange(N, device="cuda")
    around = torch.cat([own, last], 1)[:, ((t // 32 + 1) * 32).clamp(max=N)]
    assert torch.isfinite(got).all()
    return got.double(), ref, own, around


def close(got, ref, own, around, what):
    worst = ((got - ref).abs() / (2.0 ** -17 * own + 2.0 ** -19 * around + 1e-300)).max()
    assert float(worst) <= 1, f"{what}: {float(worst):.3g} of its tolerance"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("N", [2, 33, 500])
@pytest.mark.parametrize("g0", [-1.1, -3.0, -6.0, -10.0, -15.0, -20.0, -60.0, "mixed"])
def test_strong_gates(g0, N, d, dtype):
    """States that forget within a few tokens: every gradient to the accuracy of its own terms."""
    gen, q, k, v, do, s0, ds = problem(N + d, 2, N, 3, d, dtype)
    u = torch.rand(2, N, 3, generator=gen, device="cuda")
    g = -3 - 17 * u if g0 == "mixed" else g0 * (1 + 0.1 * u)
    close(*both(q, k, v, g.contiguous(), do, s0, ds), f"g = {g0}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("gate", [-math.inf, -1000.0, -300.0, -104.5, -90.0])
@pytest.mark.parametrize("H", [2, 160])
def test_packed_sequences_leave_each_other_alone(H, gate, d, dtype):
    """Sequences of very different magnitudes, the loud ones last, behind gates that let nothing through: within 2^-17 of
    the magnitudes of <q, dq> and <k, dk> over the rest of the own sequence; zero where e^g is zero in fp32.  With many
    heads a segment holds several sequences."""
    lens, loud = [70, 1, 300, 33, 5, 600], [1.0, 1e2, 1e-2, 1e3, 1e-3, 1e4]
    N, B, scale = sum(lens), 1, 0.3
    gen, q, k, v, do, _, _ = problem(d, B, N, H, d, dtype, False)
    g = -0.02 * torch.rand(B, N, H, generator=gen, device="cuda")
    at = 0
    for L, x in zip(lens, loud):
        g[:, at] = gate
        do[:, at:at + L] *= x
        q[:, at:at + L] *= x
        at += L
    got = lcla.gated_backward(do, q, k, v, g, scale)[3][:, :, -2:].double()
    do, q, k, v, g = (x[:, :, -2:] for x in (do, q, k, v, g))
    at = 0
    for L in lens:
        part = [x[:, at:at + L].contiguous() for x in (do, q, k, v, g)]
        ref = ref_backward(*part, None, None, scale)[3]
        A = ref_backward(*(mag(x) for x in part[:4]), part[4], None, None, scale)
        each = (mag(part[1]).double() * A[0]).sum(-1) + (mag(part[2]).double() * A[1]).sum(-1)
        lim = 2.0 ** -17 * each.flip(1).cumsum(1).flip(1)
        err = (got[:, at:at + L] - ref).abs()
        if gate < -104:
            assert (got[:, at] == 0).all()
            err, lim = err[:, 1:], lim[:, 1:]
        else:      # what little the gate lets through of the sequence before it
            err, lim = err[:, 1:], lim[:, 1:] + math.exp(gate) * 1e12
        assert bool((err <= lim).all()), f"{gate}, sequence at {at}: {float((err / lim).max()):.3g}"
        at += L


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [32, 64])
def test_a_loud_token_does_not_reach_tokens_that_it_cannot(d, dtype):
    """Gates of -1.2 and one late token with a million times the gradient: 14 tokens before it nothing of that is left.
    Many heads, so that segments are long."""
    gen, q, k, v, do, s0, ds = problem(3 * d, 2, 700, 80, d, dtype)
    g = -1.2 - 0.1 * torch.rand(2, 700, 80, generator=gen, device="cuda")
    do[:, 640] *= 1e6
    got = lcla.gated_backward(do, q, k, v, g, 0.3, state_in=s0, dstate_out=ds)[3][:, :, 7:9].double()
    some = [x[:, :, 7:9].contiguous() for x in (q, k, v, g, do)]
    _, ref, own, around = both(*some, s0[:, 7:9].contiguous(), ds[:, 7:9].contiguous())
    close(got, ref, own, around, "long segments")
    close(*both(*some, s0[:, 7:9].contiguous(), ds[:, 7:9].contiguous()), "short segments")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,d", [(2048, 32), (1531, 64), (4700, 64)])
@pytest.mark.parametrize("bias", [1.0, 3.0, 5.0, 8.0])
def test_gates_of_all_memories_in_the_2_norm(bias, N, d, dtype):
    """With a memory of m tokens a gradient is a sum of some m terms of either sign, and its rounding one of the terms of
    the rest of its segment, at most 1024 tokens on either side.  Each term is within 2^-21 of itself, at random, so the
    norm is within 2^-21 sqrt(2048 / m): below 2^-16 for m >= 2."""
    for H in (2, 150):
        gen, q, k, v, do, _, _ = problem(N, 1, N, H, d, dtype, False)
        g = torch.nn.functional.logsigmoid(torch.randn(1, N, H, generator=gen, device="cuda") + bias)
        got = lcla.gated_backward(do, q, k, v, g, 0.3)[3][:, :, -2:].double()
        ref = ref_backward(*(x[:, :, -2:] for x in (do, q, k, v, g)), None, None, 0.3)[3]
        rel = (got - ref).norm(dim=1) / ref.norm(dim=1)
        print(f"H {H}: {float(rel.max()):.2g}")
        assert float(rel.max()) <= 2.0 ** -16, float(rel.max())


@pytest.mark.parametrize("d", [32, 64])
def test_single_strong_gates_among_mild_ones(d):
    """A gate of -3 to -12 in a tile that keeps its state otherwise: its gradient is e^g of its neighbours', and what goes
    around the tile keeps their roundings: within 2^-17 of its own terms and 2^-20 of theirs."""
    gen, q, k, v, do, s0, ds = problem(d, 1, 640, 3, d, torch.float32)
    g = -1e-3 * torch.rand(1, 640, 3, generator=gen, device="cuda")
    at = torch.arange(9, 640, 64, device="cuda")
    g[:, at] = torch.linspace(-3, -12, len(at), device="cuda")[None, :, None]
    got, ref, own, _ = both(q, k, v, g, do, s0, ds)
    err = (got - ref).abs()
    near = torch.nn.functional.max_pool1d(own.transpose(1, 2), 65, 1, 32).transpose(1, 2)
    assert bool((err <= 2.0 ** -17 * own + 2.0 ** -20 * near).all())


def test_the_first_gate_without_a_state_has_no_gradient():
    gen, q, k, v, do, _, ds = problem(1, 2, 70, 3, 32, torch.float32)
    dg = lcla.gated_backward(do, q, k, v, torch.zeros(2, 70, 3, device="cuda"), dstate_out=ds)[3]
    assert (dg[:, 0] == 0).all() and (dg[:, 1:] != 0).any()
