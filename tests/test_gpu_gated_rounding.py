"""bf16 outputs of the gated recurrence are its fp32 results rounded once.

Inputs whose outputs are single products, so that no sum adds its own roundings:
what is left is the accuracy with which computed values (states, weighted scores,
weighted values) enter the matrix units.
"""
import math

import pytest
import torch

import block_causal_relu_b200 as lcla

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def step_of(x):
    """2^e of 2^e <= |x| < 2^(e+1)."""
    return torch.ldexp(torch.ones_like(x), torch.frexp(x)[1] - 1)


def beside_the_middle(gen, *shape):
    """(bf16 values b, half a bf16 step h, a 2^-20 off it e): b + h + e is exact in fp32 and rounds towards e."""
    b = torch.randn(*shape, generator=gen, device="cuda").to(BF).float()
    b = torch.where(b.abs() < 2.0 ** -6, torch.ones_like(b), b)
    sign = torch.where(torch.rand(*shape, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
    return b, step_of(b) * 2.0 ** -8 * b.sign(), step_of(b) * 2.0 ** -20 * sign


@pytest.mark.parametrize("N", [1, 3, 40, 700])
@pytest.mark.parametrize("d", [32, 64])
def test_states_keep_24_bits(N, d):
    """q picks one entry of a carried state that nothing changes.  The fp32 value lies 2^-20 of itself off the middle of
    two bf16 values; sums of it and zeros cut off at most 2^-23."""
    gen = torch.Generator(device="cuda").manual_seed(N + d)
    B, H = 2, 3
    s0 = sum(beside_the_middle(gen, B, H, d, d))
    q = torch.zeros(B, N, H, d, device="cuda", dtype=BF)
    pick = torch.arange(N, device="cuda") % d
    q[:, torch.arange(N, device="cuda"), :, pick] = 1
    zero, g = torch.zeros_like(q), torch.zeros(B, N, H, device="cuda")
    out, s1 = lcla.gated_forward(q, zero, zero, g, 1.0, state_in=s0)
    want = s0[:, :, :, pick].permute(0, 3, 1, 2).to(BF)       # out[t][c] = S[c][t mod d]
    assert torch.equal(out, want) and torch.equal(s1, s0)
    # dq_t = S^T do_t and, of a carried gradient, dk_t = R^T v_t and dv_t = R k_t
    dq, dk, dv, *_ = lcla.gated_backward(q, zero, q, q, g, 1.0, dstate_out=s0)
    assert torch.equal(dv, want)
    assert torch.equal(dk, s0[:, :, pick].permute(0, 2, 1, 3).to(BF))
    dq, *_ = lcla.gated_backward(q, zero, zero, zero, g, 1.0, state_in=s0)
    assert torch.equal(dq, s0[:, :, pick].permute(0, 2, 1, 3).to(BF))


@pytest.mark.parametrize("d", [32, 64])
def test_scores_keep_24_bits(d):
    """A score of three products 2^-20 off the middle of two bf16 values, against values that pick one token each."""
    gen = torch.Generator(device="cuda").manual_seed(d)
    B, N, H = 2, 32, 3
    terms = beside_the_middle(gen, B, N, H)
    one = torch.zeros(B, N, H, d, device="cuda", dtype=BF)
    one[..., :3] = 1
    x = torch.zeros_like(one)
    for i, t in enumerate(terms):
        x[..., i] = t.to(BF)
    pick = torch.zeros_like(one)
    pick[:, torch.arange(N, device="cuda"), :, torch.arange(N, device="cuda")] = 1
    g = torch.zeros(B, N, H, device="cuda")
    score = sum(terms).to(BF).transpose(1, 2)                     # [B, H, key]
    after = torch.ones(N, N, device="cuda").tril()                # [query, key]
    want = torch.zeros_like(one)
    want[..., :N] = (score[:, :, None] * after.to(BF)).transpose(1, 2)
    out, _ = lcla.gated_forward(one, x, pick, g, 1.0)             # out_t = sum over s <= t of (1 . x_s) pick_s
    assert torch.equal(out, want)
    dq, *_ = lcla.gated_backward(one, one, pick, x, g, 1.0)       # dq_t = sum over s <= t of (do_t . v_s) k_s
    assert torch.equal(dq, want)
    want[..., :N] = (score[:, :, None] * after.t().to(BF)).transpose(1, 2)
    _, _, dv, *_ = lcla.gated_backward(pick, x, one, one, g, 1.0)  # dv_s = sum over t >= s of (k_s . q_t) do_t
    assert torch.equal(dv, want)
    _, dk, *_ = lcla.gated_backward(x, pick, one, one, g, 1.0)    # dk_s = sum over t >= s of (v_s . do_t) q_t
    assert torch.equal(dk, want)


@pytest.mark.parametrize("d", [32, 64])
def test_weighted_values_keep_24_bits(d):
    """Sequences of 64 tokens in which one token alone has a value: its weight goes through a tile's scores, or through
    the state and out of it again.  Each weight is within 2^-21, a value meets at most two, and its roundings and cut-off
    bits on the way (three sums, two products, the split) stay below 2^-22 each: 2^-19 of the output beside half a step."""
    gen = torch.Generator(device="cuda").manual_seed(d)
    B, N, H = 1, 4096, 70 * 32 // d
    t = torch.arange(N, device="cuda")
    g = -0.05 * torch.rand(B, N, H, generator=gen, device="cuda")
    g[:, t % 64 == 0] = -math.inf
    one = torch.zeros(B, N, H, d, device="cuda", dtype=BF)
    one[..., 0] = 1
    G = g.double()
    G[:, t % 64 == 0] = 0
    G = G.reshape(B, N // 64, 64, H).cumsum(2)

    def check(o, r):
        lim = step_of(r) * 2.0 ** -8 + 2.0 ** -19 * r.abs()
        over = int(((o.double() - r).abs() > lim).sum())
        assert over == 0, f"{over} of {o.numel()} outputs are not the rounded result"

    v = torch.randn(B, N, H, d, generator=gen, device="cuda").to(BF)
    v = torch.where((t % 64 == 0)[None, :, None, None], v, torch.zeros_like(v))
    out, _ = lcla.gated_forward(one, one, v, g, 1.0)
    src = v.double().reshape(B, N // 64, 64, H, d)
    check(out, (src[:, :, :1] * G.exp()[..., None]).reshape(B, N, H, d))
    do = torch.randn(B, N, H, d, generator=gen, device="cuda").to(BF)
    do = torch.where((t % 64 == 63)[None, :, None, None], do, torch.zeros_like(do))
    _, _, dv, *_ = lcla.gated_backward(do, one, one, v, g, 1.0)
    src = do.double().reshape(B, N // 64, 64, H, d)
    check(dv, (src[:, :, 63:] * (G[:, :, 63:] - G).exp()[..., None]).reshape(B, N, H, d))
