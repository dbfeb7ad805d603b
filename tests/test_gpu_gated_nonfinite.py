"""NaNs and infinities reach what the formulas take them to, and nothing else:
not the outputs of earlier tokens of the same tile, whose scores with them are
masked."""
import math

import pytest
import torch

import block_causal_relu_b200 as lcla
from test_gpu_gated import make, mag, ref_backward, ref_forward

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]
# N, tokens that are not finite
CASES = [(1, [0]), (6, [3]), (20, [19]), (32, [0, 31]), (33, [32]), (100, [40]), (700, [350, 351]), (700, [699])]


def same(o, r, A, dtype, what):
    """Finite where the reference is, and there within the tolerances of finite inputs."""
    fine = torch.isfinite(r)
    assert torch.equal(torch.isfinite(o), fine), f"{what}: {int((torch.isfinite(o) != fine).sum())} entries"
    if not fine.any():
        return
    lim = 2.0 ** -(16 if dtype == torch.bfloat16 else 17) * A[fine] + 1e-30
    if dtype == torch.bfloat16:
        lim = lim + 2.0 ** -8 * r[fine].abs() * (1 + 2.0 ** -8)
    assert bool(((o.double()[fine] - r[fine]).abs() <= lim).all()), what


def spoil(x, tokens, bad, head, entry):
    """Entry `entry` of one head (None: all of them) of the given tokens."""
    for t in tokens:
        if entry is None:
            x[:, t, head] = bad
        else:
            x[:, t, head, entry] = bad


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("which", ["q", "k", "v", "v all"])
def test_forward(which, d, dtype, bad):
    for i, (N, tokens) in enumerate(CASES):
        B, H = 2, 3
        q, k, v, g, s0 = make(i, B, N, H, d, dtype, True, "mixed")
        clean = [mag(x) for x in (q, k, v)]
        x = {"q": q, "k": k, "v": v}[which[0]]
        spoil(x, tokens, bad, 1, None if "all" in which else d - 3)
        out, s1 = lcla.gated_forward(q, k, v, g, 0.5, state_in=s0)
        r, rs, _ = ref_forward(q, k, v, g, s0, 0.5)
        A, As, _ = ref_forward(*clean, g, mag(s0), 0.5)
        same(out, r, A, dtype, f"out, N = {N}")
        same(s1, rs, As, torch.float32, f"state, N = {N}")


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("which", ["q", "k", "v", "do", "do all"])
def test_gradient(which, d, dtype, bad):
    for i, (N, tokens) in enumerate(CASES):
        B, H = 1, 3
        q, k, v, g, s0 = make(i, B, N, H, d, dtype, True, "mixed")
        do = torch.randn(B, N, H, d, device="cuda").to(dtype)
        clean = [mag(x) for x in (do, q, k, v)]
        x = {"q": q, "k": k, "v": v, "d": do}[which[0]]
        spoil(x, tokens, bad, 1, None if "all" in which else d - 3)
        got = lcla.gated_backward(do, q, k, v, g, 0.5, state_in=s0, want_dstate_in=True)
        ref = ref_backward(do, q, k, v, g, s0, None, 0.5)
        A = ref_backward(*clean, g, mag(s0), None, 0.5)
        for name, o, r, a in zip(("dq", "dk", "dv"), got, ref, A):
            same(o, r, a, dtype, f"{name}, N = {N}")
        same(got[4], ref[4], A[4], torch.float32, f"dstate_in, N = {N}")
        # dg: the same, but for the tokens up to one with a bad k or v, which may be NaNs too
        dg, rg = got[3].clone(), ref[3].clone()
        if which[0] in "kv":
            assert not torch.isfinite(dg[:, tokens[-1] + 1:, 1]).any()
            lost = ~torch.isfinite(dg)
            lost[:, tokens[-1] + 1:] = False
            lost[:, :, [0, 2]] = False
            dg[lost], rg[lost] = math.nan, math.nan
        each = (clean[1].double() * A[0]).sum(-1) + (clean[2].double() * A[1]).sum(-1)
        Ag = each.flip(1).cumsum(1).flip(1)
        same(dg, rg, Ag, torch.float32, f"dg, N = {N}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [32, 64])
def test_garbage_behind_the_last_token_of_a_padded_batch(d, dtype):
    """Rows of uninitialised memory behind a sequence's end change nothing of the sequence."""
    N, live = 400, 237
    q, k, v, g, s0 = make(9, 1, N, 3, d, dtype)
    want, _ = lcla.gated_forward(q, k, v, g, state_in=s0)
    for x in (q, k, v):
        x[:, live:] = math.nan
    out, s1 = lcla.gated_forward(q, k, v, g, state_in=s0)
    assert torch.equal(out[:, :live], want[:, :live])
    assert not torch.isfinite(out[:, live:]).any() and not torch.isfinite(s1).any()


@pytest.mark.parametrize("d", [32, 64])
def test_the_state_in_place_and_blocks(d):
    """A step whose block holds a NaN: the state is read before it is written, and save = 0 leaves it alone."""
    q, k, v, g, s0 = make(4, 2, 40, 3, d, torch.bfloat16)
    v[:, 20, 1, 5] = math.nan
    r, rs, _ = ref_forward(q, k, v, g, s0, 0.5)
    A, As, _ = ref_forward(mag(q), mag(k), torch.nan_to_num(mag(v)), g, mag(s0), 0.5)
    state = s0.clone()
    out = lcla.gated_step(q, k, v, g, state, False, 0.5)
    assert torch.equal(state, s0)
    same(out, r, A, torch.bfloat16, "out")
    out = lcla.gated_step(q, k, v, g, state, True, 0.5)
    same(out, r, A, torch.bfloat16, "out")
    same(state, rs, As, torch.float32, "state")
