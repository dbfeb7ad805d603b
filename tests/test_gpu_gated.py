"""The gated recurrence on the GPU (whole sequence, step, gradient) against a
token-by-token recurrence in 64 bits.

Tolerances go by the sizes of the terms: the reference is run a second time on
magnitudes (|q|, |k|, |v|, |state|), which gives for each output the sum A of
its terms' magnitudes.
  bf16: a weighted score and a state entry enter the matrix units as two bf16
  terms (relative error 2^-18 each), the sums are fp32 (under 64 additions of
  2^-23 in a chain, where the units cut off), the weights are within 2^-21:
  below 2^-16 A, then half a step of the output, 2^-8 |o|.
  fp32: two tf32 terms per factor, 2^-22 each and 2^-22 for the product left
  out, over two products; the same sums and weights: below 2^-17 A.
  States, and gradients that meet three bf16 terms: 2^-17 A as well.
  dg sums <q, dq> - <k, dk> over the rest of its segment: 2^-17 of the sum of
  those terms' magnitudes over all later tokens, plus <S, R> at the end.
"""
import math

import pytest
import torch

import block_causal_relu_b200 as lcla

pytestmark = pytest.mark.gpu


def make(seed, B, N, H, d, dtype, state=True, gates="mixed"):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v = (r(B, N, H, d).to(dtype) for _ in range(3))
    if gates == "mixed":
        g = torch.nn.functional.logsigmoid(r(B, N, H) * 2 + torch.linspace(-2, 7, H, device="cuda"))
    elif gates == "none":
        g = torch.zeros(B, N, H, device="cuda")
    elif gates == "strong":      # decays far below fp32 between tokens that barely decay
        g = torch.where(torch.rand(B, N, H, generator=gen, device="cuda") < 0.3, -300.0, -1e-3)
    elif gates == "resets":
        g = torch.where(torch.rand(B, N, H, generator=gen, device="cuda") < 0.05, -math.inf, -0.02)
    elif gates == "all resets":
        g = torch.full((B, N, H), -math.inf, device="cuda")
    elif gates == "growth":      # a state that grows
        g = torch.full((B, N, H), 0.01, device="cuda")
    s0 = r(B, H, d, d) * 2 if state else None
    return q, k, v, g.contiguous(), s0


def ref_forward(q, k, v, g, s0, scale):
    q, k, v, a = q.double(), k.double(), v.double(), g.double().exp()
    B, N, H, d = q.shape
    S = torch.zeros(B, H, d, d, dtype=torch.float64, device=q.device) if s0 is None else s0.double()
    out, states = [], []
    for t in range(N):
        states.append(S)
        S = S * a[:, t, :, None, None] + v[:, t, :, :, None] * k[:, t, :, None, :]
        out.append((S @ q[:, t, :, :, None])[..., 0] * scale)
    return (torch.stack(out, 1) if N else q), S, states


def ref_backward(do, q, k, v, g, s0, ds, scale):
    do, qd, kd, vd, a = do.double(), q.double(), k.double(), v.double(), g.double().exp()
    B, N, H, d = q.shape
    _, _, states = ref_forward(q, k, v, g, s0, scale)
    R = torch.zeros(B, H, d, d, dtype=torch.float64, device=q.device) if ds is None else ds.double()
    dq, dk, dv, dg = (torch.zeros_like(x) for x in (qd, kd, vd, a))
    for t in range(N - 1, -1, -1):
        R = R + scale * do[:, t, :, :, None] * qd[:, t, :, None, :]
        S = states[t] * a[:, t, :, None, None] + vd[:, t, :, :, None] * kd[:, t, :, None, :]
        dq[:, t] = scale * (do[:, t, :, None, :] @ S)[..., 0, :]
        dk[:, t] = (vd[:, t, :, None, :] @ R)[..., 0, :]
        dv[:, t] = (R @ kd[:, t, :, :, None])[..., 0]
        R = R * a[:, t, :, None, None]
        dg[:, t] = (R * states[t]).sum((-1, -2))
    return dq, dk, dv, dg, R


def mag(x):
    return None if x is None else x.abs()


def within(o, r, A, dtype, bits, what):
    err, lim = (o.double() - r).abs(), 2.0 ** -bits * A + 1e-30
    if dtype == torch.bfloat16:
        lim = lim + 2.0 ** -8 * r.abs() * (1 + 2.0 ** -8)
    assert torch.isfinite(o).all(), f"{what}: not finite"
    worst = float((err / lim).max()) if err.numel() else 0.0
    assert worst <= 1, f"{what}: {worst:.2f} of its tolerance"


SHAPES = [  # B, N, H, d, state
    (1, 1, 1, 32, False), (3, 2, 2, 64, True), (2, 4, 3, 32, True), (1, 5, 2, 64, True), (2, 8, 1, 64, False),
    (1, 9, 3, 32, True), (2, 16, 3, 32, True), (1, 17, 1, 64, True), (1, 32, 5, 32, False),
    (2, 33, 4, 32, True), (1, 63, 3, 64, False), (1, 64, 1, 32, True), (2, 257, 5, 64, True), (1, 700, 9, 32, True),
    (1, 1531, 2, 64, False), (1, 2048, 1, 32, True),
]


@pytest.mark.parametrize("gates", ["mixed", "none", "strong", "resets", "all resets", "growth"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,H,d,state", SHAPES)
def test_forward(B, N, H, d, state, dtype, gates):
    q, k, v, g, s0 = make(N * 7 + H, B, N, H, d, dtype, state, gates)
    scale = -0.7
    out, s1 = lcla.gated_forward(q, k, v, g, scale, state_in=s0)
    r, rs, _ = ref_forward(q, k, v, g, s0, scale)
    A, As, _ = ref_forward(mag(q), mag(k), mag(v), g, mag(s0), abs(scale))
    within(out, r, A, dtype, 16 if dtype == torch.bfloat16 else 17, "out")
    within(s1, rs, As, torch.float32, 17, "state")


@pytest.mark.parametrize("gates", ["mixed", "none", "strong", "resets", "growth"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,H,d,state", SHAPES)
def test_gradient(B, N, H, d, state, dtype, gates):
    q, k, v, g, s0 = make(N * 3 + H, B, N, H, d, dtype, state, gates)
    gen = torch.Generator(device="cuda").manual_seed(N)
    do = torch.randn(B, N, H, d, generator=gen, device="cuda").to(dtype)
    ds = torch.randn(B, H, d, d, generator=gen, device="cuda") if state else None
    scale = 0.3
    got = lcla.gated_backward(do, q, k, v, g, scale, state_in=s0, dstate_out=ds, want_dstate_in=True)
    ref = ref_backward(do, q, k, v, g, s0, ds, scale)
    A = ref_backward(mag(do), mag(q), mag(k), mag(v), g, mag(s0), mag(ds), scale)
    for name, o, r, a in zip(("dq", "dk", "dv"), got, ref, A):
        within(o, r, a, dtype, 16 if dtype == torch.bfloat16 else 17, name)
    within(got[4], ref[4], A[4], torch.float32, 17, "dstate_in")
    each = (mag(q).double() * A[0]).sum(-1) + (mag(k).double() * A[1]).sum(-1)
    Ag = each.flip(1).cumsum(1).flip(1)
    if ds is not None:
        _, last, _ = ref_forward(mag(q), mag(k), mag(v), g, mag(s0), scale)
        Ag = Ag + (last * ds.double().abs()).sum((-1, -2))[:, None]
    within(got[3], ref[3], Ag, torch.float32, 17, "dg")
    assert (got[3][torch.isinf(g)] == 0).all(), "a reset has no gradient"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,d", [(9001, 32), (5003, 64)])
def test_more_segments_than_a_scan_takes_at_once(N, d, dtype):
    """One head of a long sequence is cut into more than 64 segments."""
    test_forward(1, N, 1, d, True, dtype, "mixed")
    test_gradient(1, N, 1, d, True, dtype, "none")


def test_gradient_against_differences():
    """The reference gradient itself, against autograd and central differences of the recurrence."""
    q, k, v, g, s0 = (x.double() for x in make(1, 1, 5, 2, 4, torch.float32))
    do, ds = torch.randn_like(q), torch.randn_like(s0)

    def loss(*x):
        o, s, _ = ref_forward(*x, 0.6)
        return (o * do).sum() + (s * ds).sum()

    leaves = [x.clone().requires_grad_() for x in (q, k, v, g, s0)]
    auto = torch.autograd.grad(loss(*leaves), leaves)
    mine = ref_backward(do, q, k, v, g, s0, ds, 0.6)
    for a, b in zip(auto, mine):
        assert float((a - b).abs().max()) < 1e-11
    h = 1e-6
    for i, x in enumerate((q, k, v, g, s0)):
        for at in range(0, x.numel(), 7):
            args = [y.clone() for y in (q, k, v, g, s0)]
            args[i].view(-1)[at] += h
            up = loss(*args)
            args[i].view(-1)[at] -= 2 * h
            num = (up - loss(*args)) / (2 * h)
            assert abs(float(num - mine[i].reshape(-1)[at])) < 1e-6 * (1 + abs(float(num)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [32, 64])
def test_stream_of_blocks(d, dtype):
    """Blocks of one to many tokens against the carried state equal one call, and save = 0 leaves the state alone."""
    B, H, lens = 2, 3, [1, 1, 16, 17, 2, 33, 64, 300, 5, 4, 9, 8]
    N = sum(lens)
    q, k, v, g, s0 = make(11, B, N, H, d, dtype)
    state = s0.clone()
    outs, t = [], 0
    for L in lens:
        blk = [x[:, t:t + L].contiguous() for x in (q, k, v, g)]
        keep = state.clone()
        tried = lcla.gated_step(*blk, state, False)
        assert torch.equal(state, keep)
        nxt = torch.empty_like(state)
        aside = lcla.gated_step(*blk, state, True, state_out=nxt)
        assert torch.equal(state, keep)
        outs.append(lcla.gated_step(*blk, state, True))
        assert torch.equal(tried, outs[-1]) and torch.equal(aside, tried) and torch.equal(nxt, state)
        t += L
    r, rs, _ = ref_forward(q, k, v, g, s0, d ** -0.5)
    A, As, _ = ref_forward(mag(q), mag(k), mag(v), g, mag(s0), d ** -0.5)
    within(torch.cat(outs, 1), r, A, dtype, 16 if dtype == torch.bfloat16 else 17, "stream")
    within(state, rs, As, torch.float32, 17, "state")


def test_resets_pack_sequences():
    """A packed batch whose sequences begin with -inf equals its sequences one by one."""
    lens, H, d = [3, 40, 1, 200, 77], 2, 32
    q, k, v, g, _ = make(2, 1, sum(lens), H, d, torch.float32, False)
    at = 0
    for L in lens:
        g[:, at] = -math.inf
        at += L
    out, _ = lcla.gated_forward(q, k, v, g)
    at = 0
    for L in lens:
        one, _ = lcla.gated_forward(*(x[:, at:at + L].contiguous() for x in (q, k, v, g)))
        A, _, _ = ref_forward(*(mag(x[:, at:at + L]) for x in (q, k, v)), g[:, at:at + L], None, d ** -0.5)
        assert bool(((out[:, at:at + L] - one).abs().double() <= 2.0 ** -16 * A).all())
        at += L


def test_empty_sequence_copies_the_state():
    q = torch.empty(2, 0, 3, 32, device="cuda")
    g = torch.empty(2, 0, 3, device="cuda")
    s0 = torch.randn(2, 3, 32, 32, device="cuda")
    out, s1 = lcla.gated_forward(q, q, q, g, state_in=s0)
    assert out.shape == q.shape and torch.equal(s1, s0)
    assert float(lcla.gated_forward(q, q, q, g)[1].abs().max()) == 0.0
    *_, ds0 = lcla.gated_backward(q, q, q, q, g, dstate_out=s0, want_dstate_in=True)
    assert torch.equal(ds0, s0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [32, 64])
def test_rows_past_the_sequence_and_dirty_workspaces(d, dtype):
    """Outputs end where the sequence does, a workspace's old contents do not matter, and calls repeat bit for bit."""
    B, N, H = 1, 403, 5
    q, k, v, g, s0 = make(5, B, N, H, d, dtype)
    code = lcla.BF16 if dtype == torch.bfloat16 else lcla.F32
    do = torch.randn(B, N, H, d, device="cuda").to(dtype)
    n = N * H * d
    first = None
    for fill in (0, 255):
        bufs = [torch.full((n + 4096,), 7.0, device="cuda", dtype=dtype) for _ in range(4)]
        outs = [b[2048:2048 + n].view(B, N, H, d) for b in bufs]
        gbuf = torch.full((N * H + 256,), 7.0, device="cuda")
        dg = gbuf[128:128 + N * H].view(B, N, H)
        wf = torch.full((lcla.gated_forward_workspace_bytes(B, H, N, d, code) or 16,), fill, device="cuda", dtype=torch.uint8)
        wb = torch.full((lcla.gated_backward_workspace_bytes(B, H, N, d, code),), fill, device="cuda", dtype=torch.uint8)
        _, s1 = lcla.gated_forward(q, k, v, g, state_in=s0, out=outs[0], workspace=wf)
        *_, ds0 = lcla.gated_backward(do, q, k, v, g, state_in=s0, dstate_out=s0, out=(*outs[1:], dg), workspace=wb,
                                      want_dstate_in=True)
        for b in bufs:
            assert (b[:2048] == 7).all() and (b[2048 + n:] == 7).all()
        assert (gbuf[:128] == 7).all() and (gbuf[128 + N * H:] == 7).all()
        now = [o.clone() for o in outs] + [dg.clone(), s1, ds0]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_state_in_place():
    q, k, v, g, s0 = make(6, 1, 900, 3, 64, torch.bfloat16)
    out, s1 = lcla.gated_forward(q, k, v, g, state_in=s0)
    same = s0.clone()
    out2, s2 = lcla.gated_forward(q, k, v, g, state_in=same, state_out=same)
    assert s2 is same and torch.equal(s1, s2) and torch.equal(out, out2)


def test_graphs_and_streams():
    """Two captured graphs with workspaces of their own, replayed at once on two streams, and eager calls beside them."""
    sets = []
    for seed in (1, 2):
        q, k, v, g, s0 = make(seed, 1, 1500, 4, 32, torch.bfloat16)
        do = torch.randn_like(q)
        want = (*lcla.gated_forward(q, k, v, g, state_in=s0), *lcla.gated_backward(do, q, k, v, g, state_in=s0)[:4])
        want += (lcla.gated_step(q[:, :1].contiguous(), k[:, :1].contiguous(), v[:, :1].contiguous(),
                                 g[:, :1].contiguous(), s0.clone(), True),)
        sets.append((q, k, v, g, s0, do, want))
    torch.cuda.synchronize()
    graphs, got = [], []
    for q, k, v, g, s0, do, _ in sets:
        one = [x[:, :1].contiguous() for x in (q, k, v, g)]
        st = s0.clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = (*lcla.gated_forward(q, k, v, g, state_in=s0), *lcla.gated_backward(do, q, k, v, g, state_in=s0)[:4])
            st.copy_(s0)
            o += (lcla.gated_step(*one, st, True),)
        graphs.append(graph)
        got.append(o)
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    with torch.cuda.stream(torch.cuda.Stream()):
        eager = lcla.gated_forward(*sets[0][:4], state_in=sets[0][4])
    torch.cuda.synchronize()
    for o, s in zip(got, sets):
        assert all(torch.equal(a, b) for a, b in zip(o, s[6]))
    assert all(torch.equal(a, b) for a, b in zip(eager, sets[0][6]))


def test_memory_of_another_stream_is_not_reused():
    """Calls on a given stream, with memory made and dropped on the current one meanwhile."""
    q, k, v, g, s0 = make(12, 1, 4000, 6, 32, torch.bfloat16)
    want = lcla.gated_forward(q, k, v, g, state_in=s0)
    c, s = lcla.rotary_tables(4000, 32)
    wantn = lcla.qk_norm_rope(q, k, c, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        for _ in range(5):
            with torch.cuda.stream(side):
                torch.cuda._sleep(2000000)      # the call below waits behind this
            got = lcla.gated_forward(q, k, v, g, state_in=s0, stream=handle)
            gotn = lcla.qk_norm_rope(q, k, c, s, stream=handle)
            lcla.gated_backward(q, q, k, v, g, state_in=s0, stream=handle)      # dropped at once
            junk = [torch.full((n,), float("nan"), device="cuda") for n in (1 << 18, 1 << 20, 1 << 22)]
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((*got, *gotn), (*want, *wantn)))
            del junk


def test_offsets_beyond_32_bits():
    """More than 2^31 elements per tensor: the end of the sequence, from the state before it."""
    H, d, N, tail = 70, 32, 970000, 2051
    gen = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn(1, N, H, d, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    assert q.numel() > 1 << 31
    g = -torch.rand(1, N, H, generator=gen, device="cuda") * 0.05
    out, s1 = lcla.gated_forward(q, k, v, g)
    # a state of 2000 tokens back is forgotten to e^-50: the tail on its own, from a little earlier
    lead = 3000
    o2, s2 = lcla.gated_forward(*(x[:, N - tail - lead:].contiguous() for x in (q, k, v, g)))
    scale = float(o2.abs().max())
    assert float((out[:, N - tail:].float() - o2[:, lead:].float()).abs().max()) <= 2.0 ** -7 * scale
    assert float((s1 - s2).abs().max()) <= 1e-5 * float(s2.abs().max())
    do = v
    dq, dk, dv, dg, _ = lcla.gated_backward(do, q, k, v, g)
    e = lcla.gated_backward(*(x[:, N - tail - lead:].contiguous() for x in (do, q, k, v, g)))
    for a, b in zip((dq, dk, dv), e):
        assert float((a[:, N - tail:].float() - b[:, lead:].float()).abs().max()) <= 2.0 ** -7 * float(b.abs().max())
    assert float((dg[:, N - tail:] - e[3][:, lead:]).abs().max()) <= 1e-4 * float(e[3].abs().max())


def test_layer():
    """Tables, norm with rotation, recurrence and both gradients in a row, against autograd of the whole in 64 bits.

    fp32 throughout: every stage is within 2^-17 of its terms' magnitudes; sums of random signs are some 30 times
    smaller than those at these sizes and three stages follow each other, hence 2^-10 of the largest entry."""
    B, N, H, d = 2, 150, 3, 32
    gen = torch.Generator(device="cuda").manual_seed(8)
    qkv = torch.randn(B, N, 3 * H * d, generator=gen, device="cuda")
    q, k, v = (qkv[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3))
    wq, wk = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda") for _ in range(2))
    g = torch.nn.functional.logsigmoid(torch.randn(B, N, H, generator=gen, device="cuda") + 3)
    do = torch.randn(B, N, H, d, generator=gen, device="cuda")
    c, s = lcla.rotary_tables(N, [8, 12, 12], extents=[5, 10])
    qn, kn = lcla.qk_norm_rope(q, k, c, s, q_weight=wq, k_weight=wk)
    vc = v.contiguous()
    out, _ = lcla.gated_forward(qn, kn, vc, g)
    dqn, dkn, dv, dg, _ = lcla.gated_backward(do, qn, kn, vc, g)
    dqkv = torch.empty_like(qkv)
    parts = [dqkv[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3)]
    _, _, dwq, dwk = lcla.qk_norm_rope_backward(dqn, dkn, q, k, c, s, q_weight=wq, k_weight=wk, out=tuple(parts[:2]))
    parts[2].copy_(dv)

    x, a, b, gg = (t.double().requires_grad_() for t in (qkv, wq, wk, g))
    cc, ss = c.double()[None, :, None], s.double()[None, :, None]

    def norm(y, w):
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w
        e, o = y[..., 0::2], y[..., 1::2]
        return torch.stack([e * cc - o * ss, e * ss + o * cc], -1).flatten(-2)

    qr, kr, vr = (x[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3))
    G = gg.cumsum(1)
    w = torch.where(torch.ones(N, N, device="cuda").tril().bool()[None, :, :, None],
                    (G[:, :, None] - G[:, None]).clamp(max=0).exp(), 0.0)
    sc = torch.einsum("bthd,bshd->btsh", norm(qr, a), norm(kr, b)) * w * d ** -0.5
    o = torch.einsum("btsh,bshd->bthd", sc, vr)
    ref = torch.autograd.grad((o * do.double()).sum(), (x, a, b, gg))
    for name, m, r in (("out", out, o.detach()), ("dqkv", dqkv, ref[0]), ("dwq", dwq, ref[1]), ("dwk", dwk, ref[2]),
                       ("dg", dg, ref[3])):
        assert float((m.double() - r).abs().max()) <= 2.0 ** -10 * float(r.abs().max()), name
