"""Rotary tables and the per-head norm with the rotation on the GPU, against
their formulas in 64 bits.

Tolerances.  An fp32 result of the norm and rotation passes through a sum of d
squares (a chain of 8 and log2(d / 8) tree steps), a reciprocal square root of
2 ulp, three products and a two-term rotation: below 24 roundings of 2^-24,
taken as 32 of the row's largest entry.  bf16 adds half a step, 2^-8 of the
value.  The weights' gradients add their terms' magnitudes times one rounding
per addition of the longest chain.  Table entries: Taylor remainders below 2e-9
and under four roundings of 2^-24 each, stated as 2e-7.
"""
import math

import pytest
import torch

import block_causal_relu_b200 as lcla

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def freqs(D, theta, scaling, factor, L0=4096, fast=32.0, slow=1.0):
    out = []
    for j in range(D // 2):
        base = theta * factor ** (D / (D - 2)) if scaling == "ntk" else theta
        f = base ** (-2.0 * j / D)
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            g = min(1.0, max(0.0, (L0 * f / (2 * math.pi) - slow) / (fast - slow)))
            f = f * g + f / factor * (1 - g)
        out.append(f)
    return out


def ref_tables(pos, dims, theta, scaling, factor):
    """Angles reduced in integers and 64 bits: pos * f is split so that no bits of far positions are lost."""
    cols = []
    for a, D in enumerate(dims):
        p = pos[a].cpu()
        hi, lo = (p >> 20).double() * 2.0 ** 20, (p & ((1 << 20) - 1)).double()
        for f in freqs(D, theta, scaling, factor):
            ah, al = hi * f, lo * f
            cols.append((torch.cos(ah) * torch.cos(al) - torch.sin(ah) * torch.sin(al),
                         torch.sin(ah) * torch.cos(al) + torch.cos(ah) * torch.sin(al)))
    amp = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
    return (torch.stack([c for c, _ in cols], 1) * amp, torch.stack([s for _, s in cols], 1) * amp)


@pytest.mark.parametrize("dims,extents,first,n", [
    ([32], None, 0, 1), ([32], None, 1 << 20, 777), ([8, 12, 12], [7, 11], 5, 1001), ([16, 24, 24], [30, 52], 999999, 513),
    ([2], None, 3, 5), ([6, 10], [9], 0, 100), ([256], None, 17, 33), ([128], None, (1 << 31) - 10, 40),
])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 3.5)])
def test_tables(dims, extents, first, n, scaling, factor):
    if scaling == "ntk" and 2 in dims:
        with pytest.raises(lcla.LclaError):
            lcla.rotary_tables(n, dims, extents=extents, first=first, scaling=scaling, factor=factor)
        return
    c, s = lcla.rotary_tables(n, dims, extents=extents, first=first, scaling=scaling, factor=factor)
    idx = first + torch.arange(n)
    pos = []
    for a in range(len(dims)):
        inner = math.prod((extents or [])[a:])
        p = idx // inner
        pos.append(p % extents[a - 1] if a else p)
    rc, rs = ref_tables(torch.stack(pos), dims, 10000.0, scaling, factor)
    assert float((c.double().cpu() - rc).abs().max()) < 2.4e-7      # amp <= 1.14 of 2e-7
    assert float((s.double().cpu() - rs).abs().max()) < 2.4e-7


def test_tables_positions_any_order_and_negative():
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-5000, 1 << 22, (3, 1234), generator=g)
    c, s = lcla.rotary_tables(1234, [8, 12, 12], positions=pos.cuda(), theta=500000.0)
    rc, rs = ref_tables(pos, [8, 12, 12], 500000.0, "none", 1.0)
    assert float((c.double().cpu() - rc).abs().max()) < 2e-7 and float((s.double().cpu() - rs).abs().max()) < 2e-7
    one = lcla.rotary_tables(1234, 32, positions=pos[0].cuda())[0]
    assert torch.equal(one, lcla.rotary_tables(1234, [32], positions=pos[:1].cuda())[0])


def test_tables_feed_the_forward():
    """The tables drive the block-causal forward as host-made ones do, streamed block by block at absolute positions."""
    B, N, H, L = 1, 400, 2, 100
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn(B, N, H, 32, generator=g, device="cuda") for _ in range(3))
    c, s = lcla.rotary_tables(N, [8, 12, 12], extents=[5, 10])
    whole, st = lcla.forward(q, k, v, c, s, L)
    state = torch.zeros(B, H, 33, 32, device="cuda")
    parts = []
    for i in range(0, N, L):
        ci, si = lcla.rotary_tables(L, [8, 12, 12], extents=[5, 10], first=i)
        assert torch.equal(ci, c[i:i + L]) and torch.equal(si, s[i:i + L])
        parts.append(lcla.step(*(x[:, i:i + L].contiguous() for x in (q, k, v)), ci, si, state, True))
    assert float((torch.cat(parts, 1) - whole).abs().max()) < 1e-4 * float(whole.abs().max())
    assert float((state - st).abs().max()) < 1e-5 * float(st.abs().max())


# ------------------------------------------------------------------ norm and rotation
def turn(x, c, s, half, rd):
    if half:
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        r = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        r = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([r, x[..., rd:]], -1)


def ref_norm(x, w, c, s, pos, half, eps):
    rd = 2 * c.shape[1]
    B, N = x.shape[:2]
    rows = pos.clamp(0, c.shape[0] - 1) if pos is not None else torch.arange(N, device=x.device).expand(B, N)
    cc, ss = c.double()[rows][:, :, None], s.double()[rows][:, :, None]
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return turn(n * w if w is not None else n, cc, ss, half, rd)


def make(seed, B, N, H, Hk, d, rd, dtype, fused, rows=None, weights=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *sh: torch.randn(*sh, generator=g, device="cuda")  # noqa: E731
    if fused:
        qkv = (r(B, N, (H + 2 * Hk) * d) * 2).to(dtype)
        q = qkv[..., :H * d].unflatten(-1, (H, d))
        k = qkv[..., H * d:(H + Hk) * d].unflatten(-1, (Hk, d)) if Hk else None
    else:
        q, k = (r(B, N, H, d) * 2).to(dtype), (r(B, N, Hk, d).to(dtype) if Hk else None)
    rows = rows or N
    ang = r(rows, rd // 2) * 3
    wq, wk = (1 + 0.3 * r(d), 1 + 0.3 * r(d)) if weights else (None, None)
    return q, k, ang.cos().contiguous(), ang.sin().contiguous(), wq, wk if Hk else None


def close(o, r, dtype, what):
    r = r.double()
    err = (o.double() - r).abs()
    lim = 32 * U32 * r.abs().amax(-1, keepdim=True) * math.sqrt(2)
    if dtype == torch.bfloat16:
        lim = lim + 2.0 ** -8 * r.abs() * (1 + 2.0 ** -8)
    worst = float((err - lim).max()) if err.numel() else -1.0
    assert worst <= 0, f"{what}: {worst:.3e} over its tolerance"


CASES = [  # B, N, H, Hk, d, rd, half, fused, positions
    (1, 1, 1, 1, 32, 32, False, False, False),
    (2, 7, 3, 1, 32, 32, True, True, True),
    (1, 130, 70, 70, 32, 32, False, False, False),
    (2, 33, 5, 2, 64, 32, True, True, True),
    (1, 19, 9, 9, 64, 6, False, False, True),      # rows of 3 table columns: no 16-byte pieces
    (3, 5, 4, 0, 96, 96, True, False, False),      # no keys; 12 of 16 lanes hold a row
    (1, 11, 2, 2, 128, 64, False, True, False),
    (2, 3, 3, 1, 256, 256, True, False, True),
    (1, 9, 2, 2, 8, 8, False, False, False),       # one lane of four holds a row
    (1, 21, 4, 4, 40, 0, False, False, False),     # the norm alone
    (1, 700, 40, 8, 64, 64, False, True, False),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,H,Hk,d,rd,half,fused,with_pos", CASES)
def test_norm_rope(B, N, H, Hk, d, rd, half, fused, with_pos, dtype):
    rows = 50 if with_pos else N
    q, k, c, s, wq, wk = make(d + N, B, N, H, Hk, d, rd, dtype, fused, rows)
    g = torch.Generator(device="cuda").manual_seed(1)
    pos = torch.randint(0, rows, (B, N), generator=g, device="cuda") if with_pos else None
    qo, ko = lcla.qk_norm_rope(q, k, c, s, q_weight=wq, k_weight=wk, eps=1e-5, positions=pos, half_layout=half)
    close(qo, ref_norm(q.double(), wq.double(), c, s, pos, half, 1e-5), dtype, "q")
    if Hk:
        close(ko, ref_norm(k.double(), wk.double(), c, s, pos, half, 1e-5), dtype, "k")
    # in place, in the buffer of the projection: the same bits
    if fused:
        q2, k2 = q, k
        lcla.qk_norm_rope(q2, k2, c, s, q_weight=wq, k_weight=wk, eps=1e-5, positions=pos, half_layout=half,
                          out=(q2, k2))
        assert torch.equal(q2, qo) and torch.equal(k2, ko)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,N,H,Hk,d,rd,half,fused,with_pos", CASES)
def test_norm_rope_gradient(B, N, H, Hk, d, rd, half, fused, with_pos, dtype):
    rows = 50 if with_pos else N
    q, k, c, s, wq, wk = make(d + N + 1, B, N, H, Hk, d, rd, dtype, fused, rows)
    g = torch.Generator(device="cuda").manual_seed(1)
    pos = torch.randint(0, rows, (B, N), generator=g, device="cuda") if with_pos else None
    gq = torch.randn(q.shape, generator=g, device="cuda").to(dtype)
    gk = torch.randn(k.shape, generator=g, device="cuda").to(dtype) if Hk else None
    got = lcla.qk_norm_rope_backward(gq, gk, q, k, c, s, q_weight=wq, k_weight=wk, eps=1e-5, positions=pos,
                                     half_layout=half)
    again = lcla.qk_norm_rope_backward(gq, gk, q, k, c, s, q_weight=wq, k_weight=wk, eps=1e-5, positions=pos,
                                       half_layout=half)
    for x, y in zip(got, again):
        assert x is y is None or torch.equal(x, y), "not the same bits twice"
    for x, gy, w, gx, gw in ((q, gq, wq, got[0], got[2]), (k, gk, wk, got[1], got[3])):
        if x is None:
            continue
        xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
        y = ref_norm(xd, wd, c, s, pos, half, 1e-5)
        rx, rw = torch.autograd.grad(y, (xd, wd), gy.double())
        # gx = r (w m - x r^2 mean(w m x)): its terms are as large as r |w| |gy| row by row
        r = 1 / torch.sqrt((xd * xd).mean(-1, keepdim=True) + 1e-5)
        size = (r * gy.double().abs().amax(-1, keepdim=True) * wd.abs().max() * math.sqrt(2) *
                (1 + (xd * r).abs().amax(-1, keepdim=True) * (xd * r).abs().mean(-1, keepdim=True))).detach()
        lim = 48 * U32 * size
        if dtype == torch.bfloat16:
            lim = lim + 2.0 ** -8 * rx.abs() * (1 + 2.0 ** -8)
        assert float(((gx.double() - rx).abs() - lim).max()) <= 0
        rows_added = B * N * x.shape[2]
        rows = pos if pos is not None else torch.arange(N, device="cuda").expand(B, N)
        # an entry of m is the sum of two products a c + b s that may cancel: its rounding goes by |a c| + |b s|,
        # which the turns of the magnitudes by +-|s| hold in one entry each
        mc, ms = c.double().abs()[rows][:, :, None], s.double().abs()[rows][:, :, None]
        back = torch.maximum(*(turn(gy.double().abs(), mc, sg * ms, half, rd).abs() for sg in (1, -1)))
        terms = (back * (xd * r).abs()).sum((0, 1, 2)).detach()
        chain = min(rows_added, 64 + rows_added // 256)
        assert float(((gw.double() - rw).abs() - (chain + 24) * U32 * terms).max()) <= 0


def test_formula_gradient_against_differences():
    q, _, c, s, wq, _ = make(5, 1, 3, 2, 0, 16, 8, torch.float32, False)
    x, w = q.double().requires_grad_(), wq.double().requires_grad_()
    assert torch.autograd.gradcheck(lambda a, b: ref_norm(a, b, c, s, None, True, 1e-5), (x, w))


def test_positions_outside_the_tables_are_clamped():
    q, k, c, s, wq, wk = make(2, 1, 6, 2, 2, 32, 32, torch.float32, False, rows=10)
    pos = torch.tensor([[-5, 0, 9, 10, 1 << 40, -(1 << 50)]], device="cuda")
    qo, _ = lcla.qk_norm_rope(q, k, c, s, q_weight=wq, positions=pos)
    close(qo, ref_norm(q.double(), wq.double(), c, s, pos, False, 1e-6), torch.float32, "clamped")


def test_rows_of_zeros_and_extremes():
    q = torch.zeros(1, 4, 2, 32, device="cuda")
    q[0, 1] = 1e18
    q[0, 2] = 1e-18
    q[0, 3, 0, 5] = float("inf")
    c, s = lcla.rotary_tables(4, 32)
    o, _ = lcla.qk_norm_rope(q, None, c, s, eps=1e-6)
    assert float(o[0, 0].abs().max()) == 0.0                      # a row of zeros stays zero with eps > 0
    assert torch.isfinite(o[0, :3]).all() and torch.isfinite(o[0, 3, 1]).all()   # inf stays in its own row
    assert abs(float(o[0, 1].square().mean()) - 1.0) < 1e-5


def test_no_tokens():
    q = torch.empty(2, 0, 3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    c, s = lcla.rotary_tables(0, 64)
    assert c.shape == (0, 32)
    qo, ko = lcla.qk_norm_rope(q, q, c, s, q_weight=w, k_weight=w)
    assert qo.shape == q.shape and ko.shape == q.shape
    *_, dw, dk = lcla.qk_norm_rope_backward(q, q, q, q, c, s, q_weight=w, k_weight=w)
    assert float(dw.abs().max()) == 0.0 and float(dk.abs().max()) == 0.0      # sums of nothing


def test_rows_around_the_output_are_left_alone():
    T, H, d = 37, 3, 64
    buf = torch.full((T + 2, 5 * d), 7.0, device="cuda", dtype=torch.bfloat16)
    out = buf[1:-1, d:4 * d].unflatten(-1, (H, d))[None]
    q, _, c, s, wq, _ = make(9, 1, T, H, 0, d, d, torch.bfloat16, False)
    lcla.qk_norm_rope(q, None, c, s, q_weight=wq, out=(out, None))
    close(out, ref_norm(q.double(), wq.double(), c, s, None, False, 1e-6), torch.bfloat16, "window")
    assert (buf[0] == 7).all() and (buf[-1] == 7).all() and (buf[:, :d] == 7).all() and (buf[:, 4 * d:] == 7).all()


def test_stream_and_graph():
    q, k, c, s, wq, wk = make(4, 2, 65, 5, 5, 64, 64, torch.bfloat16, False)
    want = lcla.qk_norm_rope(q, k, c, s, q_weight=wq, k_weight=wk)
    gq, gk = torch.randn_like(q), torch.randn_like(k)
    want_b = lcla.qk_norm_rope_backward(gq, gk, q, k, c, s, q_weight=wq, k_weight=wk)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = lcla.qk_norm_rope(q, k, c, s, q_weight=wq, k_weight=wk)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tabs = lcla.rotary_tables(65, 64, first=3)
        f = lcla.qk_norm_rope(q, k, c, s, q_weight=wq, k_weight=wk)
        b = lcla.qk_norm_rope_backward(gq, gk, q, k, c, s, q_weight=wq, k_weight=wk)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((*f, *b), (*want, *want_b)))
    assert torch.equal(tabs[0], lcla.rotary_tables(65, 64, first=3)[0])
