"""What is measured of the gated linear attention operators: rotary tables, the
per-head norm of queries and keys with the rotation, and the gated recurrence
(whole sequence, step, gradient).

``run`` computes them from elementary torch operations, or through the package
where ``own`` is true.  Definitions (d = head dim, S fp32 [value][key] per head):

    S_t = exp(g_t) S_{t-1} + v_t k_t^T,   out_t = scale * S_t q_t
    y = R(x * rsqrt(mean(x^2) + eps) * w)
"""
import math

import torch

own = False

DEV = "cuda"
THETA = 10000.0
EPS = 1e-6
CHUNK = 64
FLOOR = -1000.0   # a log decay below this is a reset: exp underflows to zero


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the tables of a minute-scale video latent, 241 frames of 44 x 80 tokens, three axes
        dict(name="tables_minute", op="tables", N=241 * 44 * 80, dims="8,12,12", extents="44,80", first=0,
             scaling="none", factor=1.0, positions=False),
        # positions of a batch of long-context requests, scaled eightfold
        dict(name="tables_positions", op="tables", N=65536, dims="64", extents="", first=0,
             scaling="yarn", factor=8.0, positions=True),
        # one block's 480p latent, all heads
        dict(name="norm_480p", op="norm", B=1, N=32760, H=70, Hk=70, d=32, rd=32, half=False, dtype="bf16",
             positions=False, fused=False),
        # one token for each of 8 streams: latency
        dict(name="norm_token", op="norm", B=8, N=1, H=70, Hk=70, d=32, rd=32, half=False, dtype="bf16",
             positions=True, fused=False),
        # training at head dim 64: part of the head, half layout, read out of the fused projection
        dict(name="norm_grad_d64", op="norm_grad", B=2, N=4680, H=35, Hk=35, d=64, rd=32, half=True, dtype="bf16",
             positions=False, fused=True),
        dict(name="norm_grad_f32", op="norm_grad", B=1, N=3001, H=16, Hk=4, d=128, rd=128, half=False, dtype="f32",
             positions=False, fused=False),
        # 480p and streaming-latent sequences in one call
        dict(name="gated_480p", op="gated", B=1, N=32760, H=70, d=32, dtype="bf16", state=False, resets=False),
        dict(name="gated_stream", op="gated", B=2, N=63960, H=70, d=32, dtype="bf16", state=True, resets=True),
        dict(name="gated_f32_d64", op="gated", B=2, N=3001, H=5, d=64, dtype="f32", state=True, resets=False),
        # one token of 64 streams against their states: serving
        dict(name="gated_token", op="gated_step", B=64, N=1, H=35, d=64, dtype="bf16", state=True, resets=False),
        # a training batch's gradient at head dim 64, and an odd fp32 one with carried states and resets
        dict(name="gated_grad_d64", op="gated_grad", B=2, N=4680, H=35, d=64, dtype="bf16", state=False, resets=False),
        dict(name="gated_grad_f32", op="gated_grad", B=1, N=5003, H=16, d=32, dtype="f32", state=True, resets=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "norm", "norm_grad", "gated", "gated", "gated_step", "gated_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "tables":
        dims, extents = rng.choice([("8,12,12", "%d,%d" % (rng.randint(3, 44), rng.randint(3, 80))),
                                    ("16,24,24", "%d,%d" % (rng.randint(3, 44), rng.randint(3, 80))),
                                    ("32", ""), ("64", ""), ("128", "")])
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return dict(op=op, N=_log(rng, 1000, 200000), dims=dims, extents=extents, first=rng.randint(0, 500000),
                    scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 3.5]),
                    positions=rng.random() < 0.4)
    if op in ("norm", "norm_grad"):
        d = rng.choice([32, 64, 64, 96, 128])
        H = rng.randint(1, 40)
        rd = rng.choice([d, d, 32, 16])
        rows = _log(rng, 16 if op == "norm" else 2000, 300000)
        B = rng.choice([1, 1, 2, 3])
        return dict(op=op, B=B, N=max(1, rows // (B * H)), H=H, Hk=rng.choice([H, max(1, H // 4)]), d=d, rd=rd,
                    half=rng.random() < 0.5, dtype=dtype, positions=rng.random() < 0.5, fused=rng.random() < 0.5)
    d = rng.choice([32, 64])
    H = rng.randint(1, 70)
    if op == "gated_step":
        return dict(op=op, B=_log(rng, 1, 64), N=rng.choice([1, 1, 1, 2, 5, 17]), H=H, d=d, dtype=dtype, state=True,
                    resets=rng.random() < 0.3)
    B = rng.choice([1, 1, 2, 3])
    rows = _log(rng, 4000, 1500000 if op == "gated" else 250000) * 32 // d
    N = max(1, min(rows // (B * H), 20000))
    return dict(op=op, B=B, N=N, H=H, d=d, dtype=dtype, state=rng.random() < 0.5, resets=rng.random() < 0.3)


# ---------------------------------------------------------------- inputs
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _ints(text):
    return [int(x) for x in text.split(",") if x]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 1000003 + 17)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device=DEV) * scale

    op, st = case["op"], dict(case=case)
    if op == "tables":
        dims = _ints(case["dims"])
        # an input of every call: where the tokens stand
        if case["positions"]:
            st["positions"] = torch.randint(0, 1 << 20, (len(dims), case["N"]), generator=gen, device=DEV)
            st["first"] = 0
        else:
            st["positions"], st["first"] = None, case["first"] + 7919 * (seed % 1009)
        return st
    if op in ("norm", "norm_grad"):
        B, N, H, Hk, d, rd = (case[x] for x in ("B", "N", "H", "Hk", "d", "rd"))
        dt = _dt(case)
        if case["fused"]:
            qkv = normal(B, N, (H + 2 * Hk) * d, scale=1.7).to(dt)
            st["q"] = qkv[..., :H * d].unflatten(-1, (H, d))
            st["k"] = qkv[..., H * d:(H + Hk) * d].unflatten(-1, (Hk, d))
        else:
            st["q"], st["k"] = normal(B, N, H, d, scale=1.7).to(dt), normal(B, N, Hk, d, scale=0.6).to(dt)
        st["wq"], st["wk"] = 1.0 + normal(d, scale=0.2), 1.0 + normal(d, scale=0.2)
        P = max(N, 4096) if case["positions"] else N
        freq = THETA ** (-torch.arange(0, rd, 2, device=DEV, dtype=torch.float64) / rd)
        ang = torch.arange(P, device=DEV, dtype=torch.float64)[:, None] * freq
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        st["positions"] = torch.randint(0, P, (B, N), generator=gen, device=DEV) if case["positions"] else None
        if op == "norm_grad":
            st["gq"], st["gk"] = normal(B, N, H, d).to(dt), normal(B, N, Hk, d).to(dt)
        return st
    B, N, H, d = (case[x] for x in ("B", "N", "H", "d"))
    dt = _dt(case)
    st["q"], st["k"], st["v"] = (normal(B, N, H, d).to(dt) for _ in range(3))
    # heads forget at different rates, from tens to thousands of tokens
    bias = torch.linspace(2.5, 8.0, H, device=DEV)
    g = torch.nn.functional.logsigmoid(normal(B, N, H) + bias)
    if case["resets"]:   # a new sequence of the pack begins here
        g = torch.where(torch.rand(B, N, 1, generator=gen, device=DEV) < 1.0 / 700, -math.inf, g)
    st["g"] = g
    st["scale"] = d ** -0.5
    st["s0"] = normal(B, H, d, d, scale=3.0) if case["state"] else None
    if op == "gated_step":
        st["next"] = torch.empty_like(st["s0"])   # two buffers that a stream's states move between
    if op == "gated_grad":
        st["do"] = normal(B, N, H, d).to(dt)
        st["ds"] = normal(B, H, d, d, scale=0.5) if case["state"] else None
    return st


# ---------------------------------------------------------------- plain forms
def _frequencies(D, case):
    j = torch.arange(0, D, 2, device=DEV, dtype=torch.float64)
    s, theta = case["factor"], THETA
    if case["scaling"] == "ntk":
        theta = THETA * s ** (D / (D - 2))
    f = theta ** (-j / D)
    if case["scaling"] == "linear":
        f = f / s
    if case["scaling"] == "yarn":   # rotations over the original 4096 positions decide what is interpolated
        gamma = ((4096 * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * (gamma + (1 - gamma) / s)
    return f


def _tables(st):
    case = st["case"]
    dims, ext, N = _ints(case["dims"]), _ints(case["extents"]), case["N"]
    pos = st["positions"]
    if pos is None:
        n = st["first"] + torch.arange(N, device=DEV)
        pos = torch.stack([n // (ext[0] * ext[1]), n // ext[1] % ext[0], n % ext[1]]) if ext else n[None]
    ang = torch.cat([pos[a].double()[:, None] * _frequencies(D, case) for a, D in enumerate(dims)], dim=1)
    amp = 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "yarn" else 1.0
    return (ang.cos() * amp).float(), (ang.sin() * amp).float()


def _turn(x, c, s, half, back=False):
    """The rotation of the first 2 * c.shape[-1] entries of each row, or its transpose."""
    rd = 2 * c.shape[-1]
    if back:
        s = -s
    a, b = (x[..., :rd // 2], x[..., rd // 2:rd]) if half else (x[..., :rd:2], x[..., 1:rd:2])
    ra, rb = a * c - b * s, a * s + b * c
    r = torch.cat([ra, rb], -1) if half else torch.stack([ra, rb], -1).flatten(-2)
    return torch.cat([r, x[..., rd:]], -1)


def _rows(st):
    c, s = st["cos"], st["sin"]
    if st["positions"] is not None:
        return c[st["positions"]][:, :, None], s[st["positions"]][:, :, None]
    return c[None, :, None], s[None, :, None]


def _norm(st, x, w):
    x = x.float()
    c, s = _rows(st)
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    return _turn(n, c, s, st["case"]["half"]).to(_dt(st["case"]))


def _norm_grad(st, x, w, gy):
    x = x.float()
    c, s = _rows(st)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    gn = _turn(gy.float(), c, s, st["case"]["half"], back=True)
    gw = (gn * x * r).double().sum((0, 1, 2)).float()
    wg = gn * w
    gx = r * wg - x * r ** 3 * (wg * x).mean(-1, keepdim=True)
    return gx.to(_dt(st["case"])), gw


def _recur(q, k, v, g, s0):
    """Unscaled outputs [B,H,N,d] and the last state, in chunks: q, k, v fp32 [B,H,N,d], g fp64 [B,H,N]."""
    B, H, N, d = q.shape
    nc = -(-N // CHUNK)
    pad = nc * CHUNK - N
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)).reshape(B, H, nc, CHUNK, d) for x in (q, k, v))
    g = torch.nn.functional.pad(g, (0, pad)).reshape(B, H, nc, CHUNK)
    G = g.cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, device=DEV, dtype=torch.bool).tril()
    w = torch.where(low, (G[..., :, None] - G[..., None, :]).clamp(max=0).exp().float(), 0.0)
    out = ((q @ k.transpose(-1, -2)) * w) @ v
    # what each chunk adds to the state, and the state before each chunk
    add = v.transpose(-1, -2) @ (k * (G[..., -1:] - G).exp().float()[..., None])
    T = torch.nn.functional.pad(G[..., -1].cumsum(-1), (1, 0))             # decay up to chunk i, [B,H,nc+1]
    if s0 is None:
        s0 = torch.zeros(B, H, d, d, device=DEV)
    terms = torch.cat([s0[:, :, None], add], 2).flatten(-2)                # the carried state counts as chunk -1
    upto = torch.ones(nc + 1, nc + 1, device=DEV, dtype=torch.bool).tril()
    W = torch.where(upto, (T[..., :, None] - T[..., None, :]).clamp(max=0).exp().float(), 0.0)
    states = (W @ terms).unflatten(-1, (d, d))
    out = out + (q * G.exp().float()[..., None]) @ states[:, :, :nc].transpose(-1, -2)
    return out.reshape(B, H, nc * CHUNK, d)[:, :, :N], states[:, :, nc]


def _heads(x):
    return x.float().transpose(1, 2)


def _gated(st):
    q, k, v = (_heads(st[x]) for x in "qkv")
    g = st["g"].transpose(1, 2).double().clamp(min=FLOOR)
    out, s1 = _recur(q, k, v, g, st["s0"])
    return (out * st["scale"]).transpose(1, 2).to(_dt(st["case"])).contiguous(), s1


def _gated_grad(st):
    q, k, v, do = (_heads(st[x]) for x in ("q", "k", "v", "do"))
    g = st["g"].transpose(1, 2).double().clamp(min=FLOOR)
    do = do * st["scale"]
    s0t = None if st["s0"] is None else st["s0"].transpose(-1, -2)
    dq, s1t = _recur(do, v, k, g, s0t)
    back = torch.cat([g[..., 1:], torch.zeros_like(g[..., :1])], -1).flip(-1)
    ds = st["ds"]
    dv, r = _recur(k.flip(2), q.flip(2), do.flip(2), back, ds)
    dk, _ = _recur(v.flip(2), do.flip(2), q.flip(2), back, None if ds is None else ds.transpose(-1, -2))
    dk, dv = dk.flip(2), dv.flip(2)
    each = (q.double() * dq).sum(-1) - (k.double() * dk).sum(-1)
    dg = each.flip(-1).cumsum(-1).flip(-1)
    if ds is not None:
        dg = dg + (s1t.transpose(-1, -2).double() * ds).sum((-1, -2))[..., None]
    ds0 = r * g[..., 0].exp().float()[..., None, None]
    dt = _dt(st["case"])
    back_out = [x.transpose(1, 2).to(dt).contiguous() for x in (dq, dk, dv)]
    return (*back_out, dg.transpose(1, 2).float().contiguous(), ds0)


# ---------------------------------------------------------------- run
def run(st):
    case, op = st["case"], st["case"]["op"]
    if own:
        import block_causal_relu_b200 as lcla
        if op == "tables":
            ext = _ints(case["extents"])
            return lcla.rotary_tables(case["N"], _ints(case["dims"]), extents=ext or None, first=st["first"],
                                      positions=st["positions"], theta=THETA, scaling=case["scaling"],
                                      factor=case["factor"], original_len=4096, device=DEV)
        if op == "norm":
            return lcla.qk_norm_rope(st["q"], st["k"], st["cos"], st["sin"], q_weight=st["wq"], k_weight=st["wk"],
                                     eps=EPS, positions=st["positions"], half_layout=case["half"])
        if op == "norm_grad":
            return lcla.qk_norm_rope_backward(st["gq"], st["gk"], st["q"], st["k"], st["cos"], st["sin"],
                                              q_weight=st["wq"], k_weight=st["wk"], eps=EPS,
                                              positions=st["positions"], half_layout=case["half"])
        if op == "gated":
            return lcla.gated_forward(st["q"], st["k"], st["v"], st["g"], st["scale"], state_in=st["s0"])
        if op == "gated_step":
            out = lcla.gated_step(st["q"], st["k"], st["v"], st["g"], st["s0"], True, st["scale"], state_out=st["next"])
            return out, st["next"]
        return lcla.gated_backward(st["do"], st["q"], st["k"], st["v"], st["g"], st["scale"], state_in=st["s0"],
                                   dstate_out=st["ds"], want_dstate_in=True)
    if op == "tables":
        return _tables(st)
    if op == "norm":
        return _norm(st, st["q"], st["wq"]), _norm(st, st["k"], st["wk"])
    if op == "norm_grad":
        gq, gwq = _norm_grad(st, st["q"], st["wq"], st["gq"])
        gk, gwk = _norm_grad(st, st["k"], st["wk"], st["gk"])
        return gq, gk, gwq, gwk
    if op == "gated":
        return _gated(st)
    if op == "gated_step":
        out, s1 = _gated(st)
        st["next"].copy_(s1)
        return out, st["next"]
    return _gated_grad(st)


def work(case):
    op = case["op"]
    if op == "tables":
        dims = _ints(case["dims"])
        b = case["N"] * sum(dims) * 4 + (case["N"] * len(dims) * 8 if case["positions"] else 0)
        return dict(bytes=b, flops=case["N"] * sum(dims) * 8)
    esz = 2 if case["dtype"] == "bf16" else 4
    if op in ("norm", "norm_grad"):
        B, N, H, Hk, d, rd = (case[x] for x in ("B", "N", "H", "Hk", "d", "rd"))
        n = B * N * (H + Hk) * d
        tab = (min(B * N, 4096) if case["positions"] else N) * rd * 4
        return dict(bytes=n * esz * (2 if op == "norm" else 3) + tab + (B * N * 8 if case["positions"] else 0),
                    flops=n * (8 if op == "norm" else 16))
    B, N, H, d = (case[x] for x in ("B", "N", "H", "d"))
    n, s = B * N * H, B * H * d * d * 4
    if op == "gated_grad":
        return dict(bytes=n * (7 * d * esz + 8) + s * (3 if case["state"] else 1), flops=n * 10 * d * d)
    return dict(bytes=n * (4 * d * esz + 4) + s * (2 if case["state"] else 1), flops=n * 4 * d * d)


# ---------------------------------------------------------------- 64 bits, from the definitions
def _exact_turn(x, ang, half, rd):
    z = torch.complex(x[..., :rd // 2], x[..., rd // 2:rd]) if half else \
        torch.view_as_complex(x[..., :rd].unflatten(-1, (-1, 2)).contiguous())
    z = z * ang
    r = torch.cat([z.real, z.imag], -1) if half else torch.view_as_real(z).flatten(-2)
    return torch.cat([r, x[..., rd:]], -1)


def _exact_norm(st, x, w, gy=None):
    case, x, w = st["case"], x.double(), w.double()
    cis = torch.complex(st["cos"].double(), st["sin"].double())
    cis = (cis[st["positions"].flatten()].reshape(case["B"], case["N"], -1) if st["positions"] is not None
           else cis.expand(case["B"], -1, -1)).unsqueeze(2)
    ms = x.square().sum(-1, keepdim=True) / case["d"] + EPS
    if gy is None:
        return _exact_turn(x / ms.sqrt() * w, cis, case["half"], case["rd"])
    gn = _exact_turn(gy.double(), cis.conj(), case["half"], case["rd"])
    h = x / ms.sqrt()
    return (gn * w - h * (gn * w * h).sum(-1, keepdim=True) / case["d"]) / ms.sqrt(), (gn * h).sum((0, 1, 2))


def _exact_gated(st, grad):
    case = st["case"]
    q, k, v, g = (st[x].double() for x in ("q", "k", "v", "g"))
    B, N, H, d = q.shape
    a = g.exp()
    S = torch.zeros(B, H, d, d, device=DEV, dtype=torch.float64) if st["s0"] is None else st["s0"].double()
    if not grad:
        out = torch.empty_like(q)
        for t in range(N):
            S = S * a[:, t, :, None, None] + v[:, t, :, :, None] * k[:, t, :, None, :]
            torch.matmul(S, q[:, t, :, :, None], out=out[:, t, :, :, None])
        return out * case["d"] ** -0.5, S
    before = torch.empty(N, B, H, d, d, device=DEV, dtype=torch.float64)
    do = st["do"].double() * case["d"] ** -0.5
    dq, dk, dv, dg = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q), torch.empty_like(g)
    for t in range(N):
        before[t] = S
        S = S * a[:, t, :, None, None] + v[:, t, :, :, None] * k[:, t, :, None, :]
        dq[:, t] = (do[:, t, :, None, :] @ S).squeeze(-2)
    R = torch.zeros_like(S) if st["ds"] is None else st["ds"].double()
    for t in range(N - 1, -1, -1):
        R = R + do[:, t, :, :, None] * q[:, t, :, None, :]
        dk[:, t] = (v[:, t, :, None, :] @ R).squeeze(-2)
        dv[:, t] = (R @ k[:, t, :, :, None]).squeeze(-1)
        R = R * a[:, t, :, None, None]
        dg[:, t] = (R * before[t]).sum((-1, -2))
    return dq, dk, dv, dg, R


def exact(case, seed):
    op = case["op"]
    if op in ("gated", "gated_step", "gated_grad"):
        if case["N"] > 70000 or (op == "gated_grad" and case["B"] * case["N"] * case["H"] * case["d"] ** 2 > 2.5e9):
            return None
        return _exact_gated(prepare(case, seed), op == "gated_grad")
    st = prepare(case, seed)
    if op == "norm":
        return _exact_norm(st, st["q"], st["wq"]), _exact_norm(st, st["k"], st["wk"])
    if op == "norm_grad":
        (gq, gwq), (gk, gwk) = _exact_norm(st, st["q"], st["wq"], st["gq"]), _exact_norm(st, st["k"], st["wk"], st["gk"])
        return gq, gk, gwq, gwk
    pos = st["positions"]
    dims, ext = _ints(case["dims"]), _ints(case["extents"])
    cols = []
    for axis, D in enumerate(dims):
        if pos is not None:
            p = pos[axis].double()
        else:
            n = torch.arange(st["first"], st["first"] + case["N"], device=DEV)
            inner = math.prod(ext[axis:])
            p = torch.div(n, inner, rounding_mode="floor")
            p = (p % ext[axis - 1] if axis else p).double()
        for j in range(D // 2):
            base = THETA * case["factor"] ** (D / (D - 2)) if case["scaling"] == "ntk" else THETA
            f = math.exp(-2.0 * j / D * math.log(base))
            if case["scaling"] == "linear":
                f /= case["factor"]
            if case["scaling"] == "yarn":
                turns = 4096 * f / (2 * math.pi)
                keep = min(1.0, max(0.0, (turns - 1.0) / 31.0))
                f = f * keep + f / case["factor"] * (1.0 - keep)
            cols.append(torch.polar(torch.ones_like(p), p * f))
    amp = 1.0 + math.log(case["factor"]) / 10 if case["scaling"] == "yarn" else 1.0
    cis = torch.stack(cols, 1) * amp
    return cis.real, cis.imag
