"""Gated linear attention in fp64, token by token: rotary tables, the per-head
RMS norm with the rotation, the gated recurrence and its gradient.  Inputs are
float arrays or bf16 bits (uint16)."""
from __future__ import annotations

import math

import numpy as np


def widen(a):
    """bf16 bits or floats -> float64, exactly."""
    a = np.asarray(a)
    if a.dtype == np.uint16:
        return (a.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return a.astype(np.float64)


def tables(pos, dims, theta=10000.0, scaling="none", factor=1.0, original_len=4096, beta_fast=32.0, beta_slow=1.0):
    """(cos, sin) [N, sum(dims) / 2] of integer positions pos [axes][N]."""
    cols = []
    for p, D in zip(pos, dims):
        base = theta * factor ** (D / (D - 2)) if scaling == "ntk" else theta
        for j in range(D // 2):
            f = base ** (-2.0 * j / D)
            if scaling == "linear":
                f /= factor
            if scaling == "yarn":
                g = min(1.0, max(0.0, (original_len * f / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow)))
                f = f * (g + (1.0 - g) / factor)
            cols.append(np.asarray(p, np.float64) * f)
    ang = np.stack(cols, 1)
    amp = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
    return np.cos(ang) * amp, np.sin(ang) * amp


def norm_rope(x, w, cos, sin, half=False, eps=1e-6):
    """x [B, N, H, d]; tables [N, rd / 2]."""
    x = widen(x)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * np.asarray(w, np.float64)
    rd = 2 * cos.shape[1]
    c, s = (np.asarray(t, np.float64)[None, :, None] for t in (cos, sin))
    first, second = (slice(0, rd // 2), slice(rd // 2, rd)) if half else (slice(0, rd, 2), slice(1, rd, 2))
    a, b = y[..., first].copy(), y[..., second].copy()
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    return y


def forward(q, k, v, g, scale, state=None):
    """S_t = e^{g_t} S_{t-1} + v_t k_t^T, out_t = scale S_t q_t: (out, last state, states before each token)."""
    q, k, v = widen(q), widen(k), widen(v)
    a = np.exp(np.asarray(g, np.float64))
    B, N, H, d = q.shape
    S = np.zeros((B, H, d, d)) if state is None else np.asarray(state, np.float64)
    out, before = np.empty_like(q), np.empty((N, B, H, d, d))
    for t in range(N):
        before[t] = S
        S = S * a[:, t, :, None, None] + v[:, t, :, :, None] * k[:, t, :, None, :]
        out[:, t] = scale * np.einsum("bhce,bhe->bhc", S, q[:, t])
    return out, S, before


def backward(do, q, k, v, g, scale, state=None, dstate=None):
    """(dq, dk, dv, dg, dstate_in) of <out, do> + <last state, dstate>."""
    _, _, before = forward(q, k, v, g, scale, state)
    do, q, k, v = widen(do), widen(q), widen(k), widen(v)
    a = np.exp(np.asarray(g, np.float64))
    R = np.zeros(before.shape[1:]) if dstate is None else np.asarray(dstate, np.float64)
    dq, dk, dv, dg = np.empty_like(q), np.empty_like(q), np.empty_like(q), np.empty_like(a)
    for t in range(q.shape[1] - 1, -1, -1):
        decay = a[:, t, :, None, None]
        S = before[t] * decay + v[:, t, :, :, None] * k[:, t, :, None, :]
        R = R + scale * do[:, t, :, :, None] * q[:, t, :, None, :]
        dq[:, t] = scale * np.einsum("bhce,bhc->bhe", S, do[:, t])
        dk[:, t] = np.einsum("bhce,bhc->bhe", R, v[:, t])
        dv[:, t] = np.einsum("bhce,bhe->bhc", R, k[:, t])
        R = R * decay
        dg[:, t] = (R * before[t]).sum((-1, -2))
    return dq, dk, dv, dg, R
