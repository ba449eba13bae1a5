"""fp64 CPU oracle of the state-space operators (test infrastructure): plain
numpy, token by token, from the definitions; it shares no code with the CUDA
side. Backward passes are the chain rule of each definition, written apart
from the kernels' forms (the scan keeps every state).

Layouts as in include/wkv_ssm.h; every array is widened to float64.
"""

from __future__ import annotations

import numpy as np


def _f64(*arrays):
    return [None if a is None else np.asarray(a, dtype=np.float64) for a in arrays]


def _sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def silu(x):
    return x * _sigmoid(x)


def dsilu(x):
    p = _sigmoid(x)
    return p + x * p * (1 - p)


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


# ---- short causal convolution ------------------------------------------------------

def _conv_pre(x, weight, bias, x_prev):
    W = weight.shape[0]
    B, T, C = x.shape
    before = np.zeros((B, W - 1, C)) if x_prev is None else x_prev
    ext = np.concatenate([before, x], axis=1)
    pre = np.zeros((B, T, C)) + (0 if bias is None else bias)
    for t in range(T):
        for j in range(W):
            pre[:, t] += weight[j] * ext[:, t + j]
    return pre, ext


def conv_forward(x, weight, bias=None, x_prev=None, act=True):
    x, weight, bias, x_prev = _f64(x, weight, bias, x_prev)
    pre, _ = _conv_pre(x, weight, bias, x_prev)
    return silu(pre) if act else pre


def conv_backward(x, weight, gy, bias=None, x_prev=None, act=True):
    """(gx, gweight, gbias, gx_prev)"""
    x, weight, gy, bias, x_prev = _f64(x, weight, gy, bias, x_prev)
    W = weight.shape[0]
    pre, ext = _conv_pre(x, weight, bias, x_prev)
    gpre = gy * dsilu(pre) if act else gy
    gext, gw = np.zeros_like(ext), np.zeros_like(weight)
    for t in range(x.shape[1]):
        for j in range(W):
            gext[:, t + j] += weight[j] * gpre[:, t]
            gw[j] += (gpre[:, t] * ext[:, t + j]).sum(0)
    return gext[:, W - 1:], gw, gpre.sum((0, 1)), gext[:, :W - 1]


# ---- per-head norm with rotation --------------------------------------------------------

def _turn(v, angle, R, interleaved):
    """v [B, T, H, K], angle [B, T, R/2]."""
    out = v.copy()
    c, s = np.cos(angle)[:, :, None], np.sin(angle)[:, :, None]
    i = np.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    out[..., a] = v[..., a] * c - v[..., b] * s
    out[..., b] = v[..., a] * s + v[..., b] * c
    return out


def norm_rotate(x, weight, inv_freq, positions, K, eps, interleaved):
    """One of q and k, [B, T, H*K]; positions [B, T]."""
    x, weight, inv_freq = _f64(x, weight, inv_freq)
    B, T, HK = x.shape
    v = x.reshape(B, T, HK // K, K)
    v = v / np.sqrt((v ** 2).mean(-1, keepdims=True) + eps) * (1 if weight is None else weight)
    R = 0 if inv_freq is None else 2 * len(inv_freq)
    if R:
        v = _turn(v, np.asarray(positions)[..., None] * inv_freq, R, interleaved)
    return v.reshape(B, T, HK)


def norm_rotate_backward(x, g, weight, inv_freq, positions, K, eps, interleaved):
    """(gx, gweight)"""
    x, g, weight, inv_freq = _f64(x, g, weight, inv_freq)
    B, T, HK = x.shape
    v, gv = x.reshape(B, T, HK // K, K), g.reshape(B, T, HK // K, K)
    R = 0 if inv_freq is None else 2 * len(inv_freq)
    if R:
        gv = _turn(gv, -np.asarray(positions)[..., None] * inv_freq, R, interleaved)
    s = np.sqrt((v ** 2).mean(-1, keepdims=True) + eps)
    gw = (gv * v / s).sum((0, 1, 2))
    gn = gv * (1 if weight is None else weight)
    # d(v/s) = dv/s - v/s^2 ds,  ds = mean(v dv)/s
    gx = gn / s - v / s ** 3 * (gn * v).mean(-1, keepdims=True)
    return gx.reshape(B, T, HK), gw


# ---- selective scan -----------------------------------------------------------------------

def _wide(m, C, N):
    """[B, T, G*N] -> [B, T, C, N]"""
    B, T, GN = m.shape
    G = GN // N
    return np.repeat(m.reshape(B, T, G, N), C // G, axis=2)


def scan_forward(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, init_state=None, dt_softplus=True, states=False):
    """(y, final state), or with `states` also every state [B, T, C, N]."""
    x, dt, A, Bm, Cm, D, z, dt_bias, init_state = _f64(x, dt, A, Bm, Cm, D, z, dt_bias, init_state)
    (B, T, C), N = x.shape, A.shape[1]
    d = dt + (0 if dt_bias is None else dt_bias)
    d = softplus(d) if dt_softplus else d
    Bw, Cw = _wide(Bm, C, N), _wide(Cm, C, N)
    h = np.zeros((B, C, N)) if init_state is None else init_state.copy()
    s, every = np.zeros((B, T, C)), np.zeros((B, T, C, N))
    for t in range(T):
        h = np.exp(d[:, t, :, None] * A) * h + (d[:, t] * x[:, t])[..., None] * Bw[:, t]
        every[:, t] = h
        s[:, t] = (Cw[:, t] * h).sum(-1)
    s = s + (0 if D is None else D * x)
    y = s if z is None else s * silu(z)
    return (y, h, every, s, d) if states else (y, h)


def scan_backward(x, dt, A, Bm, Cm, gy, D=None, z=None, dt_bias=None, init_state=None, g_final=None, dt_softplus=True):
    """dict of the gradients of every operand"""
    x, dt, A, Bm, Cm, gy, D, z, dt_bias, init_state, g_final = _f64(x, dt, A, Bm, Cm, gy, D, z, dt_bias, init_state,
                                                                   g_final)
    _, _, every, s, d = scan_forward(x, dt, A, Bm, Cm, D, z, dt_bias, init_state, dt_softplus, states=True)
    (B, T, C), N = x.shape, A.shape[1]
    G = Bm.shape[2] // N
    Bw, Cw = _wide(Bm, C, N), _wide(Cm, C, N)
    gs = gy if z is None else gy * silu(z)
    gh = np.zeros((B, C, N)) if g_final is None else g_final.copy()
    h0 = np.zeros((B, C, N)) if init_state is None else init_state
    out = {"gx": np.zeros_like(x), "gA": np.zeros_like(A), "gB": np.zeros_like(Bm), "gC": np.zeros_like(Cm)}
    gd = np.zeros_like(x)
    fold = lambda m: m.reshape(B, G, C // G, N).sum(2).reshape(B, G * N)  # noqa: E731
    for t in range(T - 1, -1, -1):
        prev = every[:, t - 1] if t else h0
        a = np.exp(d[:, t, :, None] * A)
        out["gC"][:, t] = fold(gs[:, t, :, None] * every[:, t])
        gh = gh + gs[:, t, :, None] * Cw[:, t]
        out["gB"][:, t] = fold(gh * (d[:, t] * x[:, t])[..., None])
        gb = (gh * Bw[:, t]).sum(-1)
        out["gx"][:, t] = gb * d[:, t] + (0 if D is None else gs[:, t] * D)
        gd[:, t] = gb * x[:, t] + (gh * prev * a * A).sum(-1)
        out["gA"] += (gh * prev * a * d[:, t, :, None]).sum(0)
        gh = gh * a
    raw = dt + (0 if dt_bias is None else dt_bias)
    out["gdt"] = gd * _sigmoid(raw) if dt_softplus else gd
    out["gdt_bias"] = out["gdt"].sum((0, 1))
    out["gD"] = (gs * x).sum((0, 1))
    out["gz"] = None if z is None else gy * s * dsilu(z)
    out["g_init"] = gh
    return out
