"""fp64 oracles of the operators around the scan: layer norm, rotary positions
and softmax attention, forward and backward, in plain numpy.

They share no code with the GPU path and are used by the tests only.
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------ layer norm
def layer_norm(x, weight=None, bias=None, eps=1e-6):
    """(y, mean, rstd) of rows x [..., C]."""
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def layer_norm_bwd(dy, x, weight=None, eps=1e-6):
    """(dx, dweight, dbias): the chain rule of layer_norm."""
    h, _, rstd = layer_norm(x, eps=eps)
    dy = np.asarray(dy, np.float64)
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = rstd[..., None] * (g - g.mean(-1, keepdims=True) - h * (g * h).mean(-1, keepdims=True))
    C = x.shape[-1]
    return dx, (dy * h).reshape(-1, C).sum(0), dy.reshape(-1, C).sum(0)


# ------------------------------------------------------------------ rotary
def rotary(x, pos, axes, theta=10000.0, halves=False, inverse=False):
    """x [T, H, D] turned by pos [P, A] (token t takes row t % P)."""
    x = np.array(x, np.float64)
    pos = np.asarray(pos, np.float64)
    R = sum(axes)
    out = x.copy()
    j = 0
    row = np.arange(x.shape[0]) % pos.shape[0]
    for a, d in enumerate(axes):
        for i in range(d // 2):
            ang = pos[row, a] * theta ** (-2.0 * i / d)
            c, s = np.cos(ang)[:, None], np.sin(ang)[:, None] * (-1 if inverse else 1)
            lo, hi = (j, j + R // 2) if halves else (2 * j, 2 * j + 1)
            out[..., lo] = x[..., lo] * c - x[..., hi] * s
            out[..., hi] = x[..., lo] * s + x[..., hi] * c
            j += 1
    return out


# ------------------------------------------------------------------ attention
def visible(lq, lk, causal, block=1):
    """Keys that each of the lq queries sees: the first n of the lk.  The
    queries are the last positions of the sequence."""
    n = np.full(lq, lk, np.int64)
    if causal:
        p = np.arange(lq) + (lk - lq)
        n = np.where(p < 0, 0, np.minimum(lk, (p // block + 1) * block))
    return n


def attention(q, k, v, causal=False, block=1, scale=None):
    """One sequence: q [lq, Hq, D], k and v [lk, Hk, D]; (o, lse)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    lq, Hq, D = q.shape
    lk, Hk, _ = k.shape
    scale = D ** -0.5 if scale is None else scale
    n = visible(lq, lk, causal, block)
    o, lse = np.zeros_like(q), np.full((lq, Hq), -np.inf)
    for h in range(Hq):
        kk, vv = k[:, h * Hk // Hq], v[:, h * Hk // Hq]
        for i in range(lq):
            if n[i] == 0:
                continue
            s = scale * (kk[:n[i]] @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            o[i, h] = (e @ vv[:n[i]]) / e.sum()
            lse[i, h] = m + np.log(e.sum())
    return o, lse


def attention_bwd(q, k, v, do, causal=False, block=1, scale=None):
    """(dq, dk, dv) of one sequence: with P the softmax and dP = do v^T,
    dS = P (dP - <do, o>), dq = scale dS k, dk = scale dS^T q, dv = P^T do."""
    q, k, v, do = (np.asarray(t, np.float64) for t in (q, k, v, do))
    lq, Hq, D = q.shape
    lk, Hk, _ = k.shape
    scale = D ** -0.5 if scale is None else scale
    n = visible(lq, lk, causal, block)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    hide = np.arange(lk)[None, :] >= n[:, None]
    for h in range(Hq):
        c = h * Hk // Hq
        s = scale * (q[:, h] @ k[:, c].T)
        s[hide] = -np.inf
        m = np.where(n > 0, s.max(-1, initial=-np.inf), 0.0)
        p = np.exp(s - m[:, None])
        t = p.sum(-1)
        p = p / np.where(t > 0, t, 1.0)[:, None]
        dp = do[:, h] @ v[:, c].T
        ds = p * (dp - (p * dp).sum(-1, keepdims=True))
        dq[:, h] = scale * (ds @ k[:, c])
        dk[:, c] += scale * (ds.T @ q[:, h])
        dv[:, c] += p.T @ do[:, h]
    return dq, dk, dv


# ------------------------------------------------------------------ 8-bit projections
def rms_norm(x, weight=None, residual=None, eps=1e-6):
    """(y, t) of rows x [..., C]: t = x + residual, y = t / rms(t) weight."""
    t = np.asarray(x, np.float64)
    if residual is not None:
        t = t + np.asarray(residual, np.float64)
    y = t / np.sqrt((t * t).mean(-1, keepdims=True) + eps)
    return (y if weight is None else y * np.asarray(weight, np.float64)), t


def group_scales(y, group=128):
    """Largest magnitude of each group of columns / 448."""
    C = y.shape[-1]
    m = np.stack([np.abs(y[..., c:c + group]).max(-1) for c in range(0, C, group)], -1)
    return np.maximum(m, 2.0 ** -100) / 448


def expand(scale, n, axis, group=128):
    return np.repeat(scale, group, axis=axis).take(np.arange(n), axis=axis)


def matmul(x, x_scale, w, w_scale):
    """y [M, N] of codes' values x [M, K], w [N, K] and their scales."""
    K, N = x.shape[1], w.shape[0]
    return (x * expand(x_scale, K, 1)) @ (w * expand(expand(w_scale, K, 1), N, 0)).T
