"""Float64 CPU oracle of the attention layer's operators, straight from their formulas (numpy; shares
no code with the GPU path).  Rows are [rows, heads, dim]; functions return whole arrays."""

from __future__ import annotations

import numpy as np


def _turn(x, positions, inv_freq, sign):
    a = len(inv_freq)
    theta = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(theta)[:, None], sign * np.sin(theta)[:, None]
    y = x.copy()
    y[..., :a] = x[..., :a] * c - x[..., a:2 * a] * s
    y[..., a:2 * a] = x[..., :a] * s + x[..., a:2 * a] * c
    return y


def norm_rope(x, weight, positions, inv_freq, eps):
    """Per-head RMS norm, then the rotation of the pairs (d, d + A)."""
    x = np.asarray(x, np.float64)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    return _turn(n, positions, inv_freq, 1.0)


def norm_rope_backward(g, x, weight, positions, inv_freq, eps):
    """(dx, dweight) of sum(g * norm_rope(x))."""
    x, w = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    u = _turn(np.asarray(g, np.float64), positions, inv_freq, -1.0)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dx = r * u * w - x * r ** 3 * (u * w * x).mean(-1, keepdims=True)
    return dx, (u * x * r).sum((0, 1))


def allowed(nq, nk, causal, window):
    """[nq, nk] truth values: which keys a query sees (the last query stands on the last key)."""
    i, j = np.arange(nq)[:, None] + (nk - nq), np.arange(nk)[None]
    ok = np.ones((nq, nk), bool)
    if causal:
        ok &= j <= i
        if window:
            ok &= j > i - window
    return ok


def probabilities(q, k, causal, window, scale):
    """One sequence: p [heads, nq, nk] and lse [nq, heads]; a row without keys has p = 0, lse = -inf."""
    q, k = np.asarray(q, np.float64), np.asarray(k, np.float64)
    k = np.repeat(k, q.shape[1] // k.shape[1], 1)
    z = np.einsum("ihd,jhd->hij", q, k) * scale
    z = np.where(allowed(q.shape[0], k.shape[0], causal, window), z, -np.inf)
    top = z.max(-1, initial=-np.inf, keepdims=True)
    e = np.exp(z - np.where(np.isinf(top), 0.0, top))
    total = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (top + np.log(total))[..., 0].T
    return e / np.where(total == 0, 1.0, total), lse


def attention(q, k, v, causal=True, window=0, scale=None):
    """One sequence: out [nq, heads, dim] and lse [nq, heads]."""
    scale = q.shape[2] ** -0.5 if scale is None else scale
    p, lse = probabilities(q, k, causal, window, scale)
    v = np.repeat(np.asarray(v, np.float64), q.shape[1] // v.shape[1], 1)
    return np.einsum("hij,jhd->ihd", p, v), lse


def attention_backward(dout, q, k, v, causal=True, window=0, scale=None):
    """One sequence: (dq, dk, dv) of sum(dout * attention(q, k, v))."""
    scale = q.shape[2] ** -0.5 if scale is None else scale
    groups, share = k.shape[1], q.shape[1] // k.shape[1]
    p, _ = probabilities(q, k, causal, window, scale)
    q, dout = np.asarray(q, np.float64), np.asarray(dout, np.float64)
    kk = np.repeat(np.asarray(k, np.float64), share, 1)
    vv = np.repeat(np.asarray(v, np.float64), share, 1)
    dp = np.einsum("ihd,jhd->hij", dout, vv)
    ds = p * (dp - (p * dp).sum(-1, keepdims=True)) * scale

    def shared(x):
        return x.reshape(x.shape[0], groups, share, x.shape[2]).sum(2)

    return (np.einsum("hij,jhd->ihd", ds, kk), shared(np.einsum("hij,ihd->jhd", ds, q)),
            shared(np.einsum("hij,ihd->jhd", p, dout)))
