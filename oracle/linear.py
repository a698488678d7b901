"""fp64 numpy oracle of linear attention with a fixed decay per head, token by token, and of the query/key norm with
rotation -- TEST INFRASTRUCTURE, like the rest of this package.

Linear attention, per batch element and head:  S_t = a S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t,  a = exp(log_decay).
Backward of <dout, o> + <dST, S_T>, with G_t the gradient of S_t:  G_t = q_t dout_t^T + a G_{t+1} (from the end's dST),
dq_t = S_t dout_t,  dk_t = G_t v_t,  dv_t = G_t^T k_t,  dS_0 = a G_1.
"""
from __future__ import annotations

import numpy as np


def fwd(q, k, v, log_decay, S0=None):
    """q, k [B, T, H, Dk], v [B, T, H, Dv], log_decay [H]: (o, S_T)."""
    B, T, H, Dk = q.shape
    a = np.exp(log_decay)[None, :, None, None]
    S = np.zeros((B, H, Dk, v.shape[-1])) if S0 is None else S0.astype(np.float64).copy()
    o = np.zeros(v.shape)
    for t in range(T):
        S = a * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = np.einsum("bhkv,bhk->bhv", S, q[:, t])
    return o, S


def bwd(q, k, v, log_decay, dout, S0=None, dST=None):
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    a = np.exp(log_decay)[None, :, None, None]
    S = np.zeros((B, H, Dk, Dv)) if S0 is None else S0.astype(np.float64).copy()
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for t in range(T):
        S = a * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        dq[:, t] = np.einsum("bhkv,bhv->bhk", S, dout[:, t])
    G = np.zeros((B, H, Dk, Dv)) if dST is None else dST.astype(np.float64).copy()
    for t in range(T - 1, -1, -1):
        G = G + q[:, t, :, :, None] * dout[:, t, :, None, :]
        dk[:, t] = np.einsum("bhkv,bhv->bhk", G, v[:, t])
        dv[:, t] = np.einsum("bhkv,bhk->bhv", G, k[:, t])
        G = a * G
    return {"dq": dq, "dk": dk, "dv": dv, "dS0": G}


def _channels(pairs, interleaved):
    p = np.arange(pairs)
    return (2 * p, 2 * p + 1) if interleaved else (p, p + pairs)


def _angles(positions, inv_freq, axes):
    """[B, T, 1, pairs] from positions [A, B, T]. The product of a position (up to 40 bits) and a float32 (24 bits) is
    exact in 80-bit arithmetic; 2 pi to 64 bits then leaves turns * 2^-61 after the whole turns are taken off."""
    x = positions[axes].astype(np.longdouble) * inv_freq.astype(np.longdouble)[:, None, None]
    two_pi = 8 * np.arctan(np.longdouble(1))
    x = (x - np.rint(x / two_pi) * two_pi).astype(np.float64)
    return np.moveaxis(x, 0, -1)[:, :, None]


def _turn(x, t, pairs, interleaved):
    a, b = _channels(pairs, interleaved)
    y = x.copy()
    y[..., a] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t)
    y[..., b] = x[..., a] * np.sin(t) + x[..., b] * np.cos(t)
    return y


def rope_fwd(x, positions, inv_freq, axes, weight=None, eps=1e-6, interleaved=False):
    """x [B, T, H, D], positions [A, B, T], axes [pairs]; eps None: no norm."""
    n = x
    if eps is not None:
        n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if weight is None else weight)
    return _turn(n, _angles(positions, inv_freq, axes), len(inv_freq), interleaved)


def rope_bwd(x, dy, positions, inv_freq, axes, weight=None, eps=1e-6, interleaved=False):
    """(dx, dweight or None)."""
    d = _turn(dy, -_angles(positions, inv_freq, axes), len(inv_freq), interleaved)
    if eps is None:
        return d, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    w = np.ones(x.shape[-1]) if weight is None else weight
    dx = r * w * d - x * r ** 3 * (w * d * x).mean(-1, keepdims=True)
    return dx, (d * x * r).sum((0, 1, 2))
