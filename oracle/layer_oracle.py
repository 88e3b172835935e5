"""Float64 oracle of the operators around the attention (numpy): norms of
queries and keys with the position rotation, the gated linear recurrence, both
with their gradients, and decoding from a shared prefix.

Written from the formulas; it shares no code with the library.
"""
from __future__ import annotations

import numpy as np

from . import taylor_oracle as T


# ------------------------------------------------------- norms with rotation

def rotation(pos, freqs, d: int, interleaved: bool) -> np.ndarray:
    """R(pos) as matrices [..., d, d] for positions [...]."""
    pos = np.asarray(pos, dtype=np.float64)
    R = np.broadcast_to(np.eye(d), pos.shape + (d, d)).copy()
    half = len(freqs)
    for j, f in enumerate(np.asarray(freqs, dtype=np.float64)):
        i, k = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        c, s = np.cos(pos * f), np.sin(pos * f)
        R[..., i, i], R[..., i, k], R[..., k, i], R[..., k, k] = c, -s, s, c
    return R


def norm_rope(x, freqs, pos, w=None, interleaved=False, eps=0.0) -> np.ndarray:
    """x [B, N, H, d], pos [B, N] -> y [B, H, N, d]; a row of zeros with eps 0 gives zeros."""
    x = np.asarray(x, dtype=np.float64)
    u = x * _inv(x, eps)
    if w is not None:
        u = u * np.asarray(w, dtype=np.float64)
    R = rotation(pos, freqs, x.shape[-1], interleaved)
    return np.einsum("bnij,bnhj->bhni", R, u)


def _inv(x, eps):
    s = (x * x).sum(-1, keepdims=True) + eps
    return np.where(s > 0, 1.0 / np.sqrt(np.where(s > 0, s, 1.0)), 0.0)


def norm_rope_grad(x, dy, freqs, pos, w=None, interleaved=False, eps=0.0):
    """(dx [B, N, H, d], dw [d]) from dy [B, H, N, d]."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    w = np.ones(d) if w is None else np.asarray(w, dtype=np.float64)
    R = rotation(pos, freqs, d, interleaved)
    du = np.einsum("bnij,bhni->bnhj", R, np.asarray(dy, dtype=np.float64))
    inv = _inv(x, eps)
    unit = x * inv
    g = du * w
    return (g - unit * (unit * g).sum(-1, keepdims=True)) * inv, (du * unit).sum((0, 1, 2))


# ------------------------------------------------------- gated recurrence

def sigmoid(z):
    z = np.asarray(z, dtype=np.float64)
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def gated_scan(gate, x, coupled=True, h0=None, lengths=None):
    """h [B, N, D] (zero rows past a length) and the last state [B, D]."""
    gate, x = np.asarray(gate, dtype=np.float64), np.asarray(x, dtype=np.float64)
    B, N, D = gate.shape
    h, last = np.zeros((B, N, D)), np.zeros((B, D))
    for b in range(B):
        s = np.zeros(D) if h0 is None else np.asarray(h0[b], dtype=np.float64).copy()
        for t in range(N if lengths is None else min(int(lengths[b]), N)):
            a = sigmoid(gate[b, t])
            s = a * s + (sigmoid(-gate[b, t]) * x[b, t] if coupled else x[b, t])
            h[b, t] = s
        last[b] = s
    return h, last


def gated_scan_grad(gate, x, dh, coupled=True, h0=None, lengths=None, dh_last=None, h=None):
    """(dgate, dx, dh0); h, if given, is the forward's rounded output, which the
    gradient then takes for the states h_0..h_{N-1}."""
    gate, x, dh = (np.asarray(z, dtype=np.float64) for z in (gate, x, dh))
    B, N, D = gate.shape
    if h is None:
        h, _ = gated_scan(gate, x, coupled, h0, lengths)
    h = np.asarray(h, dtype=np.float64)
    dgate, dx, dh0 = np.zeros((B, N, D)), np.zeros((B, N, D)), np.zeros((B, D))
    for b in range(B):
        carry = np.zeros(D) if dh_last is None else np.asarray(dh_last[b], dtype=np.float64).copy()
        for t in reversed(range(N if lengths is None else min(int(lengths[b]), N))):
            a, keep = sigmoid(gate[b, t]), sigmoid(-gate[b, t])
            G = dh[b, t] + carry
            before = h[b, t - 1] if t else (np.zeros(D) if h0 is None else np.asarray(h0[b], dtype=np.float64))
            dgate[b, t] = G * (before - x[b, t] if coupled else before) * a * keep
            dx[b, t] = G * keep if coupled else G
            carry = G * a
        dh0[b] = carry
    return dgate, dx, dh0


# ------------------------------------------------------- shared prefix

def shared_prefix_decode(q, k, v, state, k_cache, v_cache, lengths, n: int, tau: float) -> np.ndarray:
    """One token per sequence: out [B, H, d_v].  state is the prefix's logical
    state [H, F, d_v + 1]; sequence b attends to the prefix, to its first
    lengths[b] cached tokens and to the new token."""
    q, k, v, state, k_cache, v_cache = (np.asarray(z, dtype=np.float64) for z in (q, k, v, state, k_cache, v_cache))
    B, H, d = q.shape
    phi = T.feature_map(q, n) * T.query_coeffs(d, n, tau)
    y = np.einsum("bhf,hfc->bhc", phi, state)
    for b in range(B):
        L = int(lengths[b])
        keys = np.concatenate([k_cache[b, :, :L], k[b, :, None]], 1)
        values = np.concatenate([v_cache[b, :, :L], v[b, :, None]], 1)
        w = T.taylor_kernel(tau * np.einsum("hld,hd->hl", keys, q[b]), n)
        y[b, :, :-1] += np.einsum("hl,hlc->hc", w, values)
        y[b, :, -1] += w.sum(-1)
    return y[..., :-1] / y[..., -1:]
