"""Oracle: operators of batches that share one prompt, in float64.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

* prefix_attention: sequence b's query rows attend to the P prefix keys, which all sequences
  share, and to the first lim of its own S keys: lim = own_len[b], or with `causal`
  own_len[b] - T + t + 1 for row t of T (the last row sees all own_len[b]), each clamped to
  0 .. own_len[b], own_len clamped to 0 .. S. Query heads hq use key head hq // (Hq // Hkv). A row
  without a key is zero.
* add_rmsnorm: the sum rounded to the stream's type, RMSNorm of it, the gain.
The 8-bit formats are those of oracle.mx.
"""
from __future__ import annotations

import numpy as np


def clamp_lens(own_len, B: int, S: int):
    n = np.full(B, S, np.int64) if own_len is None else np.asarray(own_len, np.int64)
    return np.clip(n, 0, S)


def limits(own_len, B: int, T: int, S: int, causal: bool):
    """Own keys visible to row t of sequence b: int64 [B, T]."""
    n = clamp_lens(own_len, B, S)[:, None]
    t = np.arange(T)[None, :]
    return np.clip(n - T + t + 1, 0, n) if causal else np.repeat(n, T, 1)


def weights(q, keys, scale, visible):
    """Softmax weights [T, n] of rows q [T, D] over keys [n, D]; zero where not visible [T, n] and in rows without a key."""
    s = np.where(visible, q @ keys.T * scale, -np.inf)
    top = s.max(1, keepdims=True, initial=-np.inf)
    e = np.where(visible, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
    tot = e.sum(1, keepdims=True)
    return e / np.where(tot > 0, tot, 1.0)


def prefix_attention(q, k, v, pk, pv, own_len, causal: bool, scale: float):
    """q [B, T, Hq, D], k, v [B, S, Hkv, D], pk, pv [P, Hkv, D] (any S, P >= 0) -> o [B, T, Hq, D] and
    A [B, T, Hq, D] = sum of weight x |value|, which error bounds are made of."""
    q, k, v, pk, pv = (np.asarray(x, np.float64) for x in (q, k, v, pk, pv))
    B, T, Hq, D = q.shape
    S, Hkv = k.shape[1], k.shape[2]
    P = pk.shape[0]
    lim = limits(own_len, B, T, S, causal)
    n = clamp_lens(own_len, B, S)
    o, A = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        vis = np.concatenate([np.ones((T, P), bool), np.arange(n[b])[None, :] < lim[b][:, None]], 1)
        for hq in range(Hq):
            h = hq // (Hq // Hkv)
            keys = np.concatenate([pk[:, h], k[b, :n[b], h]])
            vals = np.concatenate([pv[:, h], v[b, :n[b], h]])
            w = weights(q[b, :, hq], keys, scale, vis)
            o[b, :, hq] = w @ vals
            A[b, :, hq] = w @ np.abs(vals)
    return o, A


def add_rmsnorm(x, delta, gain, eps: float, round_to):
    """(x_out, y) float64: x_out = round_to(x + delta), y = x_out / sqrt(mean(x_out^2) + eps) * gain."""
    x = np.asarray(x, np.float64)
    if delta is not None:
        x = np.asarray(round_to(x + np.asarray(delta, np.float64)), np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x, x * r * (1.0 if gain is None else np.asarray(gain, np.float64))
