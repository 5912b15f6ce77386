"""Oracle: the operators of sequences in pages, in float64.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

* norm_rope: for every head x of 128, y = x / sqrt(mean(x^2) + eps) * gain (gain None: y = x); dims (2c, 2c + 1), or
  (c, c + C) with halves, turn by the angle a_c: (y_i cos a - y_j sin a, y_j cos a + y_i sin a); the others are y.
* angles: position on the pair's axis times its frequency.
* paged_attention: row i of sequence b lies at row i % R of page table[b, i // R]; query row t < q_len[b] sees rows
  j < lim, lim = kv_len, or kv_len - q_len + t + 1 with `causal`, clamped to 0 .. kv_len. A row without a key is zero;
  a page number that is none stands for a page of zeros.
"""
from __future__ import annotations

import numpy as np

from .batch import weights


def angles(pos, freqs, pairs):
    """pos [..., axes] integers, freqs [C] radians a position, pairs of each axis -> [..., C]."""
    axis = np.repeat(np.arange(len(pairs)), pairs)
    return np.asarray(pos, np.float64)[..., axis] * np.asarray(freqs, np.float64)


def frequencies(axes, theta: float):
    return np.concatenate([float(theta) ** (-2.0 * np.arange(d // 2) / d) for d in axes])


def partners(C: int, halves: bool, D: int = 128):
    """(first dims [C], second dims [C]) of the pairs."""
    c = np.arange(C)
    return (c, c + C) if halves else (2 * c, 2 * c + 1)


def norm_rope(x, gain, eps: float, a, halves: bool):
    """x [..., H, 128], a [..., C] -> (y rotated [..., H, 128], m [..., H, 128]: the magnitudes that errors scale with)."""
    x = np.asarray(x, np.float64)
    if gain is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    i, j = partners(a.shape[-1], halves)
    c, s = np.cos(a)[..., None, :], np.sin(a)[..., None, :]
    y, m = x.copy(), np.abs(x)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    m[..., i] = m[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    return y, m


def rows_of(pages, table, n: int):
    """Rows 0 .. n - 1 [n, H, D] of the sequence whose pages `table` [width] tells, from pages [pages, R, H, D]."""
    P, R = pages.shape[:2]
    out = np.zeros((n, *pages.shape[2:]), np.float64)
    for k in range(-(-n // R)):
        if 0 <= table[k] < P:
            part = pages[table[k], :min(R, n - k * R)]
            out[k * R:k * R + len(part)] = part
    return out


def paged_attention(q, k, v, table, kv_len, q_len, causal: bool, scale: float, max_len: int):
    """q [B, T, Hq, D], k, v [pages, R, Hkv, D] -> (o, A = sum of weight x |value|, mag = the largest sum of magnitudes
    of a row's scores [B, T, Hq], vmax [B, Hq], live [B, T]: rows that are computed)."""
    q = np.asarray(q, np.float64)
    B, T, Hq, D = q.shape
    G = Hq // k.shape[2]
    n = np.clip(np.asarray(kv_len, np.int64), 0, max_len)
    r = np.full(B, T) if q_len is None else np.clip(np.asarray(q_len, np.int64), 0, T)
    o, A = np.zeros(q.shape), np.zeros(q.shape)
    mag, vmax, live = np.zeros((B, T, Hq)), np.zeros((B, Hq)), np.arange(T)[None, :] < r[:, None]
    for b in range(B):
        if n[b] == 0 or r[b] == 0:
            continue
        keys, vals = rows_of(k, table[b], n[b]), rows_of(v, table[b], n[b])
        lim = np.clip(n[b] - r[b] + np.arange(r[b]) + 1, 0, n[b]) if causal else np.full(r[b], n[b])
        vis = np.arange(n[b])[None, :] < lim[:, None]
        for h in range(Hq):
            w = weights(q[b, :r[b], h], keys[:, h // G], scale, vis)
            o[b, :r[b], h] = w @ vals[:, h // G]
            A[b, :r[b], h] = w @ np.abs(vals[:, h // G])
            mag[b, :r[b], h] = scale * (np.abs(q[b, :r[b], h]) @ np.abs(keys[:, h // G]).T).max(1)
            vmax[b, h] = np.abs(vals[:, h // G]).max()
    return o, A, mag, vmax, live
