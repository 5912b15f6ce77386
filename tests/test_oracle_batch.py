"""Pins of the batch oracle: brute force in Python floats, the shared-prefix identity, closed cases."""
import math

import numpy as np
import pytest

from oracle import attention as oatt
from oracle import batch as ob


def _rand(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("causal", [False, True])
def test_prefix_attention_brute_force(causal):
    B, T, Hq, Hkv, P, S, D = 3, 4, 4, 2, 5, 6, 8
    q, k, v = _rand(1, B, T, Hq, D), _rand(2, B, S, Hkv, D), _rand(3, B, S, Hkv, D)
    pk, pv = _rand(4, P, Hkv, D), _rand(5, P, Hkv, D)
    lens = [6, 2, 0]
    got, A = ob.prefix_attention(q, k, v, pk, pv, lens, causal, 0.3)
    for b in range(B):
        for t in range(T):
            for hq in range(Hq):
                h = hq // 2
                lim = lens[b] if not causal else min(max(lens[b] - T + t + 1, 0), lens[b])
                kv = [(pk[j, h], pv[j, h]) for j in range(P)] + [(k[b, j, h], v[b, j, h]) for j in range(lim)]
                e = [math.exp(0.3 * sum(float(x) * float(y) for x, y in zip(q[b, t, hq], kk))) for kk, _ in kv]
                for d in range(D):
                    ref = sum(w * float(vv[d]) for w, (_, vv) in zip(e, kv)) / sum(e)
                    mag = sum(w * abs(float(vv[d])) for w, (_, vv) in zip(e, kv)) / sum(e)
                    assert abs(got[b, t, hq, d] - ref) < 1e-12 and abs(A[b, t, hq, d] - mag) < 1e-12


def test_prefix_equals_the_joint_sequence():
    """With full lengths and no mask over the own keys, prefix + own is image rows over text + image."""
    T, H, P, D = 6, 2, 3, 128
    q, k, v = _rand(1, 1, T, H, D), _rand(2, 1, T, H, D), _rand(3, 1, T, H, D)
    pk, pv = _rand(4, P, H, D), _rand(5, P, H, D)
    got, _ = ob.prefix_attention(q, k, v, pk, pv, None, False, 1 / math.sqrt(D))
    full = oatt.attention_masked(np.concatenate([np.zeros((P, H, D)), q[0]]).astype(np.float32),
                                 np.concatenate([pk, k[0]]).astype(np.float32),
                                 np.concatenate([pv, v[0]]).astype(np.float32), P)
    assert np.abs(full.reshape(P + T, H, D)[P:] - got[0]).max() < 1e-5


def test_rows_without_keys_are_zero_and_lengths_clamp():
    q, k, v = _rand(1, 2, 3, 1, 8), _rand(2, 2, 4, 1, 8), _rand(3, 2, 4, 1, 8)
    none = np.zeros((0, 1, 8))
    o, _ = ob.prefix_attention(q, k, v, none, none, [2, -5], True, 1.0)
    assert (o[0, 0] == 0).all() and (o[1] == 0).all()       # row 0 of 3 with 2 keys; an empty sequence
    assert np.abs(o[0, 1, 0] - v[0, 0, 0]).max() < 1e-15    # one key: its value
    big, _ = ob.prefix_attention(q, k, v, none, none, [9, 4], False, 1.0)
    full, _ = ob.prefix_attention(q, k, v, none, none, None, False, 1.0)
    assert np.array_equal(big, full)


def test_add_rmsnorm_closed_cases():
    x = np.array([[3.0, 4.0, 0.0, 0.0]])
    s, y = ob.add_rmsnorm(x, None, None, 0.0, None)
    assert np.abs(y - x / 2.5).max() < 1e-15
    s, y = ob.add_rmsnorm(x, np.full((1, 4), 2.0 ** -20), 2.0, 0.0, lambda a: a.astype(np.float16))
    assert np.array_equal(s, x + [[0, 0, 2.0 ** -20, 2.0 ** -20]])  # 3 + 2^-20 rounds to 3 in fp16
    assert np.abs((y * y).mean() - 4.0) < 1e-12
