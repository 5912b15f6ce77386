"""The batch operators at the edges of their arithmetic. Helpers are those of test_gpu_batch."""
import numpy as np
import pytest

from oracle import mx as omx
from test_gpu_batch import _normal, _sf, qi  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("plus_one", [False, True])
def test_add_rmsnorm_of_gains_that_overflow(qi, plus_one):
    """An infinite y has the codes and the scale that the framework's quantiser gives an infinity, whether the
    gain is infinite or the product overflows; the other blocks of its row are those of a row without it."""
    import torch
    x = _normal(1, 5, 512, dtype="fp32")
    x[:, 70] = x[:, 70].abs() + 4.0                       # (y of this column passes 1 by far)
    x[2, 3] = 0.0                                         # 0 x inf is no number
    w = _normal(2, 512, dtype="fp32")
    bad = w.clone()
    bad[3], bad[40] = float("inf"), -float("inf")         # blocks 0 and 1
    bad[70] = torch.finfo(torch.float32).max              # block 2: finite, its product is not
    _, q, sf = qi.add_rmsnorm_mxfp8(x, None, bad, plus_one=plus_one)
    _, q0, sf0 = qi.add_rmsnorm_mxfp8(x, None, w, plus_one=plus_one)
    # the same with the quantiser: y as fp32 gives it, infinities as infinities of a 16-bit type
    y = torch.zeros(5, 512, dtype=torch.float16, device="cuda")
    y[:, 3] = torch.copysign(torch.tensor(float("inf")).cuda(), x[:, 3])
    y[:, 40] = -torch.copysign(torch.tensor(float("inf")).cuda(), x[:, 40])
    y[:, 70] = float("inf")
    y[2, 3] = float("nan")
    want, wsf = qi.quant_mxfp8(y.view(torch.int16), bf16=False)
    e, we, e0 = (_sf(s, 5, 512) for s in (sf, wsf, sf0))
    for col, blk in ((3, 0), (40, 1), (70, 2)):
        assert np.array_equal(e[[0, 1, 3, 4], blk], we[[0, 1, 3, 4], blk])
        assert torch.equal(q[:, col] & 127, want[:, col] & 127)
    rows = torch.tensor([0, 1, 3, 4]).cuda()
    for col in (3, 40, 70):
        assert torch.equal(q[rows, col], want[rows, col])
    assert np.array_equal(e[:, 3:], e0[:, 3:]) and torch.equal(q[:, 96:], q0[:, 96:])


@pytest.mark.parametrize("rows", [3, 320])                # 512 and 128 threads a row
@pytest.mark.parametrize("K", [384, 4096, 12288, 16384])
@pytest.mark.parametrize("kind", ["normal", "alike", "plain"])
def test_add_rmsnorm_of_a_dominant_channel(qi, kind, K, rows):
    """Rows whose one channel is thousands of times the rest (or, plain, has none): codes and scales are
    those of y within 2^-24. The mean square is a sum of pairs of squares, each with two roundings of at most
    2^-24 (relative, all terms >= 0), from there on with error terms (2^-47 and less): within 2^-23, and y,
    its inverse root, within 2^-24. Gains put every y next to a border between two codes, so that a mean that
    is further off shows; the y that lie nearer to their border than that (with 2 % of room) are left out."""
    import torch
    rng = np.random.default_rng(K)
    x = rng.standard_normal(K).astype(np.float32)
    if kind == "alike":
        x = np.full(K, np.sqrt(3.9), np.float32) * np.where(rng.random(K) < 0.5, -1, 1).astype(np.float32)
    if kind != "plain":
        x[5] = 8192.0
    r = 1.0 / np.sqrt((x.astype(np.float64) ** 2).mean() + 1e-6)
    mid = rng.choice([1.0625, 3.125, 17.0, 19.0, 136.0], K)     # between codes of a block of scale 1
    off = np.exp2(rng.uniform(-24, -20, K)) * np.where(rng.random(K) < 0.5, -1, 1)
    y = mid * (1 + off)
    y[::32] = 300.0                                              # fixes each block's scale
    w = (y / (x * r)).astype(np.float32)
    y = x * r * w.astype(np.float64)
    (lo, le), (hi, he) = (omx.quantize(y[None] * (1 + s * 1.02 * 2.0 ** -24)) for s in (-1, 1))
    sure = omx.dequantize(lo, le) == omx.dequantize(hi, he)
    assert np.array_equal(le, he) and 0.6 < sure.mean() < 1
    xs = torch.from_numpy(np.tile(x, (rows, 1))).cuda()
    _, q, sf = qi.add_rmsnorm_mxfp8(xs, None, torch.from_numpy(w).cuda())
    e = _sf(sf, rows, K).astype(np.int64) - 127
    assert (e == le).all()
    val = omx.dequantize(omx.E4M3_TABLE[q.cpu().numpy()], e)
    off_by = (val != omx.dequantize(lo, le)) & sure
    assert not off_by.any(), f"{off_by[0].sum()} of {K} codes off"
