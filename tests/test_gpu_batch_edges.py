"""The batch operators at the edges of their arithmetic. Helpers are those of test_gpu_batch."""
import numpy as np
import pytest

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
