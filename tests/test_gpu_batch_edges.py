"""The batch operators at the edges of their arithmetic. Helpers are those of test_gpu_batch."""
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import batch as ob
from oracle import mx as omx
from test_gpu_batch import _normal, _np, _sf, qi  # noqa: F401
from test_gpu_batch_use import KINDS, _case

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


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("B,T,Hq,Hkv,P,S", [(1, 1, 4, 2, 9000, 20), (2, 40, 2, 1, 9000, 64), (24, 1, 8, 2, 6000, 50),
                                            (2, 5, 3, 1, 700, 6000), (1, 200, 1, 1, 300, 7000)])
def test_attention_behind_keys_that_take_all(qi, B, T, Hq, Hkv, P, S, bits):
    """fp16: a few keys of every row have about 2^26 times the weight of each other one and the value zero
    (sinks); the output is what the thousands of others leave. A probability enters the product as w 2^7 or
    more, w its ratio to the row's largest, in fp16: one below 2^-21 is off by at most 2^-25 2^-7 = 2^-32, n keys
    by n 2^-32 max|v| over the sum, at least 0.7 of the number of sinks (in 8 bits 14.25 becomes 14: 2^-0.45 of
    the weight); the other terms are those of the bound in test_gpu_batch."""
    import torch
    q = _normal(1, B, T, Hq, 128, std=0.05)
    k, v = _normal(2, B, S, Hkv, 128, std=0.05), _normal(3, B, S, Hkv, 128, std=0.1) + 1
    pk, pv = _normal(4, P, Hkv, 128, std=0.05), _normal(5, P, Hkv, 128, std=0.1) + 1
    q[..., 7] = 14.25                                    # 14.25^2 / sqrt(128) log2 e = 25.9
    sinks = 0
    for key, val, rows in ((pk, pv, P), (k.transpose(0, 1), v.transpose(0, 1), S)):
        key[..., 7] = 0
        at = [i for i in range(rows) if i % 1024 in (3, 67, 131, 195)]   # in each half of two tiles in eight
        key[at], val[at] = 0, 0
        key[at, ..., 7] = 14.25
        sinks += len(at)
    kw = dict(prefix_k=pk, prefix_v=pv)
    if bits == 8:
        cache = qi.kv8_write(qi.kv8_cache(1, P, Hkv), pk[None], pv[None])
        kw = dict(prefix8=cache.prefix(0, P))
        pk, pv = (t[0] for t in qi.kv8_read(cache, P, torch.float16))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = _np(qi.prefix_attention(q, k, v, status=status, **kw))
    assert status.item() == 0
    args = [_np(x) for x in (q, k, v, pk, pv)]
    scale = 1 / np.sqrt(128)
    ref, A = ob.prefix_attention(*args, None, False, scale)
    n, vmax = P + S, max(np.abs(args[2]).max(), np.abs(args[4]).max())
    mag = scale * np.abs(args[0]).max() * 14.25 + scale * 128 * 0.3 * 0.3   # a score's sum of magnitudes, at most
    tol = (2.0 ** -11 * (A + np.abs(ref)) * (1 + 2.0 ** -8) + 2 * (mag * (128 * 2.0 ** -23 + 3 * 2.0 ** -24) + 2.0 ** -22) * A
           + (2 * n * 2.0 ** -23 + 8 * 2.0 ** -22) * A + n * 2.0 ** -32 * vmax / (0.7 * sinks) + 2.0 ** -25)
    assert (tol < 0.1 * np.abs(ref).max()).all()         # (the tail is far above what the bound allows)
    err = np.abs(o - ref)
    assert (err <= tol).all(), f"max error {err.max():.3e}, {(err / tol).max():.2f} of the bound"


# few rows joined in a cluster, with partials from codes; 128 rows joined
@pytest.mark.parametrize("kind,bits", [(0, 16), (1, 8), (5, 8)])
def test_an_expired_wait_is_told(qi, kind, bits):
    """A launch that waits for bytes of Q that never come gives up after its limit of two seconds a wait. Without a
    status word the check tells, once; with one the word does, and the check has nothing to say. What follows
    runs as before."""
    import torch
    a = _case(qi, KINDS[kind], 3, bits=bits)
    want = qi.prefix_attention(**a)
    qi.prefix_attention_check()
    st = torch.cuda.Stream()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    qi.debug_inject(3)
    qi.prefix_attention(stream=st, **a)
    with pytest.raises(qi.QiError, match="DEVICE_TIMEOUT"):
        qi.prefix_attention_check(st)
    qi.prefix_attention_check(st)
    qi.debug_inject(3)
    qi.prefix_attention(status=status, **a)
    assert status.item() != 0
    qi.prefix_attention_check()
    qi.debug_inject(3)
    qi.debug_inject(0)
    assert torch.equal(qi.prefix_attention(**a), want)
    qi.prefix_attention_check()


def test_the_first_call_of_a_process_captured(qi):
    """Nothing that the library does once per process or device stands in the way of a capture."""
    code = """
import torch, diffusion_transformer_text_gb300 as qi
q, k, v = (torch.randn(2, n, 4, 128, device="cuda").half() for n in (1, 50, 50))
pk = torch.randn(1, 300, 4, 128, device="cuda").half()
x = torch.randn(8, 512, device="cuda")
cache = qi.kv8_cache(1, 300, 4)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    qi.kv8_write(cache, pk, pk)
    got = [qi.prefix_attention(q, k, v, prefix8=cache.prefix(0, 300)), *qi.add_rmsnorm_mxfp8(x)]
g.replay()
torch.cuda.synchronize()
want = [qi.prefix_attention(q, k, v, prefix8=cache.prefix(0, 300)), *qi.add_rmsnorm_mxfp8(x)]
qi.prefix_attention_check()
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


@pytest.mark.parametrize("c", [dict(B=1, T=300, Hq=4, Hkv=2, P=140, S=300), dict(B=1, T=1, Hq=8, Hkv=2, P=2000, S=64),
                               dict(B=3, T=1, Hq=128, Hkv=1, P=30, S=70), dict(B=2, T=200, Hq=1, Hkv=1, P=50, S=200)])
def test_strides_of_dimensions_of_size_one(qi, c):
    """They are never followed, so they may be anything, and say nothing about where the outputs lie: on and
    off 32-byte boundaries the results are the same."""
    import torch
    a = _case(qi, c, 9)
    want = qi.prefix_attention(**a)
    for start in (0, 8):
        buf = torch.zeros(want.numel() + 16, dtype=want.dtype, device="cuda")
        for odd in (0, 3, 8, 2 ** 40):
            st = [odd if n == 1 else s for n, s in zip(want.shape, want.stride())]
            out = buf[start:].as_strided(want.shape, (*st[:3], 1))
            assert torch.equal(qi.prefix_attention(out=out, **a), want)
            assert buf[:start].count_nonzero() == 0 and buf[start + want.numel():].count_nonzero() == 0
            buf.zero_()


def test_threads_whose_errors_count(qi):
    """Four threads, each on a stream of its own, all operators: every round is compared, and an error in a
    thread is the test's."""
    import torch
    from concurrent.futures import ThreadPoolExecutor

    def together(a, x, kv):
        cache = qi.kv8_write(qi.kv8_cache(2, 64, 4), kv, kv)
        return (qi.prefix_attention(**a), *qi.add_rmsnorm_mxfp8(x), *cache, *qi.kv8_read(cache, 64, torch.bfloat16))

    work = [(_case(qi, c, 7 * i, bits=8 if i % 2 else 16), _normal(i, 40 + i, 1024, dtype="fp32"),
             _normal(i + 1, 2, 30 + i, 4, 128)) for i, c in enumerate(KINDS)]
    want = [together(*w) for w in work]
    torch.cuda.synchronize()

    def run(i):
        st = torch.cuda.Stream()
        same = 0
        for n in range(20):
            j = (i + n) % len(work)
            with torch.cuda.stream(st):
                got = together(*work[j])
            st.synchronize()
            same += all(torch.equal(g, w) for g, w in zip(got, want[j]))
            with pytest.raises(ValueError):               # a refusal is raised in its own thread
                qi.prefix_attention(work[j][0]["q"][..., :64], None, None)
        return same

    with ThreadPoolExecutor(4) as pool:
        assert [f.result(timeout=120) for f in [pool.submit(run, i) for i in range(4)]] == [20] * 4


@pytest.mark.parametrize("rows", [3, 700])
@pytest.mark.parametrize("with_delta", [False, True])
def test_norm_without_the_sum(qi, rows, with_delta):
    """The library's call with x_out = NULL: the same codes and scales, and x as it was."""
    import torch
    K = 512
    x, d, w = _normal(1, rows, K, dtype="fp32"), _normal(2, rows, K), _normal(3, K, dtype="bf16")
    d = d if with_delta else None
    _, q0, sf0 = qi.add_rmsnorm_mxfp8(x, d, w)
    q, sf, x0 = torch.zeros_like(q0), torch.zeros_like(sf0), x.clone()
    args = qi._NORM_HEAD.pack(x.data_ptr(), d.data_ptr() if with_delta else 0, 0, w.data_ptr(), q.data_ptr(), sf.data_ptr(), 0, 1e-6)
    args += qi._NORM_TAIL.pack(K, K, K, qi.DT_F32, qi.DT_F16, rows, K, 0)
    qi._check(qi.lib().qi_add_rmsnorm_mxfp8(args, torch.cuda.current_stream().cuda_stream))
    assert torch.equal(q, q0) and torch.equal(sf, sf0) and torch.equal(x, x0)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("B,T,Hq,Hkv,P,S", [(16, 1, 150, 150, 1000, 100), (4, 1, 200, 200, 1000, 20)])
def test_weights_of_few_rows_add_up_to_one(qi, B, T, Hq, Hkv, P, S, bits, dtype):
    """Blocks of at most 16 rows with several key tiles each, all values the same: so is every output, bit for
    bit, whatever the weights (some rows have most of theirs on one key of a later tile). Fp32 sums of terms of
    one sign: n / 16 < 70 product steps of at most 4 2^-23 each, n / 128 additions a thread and 20 joins, below
    2^-14 together; half a step of the types at a value just below 2 is 2^-12 of it or more."""
    import torch
    val = 2 - 2.0 ** (-10 if dtype == "fp16" else -7)
    q, k = _normal(1, B, T, Hq, 128, std=3.0, dtype=dtype), _normal(2, B, S, Hkv, 128, std=1.3, dtype=dtype)
    pk = _normal(3, P, Hkv, 128, std=1.3, dtype=dtype)
    if bits == 8:
        val = 1.75                                        # the largest code, 448, times 2^-8
        cache = qi.kv8_write(qi.kv8_cache(1, P, Hkv), pk[None], torch.full_like(pk[None], val))
        kw = dict(prefix8=cache.prefix(0, P))
    else:
        kw = dict(prefix_k=pk, prefix_v=torch.full_like(pk, val))
    o = qi.prefix_attention(q, k, torch.full_like(k, val), **kw)
    assert (o == val).all(), f"{(o != val).float().mean().item():.4f} of the outputs are not {val}"
