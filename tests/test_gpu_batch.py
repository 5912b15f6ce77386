"""Operators of batches that share a prompt, against the float64 oracle on the same 16-bit inputs.

Attention bound, per output element, with u the half step of the 16-bit type relative to a value
(fp16 2^-11, bf16 2^-8), w the exact softmax weights and A = sum w |v|:
* each probability is rounded to the type once: at most u A, plus, in fp16, half a subnormal step
  2^-25 per key for probabilities below 2^-14 (relative to a sum that is at least 1): n 2^-25 max|v|;
* the output is rounded once: u |o|;
* a score's error ds changes a weight by the factor e^ds, numerator and denominator alike: 2 ds A. A
  score is 128 exact products summed in fp32 (at most 128 steps of 2^-23 of the sum of magnitudes,
  truncation allowed for), scaled, and 2^x adds 2^-22 relative and the rounding of its argument;
* P V and the row sum add up n terms in fp32: n 2^-23 A each; merging parts adds a few 2^-22.
"""
import math

import numpy as np
import pytest

from oracle import batch as ob
from oracle import mx as omx

pytestmark = pytest.mark.gpu

U = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def qi():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import diffusion_transformer_text_gb300 as q
    q.build()
    q.lib()
    return q


def _dt(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _normal(seed, *shape, std=1.0, dtype="fp16"):
    import torch
    a = np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * np.float32(std)
    return torch.from_numpy(a).to(_dt(dtype)).cuda()


def _np(t):
    return t.detach().double().cpu().numpy()


def _bound(q, k, v, pk, pv, lens, scale, ref, A, dtype):
    """The bound of the module's docstring, [B, T, Hq, 128]."""
    B, T, Hq, D = q.shape
    G = Hq // pk.shape[1]
    n = ob.clamp_lens(lens, B, k.shape[1])
    out = np.zeros(ref.shape)
    for b in range(B):
        for hq in range(Hq):
            keys = np.abs(np.concatenate([pk[:, hq // G], k[b, :n[b], hq // G]]))
            if not len(keys):
                continue
            vmax = max(np.abs(pv[:, hq // G]).max(initial=0), np.abs(v[b, :n[b], hq // G]).max(initial=0))
            mag = scale * (np.abs(q[b, :, hq]) @ keys.T).max(1, keepdims=True)     # largest sum of magnitudes of a score
            ds = mag * (128 * 2.0 ** -23 + 3 * 2.0 ** -24) + 2.0 ** -22
            a = A[b, :, hq]
            out[b, :, hq] = (U[dtype] * (a + np.abs(ref[b, :, hq])) * (1 + 2.0 ** -8) + 2 * ds * a
                             + (2 * len(keys) * 2.0 ** -23 + 8 * 2.0 ** -22) * a
                             + (len(keys) * 2.0 ** -25 * vmax if dtype == "fp16" else 0.0) + 2.0 ** -25)
    return out


def _spread(t, layout):
    """The tensor's values in another layout (same shape, other strides): heads outside rows, or rows far apart."""
    import torch
    if t is None or layout == "bshd":
        return t
    if layout == "bhsd":
        return t.transpose(-3, -2).contiguous().transpose(-3, -2)
    wide = torch.full((*t.shape[:-2], t.shape[-2] + 3, t.shape[-1]), float("nan"), dtype=t.dtype, device=t.device)
    wide[..., 1:-2, :] = t
    return wide[..., 1:-2, :]


def _check_attention(qi, B, T, Hq, Hkv, P, S, causal=False, lens=None, dtype="fp16", layout="bshd", bits=16, std=1.2,
                     seed=0, garbage=True):
    import torch
    q = _normal(seed + 1, B, T, Hq, 128, std=std, dtype=dtype)
    k, v = _normal(seed + 2, B, S, Hkv, 128, std=std, dtype=dtype), _normal(seed + 3, B, S, Hkv, 128, dtype=dtype)
    pk, pv = _normal(seed + 4, P, Hkv, 128, std=std, dtype=dtype), _normal(seed + 5, P, Hkv, 128, dtype=dtype)
    kw = {}
    if bits == 8:
        cache = qi.kv8_write(qi.kv8_cache(1, P, Hkv), pk[None], pv[None])
        kw["prefix8"] = cache.prefix(0, P)
        pk, pv = (t[0] for t in qi.kv8_read(cache, P, pk.dtype))
    elif P:
        kw["prefix_k"], kw["prefix_v"] = _spread(pk, layout), _spread(pv, layout)
    if lens is not None:
        kw["own_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if garbage:  # what lies behind a sequence may be anything
            for b, n in enumerate(ob.clamp_lens(lens, B, S)):
                k[b, n:], v[b, n:] = float("nan"), float("inf")
    scale = 1 / math.sqrt(128)
    own = {} if S == 0 else dict(k=_spread(k, layout), v=_spread(v, layout))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((B, T, Hq + 2, 128), 7.0, dtype=q.dtype, device="cuda")
    o = qi.prefix_attention(_spread(q, layout), own.get("k"), own.get("v"), causal=causal, out=out[:, :, 1:-1],
                            status=status, **kw)
    assert status.item() == 0
    assert (out[:, :, 0] == 7).all() and (out[:, :, -1] == 7).all()
    args = (_np(q), _np(k), _np(v), _np(pk), _np(pv))
    ref, A = ob.prefix_attention(*args, lens, causal, scale)
    err = np.abs(_np(o) - ref)
    tol = _bound(*args, lens, scale, ref, A, dtype)
    empty = (ob.limits(lens, B, T, S, causal) == 0) & (P == 0)
    assert (_np(o)[empty] == 0).all()
    assert (err <= tol).all(), f"max error {err.max():.3e}, {(err / tol).max():.2f} of the bound at {np.unravel_index((err / tol).argmax(), err.shape)}"


CASES = [
    dict(B=1, T=1, Hq=1, Hkv=1, P=1, S=1),
    dict(B=1, T=1, Hq=4, Hkv=4, P=22, S=17),
    dict(B=2, T=3, Hq=2, Hkv=2, P=0, S=1),                                        # no prefix
    dict(B=2, T=3, Hq=2, Hkv=1, P=130, S=0),                                      # no own keys
    dict(B=3, T=1, Hq=4, Hkv=2, P=0, S=40, lens=[0, 40, 7]),                      # an empty row, no prefix
    dict(B=3, T=5, Hq=3, Hkv=1, P=0, S=20, lens=[3, 0, 20], causal=True),         # rows before the first key
    dict(B=4, T=1, Hq=6, Hkv=2, P=127, S=129, lens=[1, 128, 129, 0], causal=True),
    dict(B=5, T=2, Hq=10, Hkv=2, P=128, S=70, lens=[70, 2, 1, 33, 64], causal=True, layout="bhsd"),
    dict(B=7, T=5, Hq=6, Hkv=2, P=129, S=33, lens=[33, 5, 6, 20, 33, 32, 31], causal=True, layout="wide"),
    dict(B=9, T=1, Hq=8, Hkv=1, P=300, S=140, lens=[140, 0, 1, 139, 128, 127, 129, 64, 65]),
    dict(B=2, T=1, Hq=128, Hkv=1, P=200, S=10),                                   # the largest group
    dict(B=2, T=43, Hq=3, Hkv=1, P=64, S=50, causal=True, lens=[50, 43]),         # 129 rows: just over one block
    dict(B=1, T=128, Hq=1, Hkv=1, P=5, S=128, causal=True),
    dict(B=2, T=129, Hq=2, Hkv=2, P=77, S=259, causal=True, lens=[259, 129]),
    dict(B=2, T=300, Hq=5, Hkv=1, P=0, S=300, causal=True, lens=[300, 180], layout="wide"),
    dict(B=1, T=260, Hq=2, Hkv=2, P=407, S=260, layout="bhsd"),
    dict(B=1, T=1, Hq=2, Hkv=1, P=5000, S=1300, lens=[1257], causal=True),        # split over the keys
    dict(B=20, T=1, Hq=4, Hkv=4, P=2000, S=30, causal=True, lens=list(range(1, 21))),
    dict(B=2, T=4, Hq=4, Hkv=2, P=9, S=12, lens=[2000000000, -7]),                # lengths are clamped
    # several units per block: codes after own tiles and the other way round, runs of one-tile units
    dict(B=16, T=1, Hq=32, Hkv=32, P=700, S=256, lens=[256 - 15 * i for i in range(16)], causal=True),
    dict(B=1, T=1, Hq=200, Hkv=200, P=300, S=300, lens=[290]),
    dict(B=40, T=1, Hq=8, Hkv=8, P=1, S=100, lens=[(37 * i) % 101 for i in range(40)]),
    dict(B=3, T=64, Hq=60, Hkv=60, P=100, S=64, lens=[64, 1, 40], causal=True),
    dict(B=30, T=20, Hq=12, Hkv=12, P=0, S=90, lens=[(31 * i) % 91 for i in range(30)]),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(c[n]) for n in ("B", "T", "Hq", "Hkv", "P", "S")))
def test_attention(qi, case, dtype):
    _check_attention(qi, dtype=dtype, seed=case["B"] * 100 + case["P"], **case)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", [c for c in CASES if c["P"] > 0][::2] + CASES[-5:-1], ids=lambda c: f"P{c['P']}-T{c['T']}-B{c['B']}")
def test_attention_8bit_prefix(qi, case, dtype):
    _check_attention(qi, dtype=dtype, bits=8, seed=case["B"] * 100 + case["P"], **case)


def test_attention_peaked_rows(qi):
    """Scores of a hundred and more: the running maximum moves and weights vanish."""
    _check_attention(qi, 2, 40, 2, 2, 300, 200, std=6.0, lens=[200, 77])
    _check_attention(qi, 4, 1, 8, 2, 3000, 200, std=6.0, lens=[200, 77, 1, 0], dtype="bf16")


def test_attention_random_shapes(qi):
    rng = np.random.default_rng(5)
    for i in range(12):
        Hkv, G = int(rng.integers(1, 4)), int(rng.integers(1, 9))
        B, T = int(rng.integers(1, 8)), int(rng.choice([1, 1, 2, 7, 30, 150]))
        P, S = int(rng.integers(1, 700)), int(rng.integers(1, 400))
        lens = [int(x) for x in rng.integers(0, S + 1, B)] if rng.random() < 0.7 else None
        _check_attention(qi, B, T, Hkv * G, Hkv, P, S, causal=bool(rng.random() < 0.5), lens=lens,
                         dtype=["fp16", "bf16"][i % 2], layout=["bshd", "bhsd", "wide"][i % 3], bits=[16, 8][i // 2 % 2],
                         seed=i)


def _batch(qi, B=6, T=1, Hq=8, Hkv=2, P=1500, S=200, seed=3):
    return (_normal(seed, B, T, Hq, 128), _normal(seed + 1, B, S, Hkv, 128), _normal(seed + 2, B, S, Hkv, 128),
            _normal(seed + 3, P, Hkv, 128), _normal(seed + 4, P, Hkv, 128))


@pytest.mark.parametrize("T", [1, 3, 200])
def test_attention_repeats_and_rows_are_independent(qi, T):
    """Bit for bit the same on a second call, and whatever the other sequences hold."""
    import torch
    q, k, v, pk, pv = _batch(qi, T=T)
    lens = torch.tensor([200, 0, 31, 128, 200, 1], dtype=torch.int32, device="cuda")
    a = qi.prefix_attention(q, k, v, pk, pv, own_len=lens, causal=True)
    assert torch.equal(a, qi.prefix_attention(q, k, v, pk, pv, own_len=lens, causal=True))
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    for x in (q2, k2, v2):
        x[[0, 1, 3, 4, 5]] = _normal(99, *x[[0, 1, 3, 4, 5]].shape)
    lens2 = lens.clone()
    lens2[[0, 3]] = torch.tensor([5, 77], dtype=torch.int32, device="cuda")
    b = qi.prefix_attention(q2, k2, v2, pk, pv, own_len=lens2, causal=True)
    assert torch.equal(a[2], b[2])


def test_attention_equals_the_block_causal_kernel_on_one_image(qi):
    """Image rows over stored text K/V: the framework's attention and this one, same inputs."""
    import torch
    L, N = 407, 600
    q, k, v = (_normal(i, L + N, 4096, std=1.3) for i in (1, 2, 3))
    i16 = lambda t: t.contiguous().view(torch.int16)
    ref = qi.attention(i16(q[L:]), i16(k), i16(v), L, q_off=L).view(torch.float16).float()
    h = lambda t: t.view(-1, 32, 128)
    o = qi.prefix_attention(h(q[L:])[None], h(k[L:])[None], h(v[L:])[None], h(k[:L]), h(v[:L]))
    # both round probabilities and outputs to fp16 once: each is within 2 u (1 + small) of the exact row
    A = h(v).float().abs().max()
    assert (o[0].float().reshape(N, -1) - ref).abs().max() <= 4.5 * 2.0 ** -11 * A


def test_attention_graph_with_growing_lengths(qi):
    """Captured once, replayed while the sequences grow: lengths are read when the kernels run."""
    import torch
    q, k, v, pk, pv = _batch(qi, S=300)
    lens = torch.zeros(6, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    qi.prefix_attention(q, k, v, pk, pv, own_len=lens, causal=True, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qi.prefix_attention(q, k, v, pk, pv, own_len=lens, causal=True, out=out)
    for n in (0, 1, 128, 129, 300):
        lens.fill_(n)
        lens[1] = 300 - n
        g.replay()
        got = out.clone()
        assert torch.equal(got, qi.prefix_attention(q, k, v, pk, pv, own_len=lens, causal=True))


def test_attention_on_two_streams_at_once(qi):
    import torch
    sets = [_batch(qi, seed=10 * i, P=2500) for i in range(2)]
    want = [qi.prefix_attention(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            got[i].append(qi.prefix_attention(*sets[i], stream=st))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_attention_refuses(qi):
    import torch
    q, k, v, pk, pv = _batch(qi)
    for bad in (dict(q=q[..., :64]), dict(q=q.float()), dict(k=k[:3]), dict(v=v.to(torch.bfloat16)),
                dict(v=v.cpu()), dict(pk=pk[:, :1]), dict(pv=None), dict(own_len=torch.zeros(5, dtype=torch.int32, device="cuda")),
                dict(own_len=torch.zeros(6, dtype=torch.int64, device="cuda")), dict(out=q[:, :, :4]),
                dict(k=k.transpose(2, 3).contiguous().transpose(2, 3)), dict(status=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        a = dict(q=q, k=k, v=v, pk=pk, pv=pv)
        a.update({n: x for n, x in bad.items() if n in a})
        kw = {n: x for n, x in bad.items() if n not in a}
        with pytest.raises(ValueError):
            qi.prefix_attention(a["q"], a["k"], a["v"], a["pk"], a["pv"], **kw)
    with pytest.raises(ValueError):
        qi.prefix_attention(q, None, None)
    with pytest.raises(qi.QiError, match="INVALID_ARG"):
        qi.prefix_attention(q, k, v, pk, pv, scale=-1.0)
    with pytest.raises(qi.QiError, match="INVALID_ARG"):  # rows that do not start on 16 bytes
        qi.prefix_attention(_normal(1, 6 * 8 * 128 + 4)[4:].view(6, 1, 8, 128), k, v, pk, pv)
    with pytest.raises(qi.QiError, match="INVALID_ARG"):  # one K row for all: stride 0
        qi.prefix_attention(q, k[:, :1].expand(-1, 200, -1, -1), v, pk, pv)
    q, k, v, pk, pv = _batch(qi, B=32, P=8192)             # sizes that go by partial results
    o = torch.zeros_like(q)
    strides = [x for t in (q, k, v, o) for x in t.stride()[:3]] + [0, *pk.stride()[:2], 0, *pv.stride()[:2]]
    L = qi.lib()

    def args(ws, size):
        head = qi._ATTN_HEAD.pack(*[t.data_ptr() for t in (q, k, v, o, pk, pv)], 0, 0, 0, 0, 0, ws, 0, 0, 0.1)
        return head + qi._ATTN_TAIL.pack(size, *strides, 0, 32, 1, 8, 2, 8192, 200)

    need = L.qi_prefix_attention_workspace(args(0, 0))
    assert need > 0
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    for ptr, size in ((0, 0), (ws.data_ptr(), need - 1), (ws.data_ptr() + 8, need)):
        with pytest.raises(qi.QiError, match="workspace"):
            qi._check(L.qi_prefix_attention(args(ptr, size), None))
    assert (o == 0).all()
    st = torch.cuda.current_stream().cuda_stream
    qi._check(L.qi_prefix_attention(args(ws.data_ptr(), need), st))
    assert torch.equal(o, qi.prefix_attention(q, k, v, pk, pv, scale=0.1))


# ---------------------------------------------------------------- 8-bit cache


def _values(seed, *shape, dtype):
    """Blocks of every size of scale, zeros, powers of two, ties and the type's extremes among them."""
    import torch
    rng = np.random.default_rng(seed)
    a = rng.standard_normal(shape) * np.exp2(rng.integers(-12, 12, (*shape[:-1], 1)))
    flat = a.reshape(-1, 32)
    flat[0] = 0
    flat[1 % len(flat)] = 448.0
    flat[2 % len(flat), :4] = [1.0, 1.0625, 1.1875, -1.0625]  # ties between neighbouring codes
    flat[3 % len(flat), 0] = 2.0 ** -24
    flat[4 % len(flat), 0] = 65504.0
    t = torch.from_numpy(a).clamp(-65504, 65504).to(_dt(dtype))
    return t.cuda()


def _quant(t):
    q, e = omx.quantize(_np(t))
    return omx.e4m3_encode(q), (e + 127).astype(np.uint8), omx.dequantize(q, e)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B,T,S,H,pos,lens", [
    (1, 1, 1, 1, None, None),
    (1, 407, 512, 4, None, None),
    (3, 5, 9, 3, [0, 4, 2], [5, 5, 1]),
    (4, 6, 8, 2, [-2, 5, 8, 2000000000], [6, 6, 6, 6]),      # rows before, across and behind the cache
    (3, 4, 6, 1, [1, 1, 1], [0, -3, 99]),
    (70, 1, 33, 2, [i % 33 for i in range(70)], None),
])
def test_kv8_write_and_read_bit_exact(qi, B, T, S, H, pos, lens, dtype):
    import torch
    dev = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
    kv = _values(B + T, B, T, 2, H, 128, dtype=dtype)
    k, v = kv[:, :, 0], kv[:, :, 1]                      # rows 2 H heads apart
    cache = qi.KV8Cache(*(torch.full_like(t, 85) for t in qi.kv8_cache(B, S, H)))
    qi.kv8_write(cache, k, v, pos=dev(pos), lens=dev(lens))
    out = tuple(torch.full((B, H, T, 128), 3.0, dtype=k.dtype, device="cuda").transpose(1, 2) for _ in range(2))
    rk, rv = qi.kv8_read(cache, T, k.dtype, pos=dev(pos), lens=dev(lens), out=out)
    for x, codes, sf, back in ((k, cache.k, cache.k_sf, rk), (v, cache.v, cache.v_sf, rv)):
        cq, ce, val = _quant(x)
        wq, ws = np.full((B, S, H, 128), 85, np.uint8), np.full((B, S, H, 4), 85, np.uint8)
        wb = np.full((B, T, H, 128), 3.0)
        for b in range(B):
            for t in range(min(T if lens is None else lens[b], T)):
                r = (0 if pos is None else pos[b]) + t
                if 0 <= r < S:
                    wq[b, r], ws[b, r], wb[b, t] = cq[b, t], ce[b, t], val[b, t]
        assert np.array_equal(codes.cpu().numpy(), wq) and np.array_equal(sf.cpu().numpy(), ws)
        # a value is exact in fp32; in 16 bits it is the nearest one (fp16 subnormals round)
        assert np.array_equal(_np(back), _np(torch.from_numpy(wb).to(k.dtype)))


def test_kv8_read_makes_its_output(qi):
    import torch
    k, v = _values(1, 2, 3, 1, 128, dtype="fp16"), _values(2, 2, 3, 1, 128, dtype="fp16")
    cache = qi.kv8_write(qi.kv8_cache(2, 3, 1), k, v)
    rk, _ = qi.kv8_read(cache, 3, torch.bfloat16)
    assert rk.dtype == torch.bfloat16 and np.array_equal(_np(rk), _np(torch.from_numpy(_quant(k)[2]).to(torch.bfloat16)))
    rk, rv = qi.kv8_read(cache, 5, torch.float16)        # rows behind the cache are zero
    assert (rk[:, 3:] == 0).all() and (rv[:, 3:] == 0).all() and np.array_equal(_np(rv[:, :3]), _np(torch.from_numpy(_quant(v)[2]).to(torch.float16)))


def test_kv8_refuses(qi):
    import torch
    cache, k = qi.kv8_cache(2, 8, 3), _normal(1, 2, 4, 3, 128)
    for bad in (dict(k=k[:1]), dict(k=k.float()), dict(v=k[:, :3]), dict(k=k[..., :64]), dict(v=k.cpu()),
                dict(pos=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(lens=torch.zeros(2, device="cuda"))):
        a = {"k": k, "v": k, **bad}
        with pytest.raises(ValueError):
            qi.kv8_write(cache, **a)
    with pytest.raises(ValueError):
        qi.kv8_write(qi.KV8Cache(*(t[:, ::2] for t in qi.kv8_cache(2, 16, 3))), k, k)
    with pytest.raises(ValueError):
        qi.kv8_read(cache, 4, torch.float16, out=(k, k[:, :3]))
    with pytest.raises(ValueError):
        qi.kv8_read(cache, 4, torch.float32)
    with pytest.raises(qi.QiError, match="INVALID_ARG"):
        qi.kv8_write(cache, k[:, :1].expand(-1, 4, -1, -1), k)


# ---------------------------------------------------------------- residual norm to MXFP8


def _sf(sf, rows, K):
    """[rows, K / 32] scale bytes of the chunk layout."""
    g = (rows + 127) // 128
    s = sf.cpu().numpy().reshape(K // 128, g, 32, 4, 4)
    r, kb = np.arange(rows)[:, None], np.arange(K // 32)[None, :]
    return s[kb // 4, r // 128, r % 32, r % 128 // 32, kb % 4]


def _check_norm(qi, rows, K, xd, dd, wd, plus_one=False, eps=1e-6, strided=False, inplace=False, scale=1.0, seed=0):
    import torch
    x = _normal(seed + 1, rows, K + (64 if strided else 0), std=2.0 * scale, dtype=xd)[:, :K]
    d = None if dd is None else _normal(seed + 2, rows, K + (128 if strided else 0), std=0.5 * scale, dtype=dd)[:, :K]
    w = None if wd is None else _normal(seed + 3, K, std=0.3, dtype=wd)
    x0 = x.clone()
    sf = torch.full((((rows + 127) // 128) * (K // 128) * 512,), 99, dtype=torch.uint8, device="cuda")
    xo, q, s = qi.add_rmsnorm_mxfp8(x, d, w, plus_one=plus_one, eps=eps, x_out=x if inplace else None, sf=sf)
    if not inplace:
        assert torch.equal(x, x0)
    gain = None if w is None else _np(w) + (1.0 if plus_one else 0.0)
    rnd = lambda a: _np(torch.from_numpy(a).to(_dt(xd)))
    ref_x, y = ob.add_rmsnorm(_np(x0), None if d is None else _np(d), gain, eps, rnd)
    # the sum: fp32 addition rounds once, then once more to a 16-bit type; the oracle rounds once
    u = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[xd]
    got_x = _np(xo)
    assert (np.abs(got_x - ref_x) <= 2 * u * np.abs(ref_x)).all() and (got_x == ref_x).mean() > 0.999
    # codes and scales: those of y up to fp32 roundings of y (relative 2^-23 with room), that is either
    # equal or, next to a border between two codes, the neighbour
    _, y = ob.add_rmsnorm(got_x, None, gain, eps, rnd)
    e = _sf(s, rows, K).astype(np.int64) - 127
    val = omx.dequantize(omx.E4M3_TABLE[q.cpu().numpy()], e)
    lo, hi = (omx.quantize(y * (1 + t * 2.0 ** -22)) for t in (-1, 1))
    near = (val == omx.dequantize(*lo)) | (val == omx.dequantize(*hi))
    assert near.all(), f"{(~near).sum()} codes off"
    exact = omx.quantize(y)
    differ = (val != omx.dequantize(*exact)).mean()
    assert differ <= 1e-4, differ
    # scale bytes of rows that are not there stay as they were
    pad = s.cpu().numpy().reshape(K // 128, -1, 32, 4, 4).transpose(1, 3, 2, 0, 4).reshape(-1, K // 32)[rows:]
    assert (pad == 99).all()


@pytest.mark.parametrize("rows,K", [(1, 128), (3, 4096), (129, 384), (200, 1408), (7, 12288), (5, 16384), (128, 2048)])
@pytest.mark.parametrize("xd,dd,wd,plus", [("fp32", "fp16", "bf16", True), ("bf16", "bf16", "fp32", False),
                                           ("fp16", "fp32", None, False), ("fp32", None, "bf16", False)])
def test_add_rmsnorm(qi, rows, K, xd, dd, wd, plus):
    _check_norm(qi, rows, K, xd, dd, wd, plus, seed=rows + K)


@pytest.mark.parametrize("xd", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("dd", ["fp32", "fp16", "bf16"])
def test_add_rmsnorm_types_strides_in_place(qi, xd, dd):
    _check_norm(qi, 33, 640, xd, dd, "bf16", True, strided=True, seed=5)
    _check_norm(qi, 33, 640, xd, dd, "fp32", True, strided=True, inplace=True, seed=6)


def test_add_rmsnorm_extremes(qi):
    import torch
    _check_norm(qi, 9, 256, "fp32", "fp32", "bf16", scale=1e-12)   # eps carries the mean
    _check_norm(qi, 9, 256, "fp32", "fp32", "bf16", scale=1e12)
    x = torch.zeros(2, 256, device="cuda")
    x[1, 5] = 3.0
    xo, q, s = qi.add_rmsnorm_mxfp8(x)
    assert (q[0] == 0).all() and (_sf(s, 2, 256)[0] == 0).all()     # an all-zero row: zero codes, the smallest scale
    assert q[1, 5] != 0 and (q[1, :5] == 0).all()


def test_add_rmsnorm_refuses(qi):
    import torch
    x, d = _normal(1, 4, 256, dtype="fp32"), _normal(2, 4, 256)
    for bad in (dict(x=x[0]), dict(x=x.double()), dict(delta=d[:3]), dict(delta=d.cpu()), dict(w=x[0, :128]),
                dict(w=x[0].double()), dict(x_out=d), dict(q=torch.empty(4, 128, dtype=torch.uint8, device="cuda")),
                dict(sf=torch.empty(4, dtype=torch.uint8, device="cuda")), dict(delta=d.t().contiguous().t())):
        with pytest.raises(ValueError):
            qi.add_rmsnorm_mxfp8(**{"x": x, "delta": d, **bad})
    with pytest.raises(qi.QiError, match="SHAPE"):
        qi.add_rmsnorm_mxfp8(_normal(1, 4, 192))
    with pytest.raises(qi.QiError, match="INVALID_ARG"):
        qi.add_rmsnorm_mxfp8(_normal(1, 4, 260)[:, :256])      # rows 520 bytes apart


# ---------------------------------------------------------------- a run of them together


def test_prompt_stored_in_8_bits_serves_a_batch_of_images(qi):
    """One block of the serving loop: the handle captures a prompt's text K/V, they go into the 8-bit
    cache, four images attend to them, and the residual norm feeds the block-scaled GEMM."""
    import torch

    import synth
    L, N, B = 22, 64, 4
    d = qi.DiT(blocks=1, L_max=L, N_max=N)
    try:
        W = synth.Weights(seed=0, nblocks=1)
        d.load_global(W.glob)
        d.load_block(0, W.block(0))
        tc, ts, _, _ = qi.rope_tables(L, 8, 8)
        d.text_kv_capture(torch.from_numpy(synth.input_f32(0, synth.J_TXT, (L, 4096))).cuda(), tc, ts)
        k16, v16 = (t.view(torch.float16).view(1, L, 32, 128) for t in d.read_kv(0, 0, L))
        cache = qi.kv8_write(qi.kv8_cache(1, 512, 32), k16, v16)
        pk, pv = (t[0] for t in qi.kv8_read(cache, L, torch.float16))
        qkv = _normal(1, B, N, 96, 128, std=1.2)
        q, k, v = qkv[:, :, :32], qkv[:, :, 32:64], qkv[:, :, 64:]
        o = qi.prefix_attention(q, k, v, prefix8=cache.prefix(0, L))
        assert torch.equal(o, qi.prefix_attention(q, k, v, pk, pv))      # the cache's values, in either form
        args = (_np(q), _np(k), _np(v), _np(pk), _np(pv))
        ref, A = ob.prefix_attention(*args, None, False, 1 / math.sqrt(128))
        assert (np.abs(_np(o) - ref) <= _bound(*args, None, 1 / math.sqrt(128), ref, A, "fp16")).all()
        x = _normal(2, B * N, 4096, std=2.0, dtype="fp32")
        x1, a8, a_sf = qi.add_rmsnorm_mxfp8(x, o.view(B * N, 4096))
        Wb = _normal(3, 512, 4096, std=0.02, dtype="bf16")
        b8, b_sf = qi.quant_mxfp8(Wb.view(torch.int16), bf16=True)
        D = d.gemm_mxfp8(a8, a_sf, b8, b_sf, B * N, 512, 4096)
        d.check()
        am = omx.dequantize(omx.E4M3_TABLE[a8.cpu().numpy()], _sf(a_sf, B * N, 4096).astype(np.int64) - 127)
        bm = omx.fake_quant(_np(Wb)).astype(np.float64)
        tol = (4096 / 32) * 2.0 ** -24 * (np.abs(am) @ np.abs(bm).T) + 1e-30
        assert (np.abs(_np(D) - am @ bm.T) <= tol).all()
    finally:
        d.close()
