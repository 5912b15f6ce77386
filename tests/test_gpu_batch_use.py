"""The batch operators as a server uses them: captured and replayed, on several streams and threads, over
caches whose offsets pass 32 bits, with every decomposition of the attention. Oracle, helpers and the
attention's error bound are those of test_gpu_batch."""
import math
import threading

import numpy as np
import pytest

from oracle import batch as ob
from test_gpu_batch import _bound, _check_attention, _normal, _np, qi  # noqa: F401

pytestmark = pytest.mark.gpu

# sizes by what the attention makes of them: few rows joined in a cluster, packed with partials, joined from
# many tiles; 128 rows packed with partials, joint, joined; few rows in 53 chunks with partials, 128 rows too
KINDS = [
    dict(B=1, T=1, Hq=32, Hkv=32, P=22, S=17),
    dict(B=16, T=1, Hq=32, Hkv=32, P=2100, S=256),
    dict(B=1, T=1, Hq=32, Hkv=32, P=9000, S=40),
    dict(B=32, T=1, Hq=32, Hkv=8, P=4000, S=300),
    dict(B=2, T=300, Hq=32, Hkv=8, P=140, S=300),
    dict(B=2, T=40, Hq=8, Hkv=2, P=900, S=700),
    dict(B=1, T=1, Hq=8, Hkv=2, P=20000, S=64),
    dict(B=1, T=30, Hq=8, Hkv=2, P=20000, S=64),
]
IDS = ["-".join(str(x) for x in c.values()) for c in KINDS]


def _case(qi, c, seed, dtype="fp16", bits=16):
    import torch
    q = _normal(seed, c["B"], c["T"], c["Hq"], 128, dtype=dtype)
    k, v = (_normal(seed + i, c["B"], c["S"], c["Hkv"], 128, dtype=dtype) for i in (1, 2))
    pk, pv = (_normal(seed + i, c["P"], c["Hkv"], 128, dtype=dtype) for i in (3, 4))
    kw = dict(prefix_k=pk, prefix_v=pv)
    if bits == 8:
        kw = dict(prefix8=qi.kv8_write(qi.kv8_cache(1, c["P"], c["Hkv"]), pk[None], pv[None]).prefix(0, c["P"]))
    lens = torch.tensor(np.random.default_rng(seed).integers(0, c["S"] + 1, c["B"]), dtype=torch.int32, device="cuda")
    return dict(q=q, k=k, v=v, own_len=lens, causal=True, **kw)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("c", KINDS, ids=IDS)
def test_attention_captured(qi, c, bits):
    """Replayed with other values and lengths in the same memory; two graphs at once on two streams."""
    import torch
    sets = [_case(qi, c, 10 + 50 * i, bits=bits) for i in range(2)]
    outs = [torch.empty_like(s["q"]) for s in sets]
    graphs = [torch.cuda.CUDAGraph() for _ in sets]
    for s, o in zip(sets, outs):
        qi.prefix_attention(out=o, **s)
    torch.cuda.synchronize()
    for g, s, o in zip(graphs, sets, outs):
        with torch.cuda.graph(g):
            qi.prefix_attention(out=o, **s)
    for turn in range(3):
        for s in sets:
            s["q"].copy_(_normal(300 + turn, *s["q"].shape))
            s["own_len"].copy_((s["own_len"] * 7 + turn) % (c["S"] + 1))
        want = [qi.prefix_attention(**s) for s in sets]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in sets]
        for _ in range(4):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_a_chain_captured(qi):
    """Rows written to the cache, read back, attended to and normed, 20 times over in one graph: each launch
    may start before the one before it is through, and each result equals that of calls one at a time."""
    import torch
    B, S, H = 3, 400, 8
    cache = qi.kv8_cache(B, S, H)
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    k, v = _normal(1, B, 5, H, 128), _normal(2, B, 5, H, 128)
    x = _normal(3, B, H * 128, dtype="fp32")
    q = _normal(4, B, 1, H, 128)

    def step(sync):
        qi.kv8_write(cache, k, v, pos=pos, lens=lens)
        sync()
        rk, rv = qi.kv8_read(cache, S, torch.float16, lens=pos + lens)
        sync()
        o = qi.prefix_attention(q, rk, rv, own_len=pos + lens, prefix8=cache.prefix(0, 300))
        sync()
        xo, a8, sf = qi.add_rmsnorm_mxfp8(x, o.view(B, H * 128), x_out=x)
        sync()
        k.copy_(k.roll(1, 1) * 0.75)
        pos.add_(lens)
        sync()
        return [t.clone() for t in (rk, rv, o, a8, sf)]

    start = [t.clone() for t in (*cache, pos, k, x)]

    def reset():
        for t, s in zip((*cache, pos, k, x), start):
            t.copy_(s)

    want = [step(torch.cuda.synchronize) for _ in range(20)]
    end = [t.clone() for t in (*cache, x)]
    reset()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [step(lambda: None) for _ in range(20)]
    for _ in range(2):
        reset()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for r, w in zip(got, want) for a, b in zip(r, w))
        assert all(torch.equal(a, b) for a, b in zip((*cache, x), end))


def test_threads_with_streams_of_their_own(qi):
    import torch
    work = [(_case(qi, c, 7 * i, bits=8 if i % 2 else 16), _normal(i, 40 + i, 1024, dtype="fp32"),
             _normal(i + 1, 2, 30 + i, 4, 128)) for i, c in enumerate(KINDS)]
    want = [(qi.prefix_attention(**a), *qi.add_rmsnorm_mxfp8(x), *qi.kv8_write(qi.kv8_cache(2, 64, 4), kv, kv))
            for a, x, kv in work]
    torch.cuda.synchronize()
    bad = []

    def run(i):
        st = torch.cuda.Stream()
        for n in range(30):
            j = (i + n) % len(work)
            a, x, kv = work[j]
            if n % 2:
                got = (qi.prefix_attention(stream=st, **a), *qi.add_rmsnorm_mxfp8(x, stream=st),)
                st.synchronize()
                got += tuple(qi.kv8_write(qi.kv8_cache(2, 64, 4), kv, kv))
                torch.cuda.synchronize()
            else:
                with torch.cuda.stream(st):
                    got = (qi.prefix_attention(**a), *qi.add_rmsnorm_mxfp8(x), *qi.kv8_write(qi.kv8_cache(2, 64, 4), kv, kv))
                st.synchronize()
            if not all(torch.equal(g, w) for g, w in zip(got, want[j])):
                bad.append((i, n))
        torch.cuda.synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_freed_while_another_stream_still_reads(qi):
    """Arguments whose last reference goes right after a call on another stream."""
    import torch
    a = _case(qi, KINDS[4], 5)
    want = qi.prefix_attention(**a)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    filler = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(4):
        b = {n: x.clone() if torch.is_tensor(x) else x for n, x in a.items()}
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for _ in range(20):
                filler.zero_()          # keeps the stream busy while the memory could be handed out again
        got.append(qi.prefix_attention(stream=st, **b))
        shapes = [(x.shape, x.dtype) for x in b.values() if torch.is_tensor(x)]
        del b
        for shape, dtype in shapes:
            torch.empty(shape, dtype=dtype, device="cuda").fill_(3)
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


# units without a tile, clusters in which only the first CTA has one, rows whose mask leaves nothing
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("c", [
    dict(B=2, T=1, Hq=8, Hkv=8, P=0, S=2000, lens=[3, 0]),
    dict(B=2, T=1, Hq=8, Hkv=8, P=0, S=2000, lens=[0, 1999], causal=True),
    dict(B=2, T=40, Hq=4, Hkv=2, P=0, S=2000, lens=[39, 0], causal=True),
    dict(B=2, T=40, Hq=4, Hkv=2, P=100, S=2000, lens=[1, 0]),
    dict(B=2, T=64, Hq=4, Hkv=2, P=900, S=700, lens=[700, 129], causal=True),
    dict(B=1, T=16, Hq=1, Hkv=1, P=1, S=5000, lens=[17], causal=True),
    dict(B=3, T=17, Hq=1, Hkv=1, P=1, S=5000, lens=[17, 16, 5000], causal=True, layout="bhsd"),
    dict(B=12, T=1, Hq=8, Hkv=8, P=3000, S=600, lens=[0] * 12),
    dict(B=300, T=1, Hq=2, Hkv=2, P=129, S=3, lens=[i % 4 for i in range(300)]),
    dict(B=1, T=1, Hq=8, Hkv=2, P=9000, S=64, lens=[63], causal=True),
    dict(B=1, T=30, Hq=8, Hkv=2, P=9000, S=64, lens=[20], causal=True),
], ids=lambda c: f"B{c['B']}-T{c['T']}-P{c['P']}-S{c['S']}")
def test_attention_few_keys_of_many(qi, c, dtype):
    _check_attention(qi, dtype=dtype, seed=c["S"] + c["B"], **c)


@pytest.mark.parametrize("dtype,low,high", [("fp16", -33, 6), ("bf16", -100, 60)])
def test_attention_one_key_of_any_scale(qi, dtype, low, high):
    """One key: the row is its value, bit for bit, whatever the scales of the 8-bit prefix (the value is the
    code times its scale, rounded once to the type; times a probability of 1 nothing else rounds)."""
    import torch
    rng = np.random.default_rng(3)
    H = 160
    codes = rng.integers(0, 255, (2, 1, H, 128)).astype(np.uint8)
    codes[(codes & 127) == 127] = 1
    sf = (rng.integers(low, high + 1, (2, 1, H, 4)) + 127).astype(np.uint8)
    t = [torch.from_numpy(a).cuda() for a in (codes[0], codes[1], sf[0], sf[1])]
    pre = qi.KV8Cache(*t)
    _, val = qi.kv8_read(qi.KV8Cache(*(x[None] for x in t)), 1, getattr(torch, {"fp16": "float16", "bf16": "bfloat16"}[dtype]))
    for T in (1, 5, 40):
        q = _normal(T, 2, T, H, 128, std=2.0 ** -12, dtype=dtype)
        q *= 0 if dtype == "bf16" else 1               # (keys of 2^69 leave the scores no room)
        o = qi.prefix_attention(q, None, None, prefix8=pre)
        assert torch.equal(o, val[0].expand(2, T, H, 128)), T


def test_attention_prefix_of_mixed_scales(qi):
    """Tiles that hold codes of very different scales, against the values that reading them back gives."""
    import torch
    rng = np.random.default_rng(4)
    for dtype, T, P, H in (("fp16", 1, 1300, 4), ("bf16", 3, 700, 2), ("fp16", 5, 129, 3)):
        codes = rng.integers(0, 255, (2, P, H, 128)).astype(np.uint8)
        codes[(codes & 127) == 127] = 0
        sf = (rng.integers(-26, -5, (2, P, H, 4)) + 127).astype(np.uint8)
        sf[0] = np.maximum(sf[0], 127 - 9)
        sf[0, :, :, 0] = 0                               # a block of K of almost nothing
        t = [torch.from_numpy(a).cuda() for a in (codes[0], codes[1], sf[0], sf[1])]
        pk, pv = (x[0] for x in qi.kv8_read(qi.KV8Cache(*(x[None] for x in t)), P, _normal(1, 1, dtype=dtype).dtype))
        q = _normal(9, 4, T, 2 * H, 128, std=0.3, dtype=dtype)
        k, v = _normal(10, 4, 0, H, 128, dtype=dtype), _normal(11, 4, 0, H, 128, dtype=dtype)
        o = qi.prefix_attention(q, k, v, prefix8=qi.KV8Cache(*t))
        args = (_np(q), _np(k), _np(v), _np(pk), _np(pv))
        scale = 1 / math.sqrt(128)
        ref, A = ob.prefix_attention(*args, None, False, scale)
        assert (np.abs(_np(o) - ref) <= _bound(*args, None, scale, ref, A, dtype)).all()


# ---------------------------------------------------------------- offsets past 32 bits


def _far(shape, strides, dtype):
    """A tensor over memory that only its own elements of are ever written."""
    import torch
    n = sum((s - 1) * t for s, t in zip(shape, strides)) + 1
    return torch.empty(n, dtype=dtype, device="cuda").as_strided(shape, strides)


@pytest.mark.parametrize("T", [1, 70])
def test_attention_far_apart(qi, T):
    """Sequences, rows and heads of keys, queries and outputs more than 2^31 elements apart."""
    import torch
    B, Hq, Hkv, P, S = 2, 4, 2, 200, 150
    a = dict(q=_normal(1, B, T, Hq, 128), k=_normal(2, B, S, Hkv, 128), v=_normal(3, B, S, Hkv, 128))
    pk, pv = _normal(4, P, Hkv, 128), _normal(5, P, Hkv, 128)
    lens = torch.tensor([150, 77], dtype=torch.int32, device="cuda")
    want = qi.prefix_attention(a["q"], a["k"], a["v"], pk, pv, own_len=lens, causal=True)
    st = {"q": (2 ** 31 + 64, Hq * 128, 128), "k": (2 ** 31 + 8, 2 ** 20, 128), "v": (128, 2 ** 24, 2 ** 31 + 256)}
    for name, s in st.items():
        far = _far(a[name].shape, (*s, 1), a[name].dtype)
        far.copy_(a[name])
        a[name] = far
    st = (2 ** 24, 256, 1)
    fk, fv = _far(pk.shape, st, pk.dtype), _far(pv.shape, (128, 2 ** 31 + 512, 1), pv.dtype)
    fk.copy_(pk), fv.copy_(pv)
    out = _far(want.shape, (128 * Hq, 2 ** 26, 128, 1) if T > 1 else (2 ** 31 + 8, 512, 128, 1), want.dtype)
    qi.prefix_attention(a["q"], a["k"], a["v"], fk, fv, own_len=lens, causal=True, out=out)
    assert torch.equal(out, want)


def test_kv8_in_a_cache_past_32_bits(qi):
    """Rows at the end of a cache of 2 x 2.1 GB a tensor; attention over the last of its prompts."""
    import torch
    S, H = 2 ** 19 + 300, 32
    cache = qi.kv8_cache(2, S, H)
    T = 200
    k, v = _normal(1, 2, T, H, 128), _normal(2, 2, T, H, 128)
    pos = torch.tensor([3, S - 150], dtype=torch.int32, device="cuda")
    qi.kv8_write(cache, k, v, pos=pos)
    small = qi.kv8_write(qi.kv8_cache(2, T, H), k, v)
    for big, sm in zip(cache, small):
        assert torch.equal(big[0, 3:203], sm[0]) and torch.equal(big[1, S - 150:], sm[1, :150])
        assert big[1, :S - 150].count_nonzero() == 0 and big[0, 203:].count_nonzero() == 0
    rk, rv = qi.kv8_read(cache, T, torch.float16, pos=pos)
    wk, wv = qi.kv8_read(small, T, torch.float16)
    for r, w in ((rk, wk), (rv, wv)):
        assert torch.equal(r[0], w[0]) and torch.equal(r[1, :150], w[1, :150]) and (r[1, 150:] == 0).all()
    # 2^19 + 300 keys of which all but the last 150 are zero: scores of 0 and values of 0
    q = _normal(3, 1, 1, H, 128, std=2.0)
    o = qi.prefix_attention(q, None, None, prefix8=cache.prefix(1, S))
    kk, vv, qq = _np(wk[1, :150]), _np(wv[1, :150]), _np(q[0, 0])
    s = np.einsum("hd,nhd->hn", qq, kk) / math.sqrt(128)
    top = np.maximum(s.max(1), 0)[:, None]
    e = np.exp(s - top)
    den = e.sum(1)[:, None] + (S - 150) * np.exp(-top)
    ref = np.einsum("hn,nhd->hd", e, vv) / den
    A = np.einsum("hn,nhd->hd", e, np.abs(vv)) / den
    mag = (np.einsum("hd,nhd->hn", np.abs(qq), np.abs(kk)).max(1) / math.sqrt(128))[:, None]
    # as the attention's bound elsewhere, with the sum's rounding over S terms (fp32, in 128-key steps of a
    # tree per unit: at most S 2^-23 in a row) and half an fp16 subnormal step per key that is not zero
    tol = (2.0 ** -11 * (A + np.abs(ref)) * (1 + 2.0 ** -8) + 2 * (mag * (128 * 2.0 ** -23 + 3 * 2.0 ** -24) + 2.0 ** -22) * A
           + (2 * S * 2.0 ** -23 + 8 * 2.0 ** -22) * A + 150 * 2.0 ** -25 * np.abs(vv).max() + 2.0 ** -25)
    assert (np.abs(_np(o[0, 0]) - ref) <= tol).all()


def test_add_rmsnorm_far_apart(qi):
    """Rows past 2^31 elements, by stride and by number."""
    import torch
    x, d = _normal(1, 18, 256, dtype="fp32"), _normal(2, 18, 256)
    want = qi.add_rmsnorm_mxfp8(x, d)
    fx, fd = _far(x.shape, (2 ** 27, 1), x.dtype), _far(d.shape, (2 ** 27 + 8, 1), d.dtype)
    fx.copy_(x), fd.copy_(d)
    got = qi.add_rmsnorm_mxfp8(fx, fd, x_out=fx)
    assert got[0] is fx and all(torch.equal(a, b) for a, b in zip(got, want))
    rows, K = 2 ** 17 + 3, 16384
    x = torch.zeros(rows, K, dtype=torch.float16, device="cuda")
    part = torch.cat([torch.arange(5), torch.arange(rows - 5, rows)]).cuda()
    x[part] = _normal(3, 10, K)
    xo, q, sf = qi.add_rmsnorm_mxfp8(x, x, x_out=x)          # in place, and the stream added to itself
    wx, wq, wsf = qi.add_rmsnorm_mxfp8(_normal(3, 10, K), _normal(3, 10, K))
    assert torch.equal(xo[part], wx) and torch.equal(q[part], wq)
    g = (rows + 127) // 128
    grid = sf.view(K // 128, g, 32, 4, 4)
    small = wsf.view(K // 128, 1, 32, 4, 4)
    for i, r in enumerate(part.tolist()):
        assert torch.equal(grid[:, r // 128, r % 32, r % 128 // 32], small[:, 0, i % 32, i // 32])


# ---------------------------------------------------------------- values that are no numbers


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_kv8_of_infinities_and_nan(qi, dtype):
    """The same codes and scales as the framework's quantiser: NaN has its code, an infinity the largest, and
    a block of nothing but NaN the scale of zero."""
    import torch
    x = _normal(1, 6, 128, dtype=dtype)
    x[0, :32] = float("nan")
    x[1, 3], x[1, 40] = float("nan"), -float("nan")
    x[2, 5], x[2, 70] = float("inf"), -float("inf")
    x[3] = -float("nan")
    x[4, 32:64], x[4, 64:96] = 0.0, -0.0
    want, sf = qi.quant_mxfp8(x.view(torch.int16), bf16=dtype == "bf16")
    cache = qi.kv8_write(qi.kv8_cache(1, 6, 1), x.view(1, 6, 1, 128), x.view(1, 6, 1, 128))
    ws = sf.view(32, 4, 4)[:6, 0]
    for c, s in ((cache.k, cache.k_sf), (cache.v, cache.v_sf)):
        assert torch.equal(s[0, :, 0], ws) and torch.equal(c[0, :, 0], want)


def test_add_rmsnorm_row_of_nan_stays_its_own(qi):
    import torch
    x = _normal(1, 5, 512, dtype="fp32")
    bad = x.clone()
    bad[1, 7], bad[3, 100] = float("nan"), float("inf")
    a, b = qi.add_rmsnorm_mxfp8(x), qi.add_rmsnorm_mxfp8(bad)
    good = torch.tensor([0, 2, 4]).cuda()
    assert torch.equal(a[1][good], b[1][good])
    assert ((b[1][1] & 127) == 127).all() and (b[1][3, 100] & 127) == 127 and (b[1][3, :100] & 127).max() == 0


def test_attention_masked_places_hold_anything(qi):
    """Own rows past own_len hold infinities, NaN and the largest values, in every decomposition."""
    import torch
    for i, c in enumerate(KINDS):
        a = _case(qi, c, 40 + i, dtype=["fp16", "bf16"][i % 2])
        a["own_len"] = a["own_len"].clamp(max=c["S"] - 1)
        want = qi.prefix_attention(**a)
        for fill in (float("nan"), float("inf"), torch.finfo(a["k"].dtype).max, torch.finfo(a["k"].dtype).min):
            b = dict(a, k=a["k"].clone(), v=a["v"].clone())
            for s, n in enumerate(a["own_len"].tolist()):
                b["k"][s, n:], b["v"][s, n:] = fill, -fill
            assert torch.equal(qi.prefix_attention(**b), want), (c, fill)


@pytest.mark.parametrize("c", KINDS, ids=IDS)
def test_attention_of_tensors_at_any_16_bytes(qi, c):
    """Every tensor 16 bytes off a 32-byte boundary, outputs with rows and heads at odd multiples of 16 bytes."""
    import torch

    def off(t, pad=0):
        wide = torch.zeros(*t.shape[:-1], t.shape[-1] + pad, dtype=t.dtype, device=t.device)
        base = torch.zeros(wide.numel() + 8, dtype=t.dtype, device=t.device)[8:].view(wide.shape)[..., :t.shape[-1]]
        base.copy_(t)
        return base

    a = _case(qi, c, 77)
    want = qi.prefix_attention(**a)
    b = {n: off(x, 8) if torch.is_tensor(x) and x.dim() > 1 else x for n, x in a.items()}
    for pad in (0, 8, 24):
        out = off(torch.zeros_like(want), pad)
        assert out.data_ptr() % 32 == 16
        assert torch.equal(qi.prefix_attention(out=out, **b), want)
        assert torch.equal(out, want)


def test_kv8_and_norm_of_tensors_at_any_16_bytes(qi):
    import torch
    k, v = _normal(1, 2, 9, 3, 128), _normal(2, 2, 9, 3, 128)
    want = qi.kv8_write(qi.kv8_cache(2, 9, 3), k, v)
    buf = torch.zeros(8 + 2 * 9 * 3 * 136, dtype=k.dtype, device="cuda")
    far = buf[8:].view(2, 9, 3, 136)[..., :128]
    far.copy_(k)
    got = qi.kv8_write(qi.kv8_cache(2, 9, 3), far, v)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    far.zero_()
    rk, _ = qi.kv8_read(want, 9, torch.float16, out=(far, torch.empty_like(v)))
    assert torch.equal(rk, qi.kv8_read(want, 9, torch.float16)[0]) and buf[:8].count_nonzero() == 0
    assert buf[8:].view(2, 9, 3, 136)[..., 128:].count_nonzero() == 0
    for dt in ("fp32", "bf16"):
        x, d = _normal(3, 5, 256, dtype=dt), _normal(4, 5, 256, dtype="fp32")
        n = 16 // x.element_size()
        fx = torch.zeros(n + 5 * (256 + n), dtype=x.dtype, device="cuda")[n:].view(5, 256 + n)[:, :256]
        fx.copy_(x)
        want = qi.add_rmsnorm_mxfp8(x, d)
        assert all(torch.equal(g, w) for g, w in zip(qi.add_rmsnorm_mxfp8(fx, d, x_out=fx), want))


def test_add_rmsnorm_into_its_arguments_and_new_scales(qi):
    """x_out may be x or delta; the scales that a call makes itself are complete, whole groups of 128 rows or not."""
    import torch
    for rows in (5, 128, 256, 300):
        x, d = _normal(rows, rows, 384), _normal(rows + 1, rows, 384)
        torch.full((rows * 384 // 32 + 70000,), 255, dtype=torch.uint8, device="cuda")   # dirties what comes next
        want = qi.add_rmsnorm_mxfp8(x, d)
        sf = torch.zeros(((rows + 127) // 128) * 3 * 512, dtype=torch.uint8, device="cuda")
        for n in ("x", "d"):
            a, b = x.clone(), d.clone()
            to = a if n == "x" else b
            got = qi.add_rmsnorm_mxfp8(a, b, x_out=to, sf=sf.zero_())
            assert got[0] is to and all(torch.equal(g, w) for g, w in zip(got, want))
