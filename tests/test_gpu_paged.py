"""Operators of sequences in pages, against the float64 oracle on the same inputs.

Rotation bound, per output element, with u the half step of the output type and m the magnitudes it is made of
(|y_i| + |y_j| of its pair):
* rounded once: u |out|, plus half a subnormal step of fp16, 2^-25;
* the angle: its low 32 bits dropped (2^-32 of a circle), the fraction rounded to fp32 (2^-25 of a half turn at most),
  the frequency rounded to fp64 when its turns are made (2^-52 of the angle); sincospif is within 2 steps of its result:
  together below 2^-21 m + 2^-51 |angle| m;
* the mean of 128 squares in fp32 (a tree of depth 8 over rounded products, and eps): 10 steps of 2^-24, half of that in
  r, rsqrtf within 2 steps, gain (1 + w) and three products: below 2^-20 m.
V is only rounded: u |v|.

Attention bound: as in test_gpu_batch.py's docstring.
"""
import math

import numpy as np
import pytest

from oracle import paged as op

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


def _int(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _spread(t, layout):
    """The values of t [a, b, heads, 128] in another layout: heads outside b, or surrounded by NaN."""
    import torch
    if t is None or layout == "plain":
        return t
    if layout == "heads first":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    wide = torch.full((*t.shape[:2], t.shape[2] + 3, 128), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :, 1:-2] = t
    return wide[:, :, 1:-2]


# ---------------------------------------------------------------- norm and rotation


def _rope_tol(y, m, a, dtype, halves):
    i, j = op.partners(a.shape[-1], halves)
    ang = np.zeros((*a.shape[:-1], 1, 128))
    ang[..., 0, i] = ang[..., 0, j] = np.abs(a)
    return U[dtype] * np.abs(y) + m * (2.0 ** -21 + 2.0 ** -51 * ang + 2.0 ** -20) * (1 + 2.0 ** -8) + 2.0 ** -25


def _check_rope(qi, B=2, T=3, Hq=4, Hkv=2, axes=(16, 56, 56), theta=1e4, halves=False, x="bf16", dtype="bf16", norm=True,
                plus_one=False, w="bf16", page=0, pos="given", far=1000, start=None, lens=None, layout="plain", inplace=False,
                seed=0, std=1.7, absent="", bad_pages=(), width=None):
    import torch
    g = np.random.default_rng(seed + 100)
    t = {n: _spread(_normal(seed + i, B, T, h, 128, std=std, dtype=x), layout)
         for i, (n, h) in enumerate((("q", Hq), ("k", Hkv), ("v", Hkv))) if n not in absent}
    if lens is not None:  # rows behind a sequence may hold anything
        for n in t:
            for b, r in enumerate(lens):
                t[n][b, max(0, r):] = float("nan")
    gains = {n: (_normal(seed + 7 + i, 128, std=0.3, dtype=w if w != "fp32" else "fp32") + (0 if plus_one else 1)).to(_dt(w))
             for i, n in enumerate("qk")} if norm else {}
    rope = qi.rope(axes, theta=theta, halves=halves) if axes else None
    freqs = op.frequencies(axes, theta) if axes else np.zeros(0)
    pairs = tuple(d // 2 for d in axes)
    first = np.zeros(B, np.int64) if start is None else np.asarray(start, np.int64)
    if pos == "given":
        p = g.integers(-far, far, (B, T, len(axes)))
    else:
        p = np.repeat((first[:, None] + np.arange(T))[..., None], max(1, len(axes)), -1)
    a = op.angles(p, freqs, pairs) if axes else np.zeros((B, T, 0))
    live = np.arange(T)[None, :] < (np.full(B, T) if lens is None else np.asarray(lens))[:, None]
    want, tol = {}, {}
    src = {n: _np(v) for n, v in t.items()}
    for n in src:
        if n == "v":
            want[n], tol[n] = src[n], U[dtype] * np.abs(src[n]) + 2.0 ** -25
        else:
            gain = _np(gains[n]) + plus_one if norm else None
            want[n], m = op.norm_rope(src[n], gain, 1e-6, a, halves)
            tol[n] = _rope_tol(want[n], m, a, dtype, halves)
    kw = dict(rope=rope, q_w=gains.get("q") if "q" in t else None, k_w=gains.get("k") if "k" in t else None,
              plus_one=plus_one, lens=None if lens is None else _int(lens), start=None if start is None else _int(start),
              pos=_int(p.tolist()) if pos == "given" and axes else None)
    outs = {n: torch.full((B, T, t[n].shape[2] + 1, 128), 7.0, dtype=_dt(dtype), device="cuda") for n in t}
    out = {n: outs[n][:, :, :-1] for n in t}
    if inplace:
        out["q"] = t["q"]
    if page:
        need = [max(0, -(-(int(first[b]) + T) // page)) for b in range(B)]
        wide = max(need) + 2 if width is None else width
        need = [min(x, wide) for x in need]
        total = sum(need) + 3
        order = g.permutation(total)
        table = np.full((B, wide), -1)
        at = 0
        for b in range(B):
            table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        for b, i, n in bad_pages:
            table[b, i] = n
        ck, cv = (_normal(seed + 20 + i, total, page, Hkv, 128, dtype=dtype) for i in range(2))
        ek, ev = _np(ck), _np(cv)
        tk, tv = np.zeros(ek.shape), np.zeros(ev.shape)
        for b in range(B):
            for r in range(T):
                row = int(first[b]) + r
                if not live[b, r] or row < 0 or row // page >= wide or not 0 <= table[b, row // page] < total:
                    continue
                here = table[b, row // page], row % page
                if "k" in want:
                    ek[here], tk[here] = want["k"][b, r], tol["k"][b, r]
                if "v" in want:
                    ev[here], tv[here] = want["v"][b, r], tol["v"][b, r]
        lay = "heads first" if layout == "heads first" else "plain"
        cache = qi.PagedKV(_spread(ck, lay), _spread(cv, lay))
        got = qi.qk_norm_rope(t.get("q"), t.get("k"), t.get("v"), dtype=_dt(dtype), out=(out.get("q"), None, None),
                              cache=cache, table=_int(table.tolist()), **kw)
        assert got[1] is None and got[2] is None
        for c, e, tl, n in ((cache.k, ek, tk, "k"), (cache.v, ev, tv, "v")):
            err = np.abs(_np(c) - e)
            assert (err <= tl).all(), f"cache {n}: {err.max():.3e}, at {np.argwhere(err > tl)[:3].tolist()}"
        names = ["q"] if "q" in t else []
    else:
        got = qi.qk_norm_rope(t.get("q"), t.get("k"), t.get("v"), dtype=_dt(dtype),
                              out=tuple(out.get(n) for n in "qkv"), **kw)
        names = list(t)
    for n in names:
        r = got["qkv".index(n)]
        assert r.data_ptr() == out[n].data_ptr()
        r = _np(r)
        err = np.where(live[..., None, None], np.abs(r - want[n]), 0.0)
        assert (err[live] <= tol[n][live]).all(), f"{n}: {np.nanmax(err):.3e}, {np.nanmax(err[live] / tol[n][live]):.2f} of the bound"
        if not (inplace and n == "q"):
            assert (r[~live] == 7).all() and (outs[n][:, :, -1] == 7).all()


ROPE = [
    dict(B=1, T=1, Hq=1, Hkv=1, axes=(128,)),
    dict(B=1, T=1, Hq=32, Hkv=8, axes=(128,), halves=True, far=10 ** 9),
    dict(B=3, T=5, Hq=3, Hkv=1),
    dict(B=2, T=7, Hq=5, Hkv=5, axes=(44, 42, 42), layout="heads first"),
    dict(B=2, T=7, Hq=5, Hkv=3, axes=(44, 42, 42), layout="wide", halves=True),
    dict(B=2, T=3, axes=(2,)), dict(B=2, T=3, axes=(10, 4)), dict(B=2, T=3, axes=(16, 14), halves=False),
    dict(B=2, T=3, axes=(16,), halves=True), dict(B=2, T=3, axes=(32, 32, 32), halves=True),
    dict(B=2, T=3, axes=(8, 24, 48, 48), halves=True), dict(B=2, T=3, axes=(8, 24, 48, 48)),
    dict(B=4, T=33, Hq=7, Hkv=2, axes=(128,), lens=[33, 0, 1, 20]),
    dict(B=2, T=3, axes=()), dict(B=2, T=3, axes=(), norm=False),
    dict(B=2, T=300, Hq=9, Hkv=3, axes=(64,), norm=False, pos="counted", start=[5, 2000000]),
    dict(B=2, T=3, axes=(64, 64), far=2 ** 31 - 1), dict(B=1, T=2, axes=(128,), pos="counted", start=[2 ** 31 - 3]),
    dict(B=2, T=4, plus_one=True, w="fp32"), dict(B=2, T=4, plus_one=True), dict(B=2, T=4, w="fp32", halves=True),
    dict(B=2, T=4, absent="k"), dict(B=2, T=4, absent="kv"), dict(B=2, T=4, absent="q"), dict(B=2, T=4, absent="qk"),
    dict(B=1, T=2000, Hq=8, Hkv=2),
]


@pytest.mark.parametrize("types", ["bf16", "fp16", "fp32 bf16", "fp32 fp16"])
@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(f"{n}{c[n]}" for n in c).replace(" ", "")[:60])
def test_rope(qi, case, types):
    x, dtype = types.split()[0], types.split()[-1]
    _check_rope(qi, x=x, dtype=dtype, seed=len(str(case)), **case)


PAGED = [
    dict(B=1, T=1, page=16, start=[0]), dict(B=1, T=1, page=16, start=[15]), dict(B=1, T=1, page=16, start=[16]),
    dict(B=3, T=40, page=16, start=[0, 9, 31], lens=[40, 17, 0]),
    dict(B=3, T=40, page=32, start=[70, 0, 1], lens=[40, 40, 39], layout="heads first"),
    dict(B=5, T=1, Hq=3, Hkv=3, page=64, start=[63, 64, 0, 200, 65], lens=[1, 1, 1, 1, 0], axes=(128,), pos="counted"),
    dict(B=2, T=9, page=256, start=[250, 300]), dict(B=2, T=9, page=16, start=None),
    dict(B=2, T=20, page=16, start=[-5, 3]),                                   # rows before the first: passed over
    dict(B=2, T=40, page=16, start=[0, 10], width=2),                          # ... past the table's reach
    dict(B=2, T=40, page=16, start=[0, 0], bad_pages=[(0, 1, 10 ** 6), (1, 0, -3), (1, 2, 2 ** 31 - 1)]),
    dict(B=2, T=3, page=16, start=[2 ** 31 - 2, 4], width=3),                  # start + t wraps: passed over
    dict(B=2, T=4, page=16, start=[3, 4], absent="v"), dict(B=2, T=4, page=16, start=[3, 4], absent="k"),
    dict(B=2, T=4, page=16, start=[3, 4], absent="q", axes=(), norm=False),    # a plain store
]


@pytest.mark.parametrize("types", ["bf16", "fp16", "fp32 fp16"])
@pytest.mark.parametrize("case", PAGED, ids=lambda c: "-".join(f"{n}{c[n]}" for n in c).replace(" ", "")[:60])
def test_rope_into_pages(qi, case, types):
    x, dtype = types.split()[0], types.split()[-1]
    _check_rope(qi, x=x, dtype=dtype, seed=len(str(case)), **case)


@pytest.mark.parametrize("halves", [False, True])
def test_rope_in_place(qi, halves):
    _check_rope(qi, B=3, T=50, Hq=6, Hkv=2, halves=halves, axes=(64, 32), inplace=True)
    _check_rope(qi, B=3, T=50, Hq=6, Hkv=2, halves=halves, axes=(64, 32), inplace=True, layout="wide", lens=[50, 3, 0])


def test_rope_magnitudes(qi):
    """Heads of zeros, tiny and huge ones (squares that fp32 still holds), infinities and NaN in their own heads alone."""
    import torch
    x = _normal(3, 1, 6, 4, 128, dtype="fp32")
    scale = torch.tensor([0.0, 1e-18, 1e-6, 1.0, 1e6, 1e17], device="cuda").view(1, 6, 1, 1)
    x = x * scale
    w = torch.ones(128, device="cuda")
    rope = qi.rope((128,))
    got, _, _ = qi.qk_norm_rope(x, None, None, rope, q_w=w, dtype=torch.bfloat16)
    a = op.angles(np.arange(6)[None, :, None], op.frequencies((128,), 1e4), (64,))
    want, m = op.norm_rope(_np(x), np.ones(128), 1e-6, a, False)
    assert (np.abs(_np(got) - want) <= _rope_tol(want, m, a, "bf16", False)).all()
    clean = _normal(4, 1, 2, 3, 128)
    ref, _, _ = qi.qk_norm_rope(clean, None, None, qi.rope((64,)), q_w=w)
    for bad in (float("inf"), float("nan")):
        for dim in (0, 63, 64, 127):
            y = clean.clone()
            y[0, 1, 1, dim] = bad
            got, _, _ = qi.qk_norm_rope(y, None, None, qi.rope((64,)), q_w=w)
            keep = torch.ones(2, 3, dtype=torch.bool, device="cuda")
            keep[1, 1] = False
            assert torch.equal(got[0][keep], ref[0][keep]) and not torch.isfinite(got[0, 1, 1]).all()
            # without a norm, dims that are not rotated take nothing of their neighbours
            for halves in (False, True):
                got, _, _ = qi.qk_norm_rope(y, None, None, qi.rope((64,), halves=halves), pos=_int([[5, 9]]))
                wrong = (~torch.isfinite(got[0, 1, 1])).nonzero().flatten().tolist()
                pair = {dim} if dim >= 64 else {dim, dim ^ 1} if not halves else {dim, (dim + 32) % 64}
                assert set(wrong) == pair


def test_rope_refuses(qi):
    import torch
    q, k, v = (_normal(i, 2, 3, h, 128) for i, h in ((1, 4), (2, 2), (3, 2)))
    cache = qi.paged_kv(4, 16, 2, torch.float16)
    table, rope = _int([[0, 1], [2, 3]]), qi.rope()
    pos = torch.zeros(2, 3, 3, dtype=torch.int32, device="cuda")
    w = torch.ones(128, device="cuda")
    qi.qk_norm_rope(q, k, v, rope, pos=pos, cache=cache, table=table)
    for bad in (dict(q=q[..., :64]), dict(q=q[0]), dict(q=q.double()), dict(k=k.bfloat16()), dict(k=k.float()), dict(v=v[:, :2]),
                dict(v=v.cpu()), dict(k=k[:, :, :1]), dict(dtype=torch.bfloat16), dict(dtype=torch.float32),
                dict(pos=pos[..., :2]), dict(pos=pos.long()), dict(pos=pos[:1]), dict(rope=None), dict(q_w=w[:64]),
                dict(q_w=w.half()), dict(q_w=w, k_w=w.bfloat16()), dict(q=None, q_w=w), dict(cache=None), dict(table=None),
                dict(table=table[:1]), dict(table=table.long()), dict(table=table.t()), dict(start=table[0].long()),
                dict(start=_int([1, 2, 3])), dict(lens=_int([1])), dict(out=(q[:, :2], None, None)),
                dict(out=(None, k.clone(), None)), dict(out=(q.float(), None, None)), dict(cache=qi.paged_kv(4, 16, 3, torch.float16)),
                dict(cache=qi.paged_kv(4, 16, 2)), dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)),
                dict(rope=rope._replace(turns=rope.turns[:63])), dict(rope=rope._replace(turns=rope.turns.cpu()))):
        kw = dict(q=q, k=k, v=v, rope=rope, pos=pos, cache=cache, table=table)
        kw.update(bad)
        with pytest.raises(ValueError):
            qi.qk_norm_rope(**kw)
    with pytest.raises(qi.QiError):
        qi.qk_norm_rope(q[:, :, :1].expand(2, 3, 4, 128), k, v)      # heads that are one


# ---------------------------------------------------------------- attention


def _paged_case(qi, B, T, Hq, Hkv, kv_len, page, q_len=None, dtype="fp16", layout="plain", std=1.2, seed=0, width=None,
                max_len=None, garbage=True, share=False, bad_pages=()):
    """(arguments of paged_attention, what the oracle takes)"""
    import torch
    g = np.random.default_rng(seed)
    n = np.clip(kv_len, 0, None)
    cap = (max(1, -(-int(n.max()) // page)) if width is None else width)
    n = np.minimum(n, cap * page if max_len is None else max_len)
    need = [-(-int(x) // page) for x in n]
    total = sum(need) + 2
    order = g.permutation(total)
    table = g.choice([-1, 2 ** 31 - 1, -2 ** 31, total], (B, cap))       # entries behind a sequence may be anything
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    if share:
        table[1:, 0] = table[0, 0]
    for b, i, x in bad_pages:
        table[b, i] = x
    q = _normal(seed + 1, B, T, Hq, 128, std=std, dtype=dtype)
    k, v = _normal(seed + 2, total, page, Hkv, 128, std=std, dtype=dtype), _normal(seed + 3, total, page, Hkv, 128, dtype=dtype)
    ok, ov = _np(k), _np(v)
    if garbage:
        used = {}
        for b in range(B):
            for i in range(need[b]):
                p = int(table[b, i])
                used[p] = max(used.get(p, 0), min(page, int(n[b]) - i * page))
        for p in range(total):
            k[p, used.get(p, 0):], v[p, used.get(p, 0):] = float("nan"), float("inf")
    cache = qi.PagedKV(_spread(k, layout), _spread(v, layout))
    args = dict(q=_spread(q, layout), cache=cache, table=_int(table.tolist()), kv_len=_int(list(map(int, kv_len))),
                q_len=None if q_len is None else _int(q_len), max_len=max_len)
    return args, (_np(q), ok, ov, table, kv_len, q_len), cap * page if max_len is None else max_len


def _attn_tol(q, o, A, mag, vmax, n_most, dtype):
    ds = mag[..., None] * (128 * 2.0 ** -23 + 3 * 2.0 ** -24) + 2.0 ** -22
    return (U[dtype] * (A + np.abs(o)) * (1 + 2.0 ** -8) + 2 * ds * A + (2 * n_most * 2.0 ** -23 + 8 * 2.0 ** -22) * A
            + (n_most * 2.0 ** -25 * vmax[:, None, :, None] if dtype == "fp16" else 0.0) + 2.0 ** -25)


def _check_attn(qi, causal=True, **kw):
    import torch
    dtype = kw.get("dtype", "fp16")
    args, (q, k, v, table, kv_len, q_len), most = _paged_case(qi, **kw)
    B, T, Hq, _ = q.shape
    out = torch.full((B, T, Hq + 2, 128), 7.0, dtype=_dt(dtype), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if q_len is not None:   # rows of q behind a chunk may hold anything
        for b, r in enumerate(q_len):
            args["q"][b, max(0, r):] = float("nan")
    got = qi.paged_attention(causal=causal, out=out[:, :, 1:-1], status=status, **args)
    assert status.item() == 0
    assert (out[:, :, 0] == 7).all() and (out[:, :, -1] == 7).all()
    ref, A, mag, vmax, live = op.paged_attention(q, k, v, table, kv_len, q_len, causal, 1 / math.sqrt(128), most)
    got = _np(got)
    assert (got[~live] == 7).all()
    err, tol = np.abs(got - ref), _attn_tol(q, ref, A, mag, vmax, min(most, max(0, max(kv_len))), dtype)
    assert (got[live][A[live].sum((1, 2)) == 0] == 0).all()
    assert (err[live] <= tol[live]).all(), f"max error {np.nanmax(err[live]):.3e}, {np.nanmax(err[live] / tol[live]):.2f} of the bound"


ATTN = [
    dict(B=1, T=1, Hq=1, Hkv=1, kv_len=[1], page=16),
    dict(B=1, T=1, Hq=8, Hkv=2, kv_len=[17], page=16),
    dict(B=3, T=1, Hq=4, Hkv=4, kv_len=[0, 128, 129], page=16),
    dict(B=3, T=1, Hq=6, Hkv=2, kv_len=[127, 0, 300], page=32, layout="heads first"),
    dict(B=3, T=1, Hq=8, Hkv=1, kv_len=[255, 256, 257], page=64),
    dict(B=2, T=1, Hq=128, Hkv=1, kv_len=[200, 77], page=128),                     # the largest group
    dict(B=2, T=1, Hq=4, Hkv=2, kv_len=[513, 40], page=256, layout="wide"),
    dict(B=2, T=1, Hq=4, Hkv=2, kv_len=[700, 1300], page=1024),
    dict(B=4, T=5, Hq=6, Hkv=2, kv_len=[5, 6, 130, 3], page=16, q_len=[5, 3, 0, 5]),   # chunks shorter than T, none, longer than the past
    dict(B=3, T=2, Hq=4, Hkv=2, kv_len=[2, 1, 0], page=16),                        # rows before the first key
    dict(B=2, T=43, Hq=3, Hkv=1, kv_len=[50, 43], page=16),                        # 129 rows: just over a block
    dict(B=2, T=129, Hq=2, Hkv=2, kv_len=[259, 129], page=32, q_len=[129, 128]),
    dict(B=3, T=300, Hq=5, Hkv=1, kv_len=[300, 1000, 180], page=64, q_len=[300, 1, 180], layout="heads first"),
    dict(B=1, T=260, Hq=2, Hkv=2, kv_len=[667], page=128),
    dict(B=1, T=1, Hq=2, Hkv=1, kv_len=[6257], page=16),                           # split over the keys
    dict(B=1, T=200, Hq=2, Hkv=1, kv_len=[5001], page=64),
    dict(B=20, T=1, Hq=4, Hkv=4, kv_len=[97 * i for i in range(20)], page=16),
    dict(B=3, T=2, Hq=4, Hkv=2, kv_len=[2000000000, -7, 20], page=16, width=3, q_len=[7, 2, -1]),   # clamped
    dict(B=3, T=4, Hq=4, Hkv=2, kv_len=[60, 61, 200], page=16, max_len=61),
    dict(B=2, T=1, Hq=4, Hkv=2, kv_len=[60, 3], page=16, width=300),               # a table far wider than the sequences
    dict(B=4, T=3, Hq=4, Hkv=2, kv_len=[60, 33, 16, 90], page=16, share=True),     # a first page in common
    dict(B=2, T=3, Hq=4, Hkv=2, kv_len=[60, 200], page=16, bad_pages=[(0, 1, -1), (1, 0, 2 ** 31 - 1), (1, 12, 99)]),
    dict(B=40, T=1, Hq=8, Hkv=8, kv_len=[(37 * i) % 301 for i in range(40)], page=32),
    dict(B=1, T=1, Hq=200, Hkv=200, kv_len=[590], page=16),
    dict(B=30, T=20, Hq=12, Hkv=12, kv_len=[20 + (31 * i) % 91 for i in range(30)], page=16, q_len=[(7 * i) % 21 for i in range(30)]),
    dict(B=3, T=64, Hq=60, Hkv=60, kv_len=[164, 101, 64], page=32),
]
NAME = lambda c: "-".join(f"{n}{c[n]}" for n in c if n not in ("kv_len", "q_len")).replace(" ", "")[:60]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", ATTN, ids=NAME)
def test_attention(qi, case, dtype):
    _check_attn(qi, dtype=dtype, seed=len(str(case)), **case)


@pytest.mark.parametrize("case", [c for c in ATTN if "bad_pages" not in c][1::2], ids=NAME)
def test_attention_without_a_mask(qi, case):
    _check_attn(qi, causal=False, dtype="bf16", seed=len(str(case)), **case)


def test_attention_peaked_rows(qi):
    _check_attn(qi, B=2, T=40, Hq=2, Hkv=2, kv_len=[500, 77], page=16, std=6.0)
    _check_attn(qi, B=4, T=1, Hq=8, Hkv=2, kv_len=[3200, 77, 1, 0], page=64, std=6.0, dtype="bf16")


def test_attention_random_shapes(qi):
    rng = np.random.default_rng(7)
    for i in range(16):
        Hkv, G = int(rng.integers(1, 4)), int(rng.integers(1, 9))
        B, T = int(rng.integers(1, 8)), int(rng.choice([1, 1, 2, 7, 30, 150]))
        kv = [int(x) for x in rng.integers(0, 900, B)]
        ql = [int(x) for x in rng.integers(0, T + 1, B)] if rng.random() < 0.5 else None
        _check_attn(qi, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, kv_len=kv, q_len=ql, page=int(rng.choice([16, 32, 64, 128, 256])),
                    causal=bool(rng.random() < 0.6), dtype=["fp16", "bf16"][i % 2],
                    layout=["plain", "heads first", "wide"][i % 3], seed=i)


@pytest.mark.parametrize("T,causal", [(1, True), (3, True), (200, True), (200, False)])
def test_attention_is_that_of_own_keys_in_a_row(qi, T, causal):
    """What prefix_attention makes of the same rows without a prefix (both round probabilities and outputs once)."""
    import torch
    lens = [400, 201, 333]
    args, (q, k, v, table, *_), most = _paged_case(qi, B=3, T=T, Hq=8, Hkv=2, kv_len=lens, page=16, garbage=False, seed=9)
    rows = [torch.from_numpy(np.stack([op.rows_of(x, t, most) for t in table])).half().cuda() for x in (k, v)]
    a = qi.paged_attention(causal=causal, **args)
    b = qi.prefix_attention(args["q"], *rows, own_len=_int(lens), causal=causal)
    assert (a - b).abs().max() <= 4.5 * U["fp16"] * np.abs(v).max()
    assert torch.equal(a, qi.paged_attention(causal=causal, **args))


def test_attention_repeats_and_rows_are_independent(qi):
    import torch
    for T in (1, 3, 200):
        args, *_ = _paged_case(qi, B=4, T=T, Hq=8, Hkv=2, kv_len=[500, 777, 300, 201], page=32, seed=T, garbage=False)
        a = qi.paged_attention(**args)
        assert torch.equal(a, qi.paged_attention(**args))
        other = set(range(args["cache"].k.shape[0])) - set(args["table"][2, :10].tolist())
        for t in args["cache"]:
            t[sorted(other)] = _normal(77, len(other), *t.shape[1:])
        q2 = args["q"].clone()
        q2[[0, 1, 3]] = _normal(78, 3, *q2.shape[1:])
        assert torch.equal(a[2], qi.paged_attention(**{**args, "q": q2})[2])


def test_attention_refuses(qi):
    import torch
    args, *_ = _paged_case(qi, B=2, T=3, Hq=4, Hkv=2, kv_len=[60, 20], page=16)
    qi.paged_attention(**args)
    q, cache, table, n = args["q"], args["cache"], args["table"], args["kv_len"]
    for bad in (dict(q=q[..., :64]), dict(q=q.float()), dict(q=q[0]), dict(q=q.bfloat16()), dict(cache=qi.PagedKV(cache.k, cache.v[:2])),
                dict(cache=qi.PagedKV(cache.k, cache.v.cpu())), dict(cache=qi.PagedKV(cache.k[..., :64], cache.v[..., :64])),
                dict(cache=qi.PagedKV(cache.k[0], cache.v[0])), dict(table=table[:1]), dict(table=table.long()), dict(table=table.cpu()),
                dict(table=table.t().contiguous().t()), dict(kv_len=None), dict(kv_len=n.long()), dict(kv_len=n[:1]),
                dict(q_len=n[:1]), dict(out=q[:, :2]), dict(out=q.bfloat16()), dict(status=n)):
        with pytest.raises(ValueError):
            qi.paged_attention(**{**args, **bad})
    for bad in (dict(max_len=0), dict(max_len=65), dict(scale=0.0), dict(q=q[:, :, :3]), dict(q=q[:, :, :1].expand(2, 3, 4, 128)),
                dict(cache=qi.PagedKV(*(t[:, :12] for t in cache)), max_len=40)):
        with pytest.raises(qi.QiError):
            qi.paged_attention(**{**args, **bad})
