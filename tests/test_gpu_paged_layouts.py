"""Layouts and steps that the paged calls document and a server makes: a table that is a part of a wider one, K and V
rotated where they stand, and steps in which some sequences have one new token and others hundreds.

The first two are compared bit by bit with the same call on contiguous tables and with outputs of their own, which
test_gpu_paged.py holds to 64 bits; steps of unlike chunks are held to 64 bits here, by the bound of test_gpu_paged.py."""
import math

import numpy as np
import pytest

from oracle import paged as op
from test_gpu_paged import _attn_tol, _int, _normal, _np, _paged_case, _spread, qi  # noqa: F401  (qi: the fixture)

pytestmark = pytest.mark.gpu


def _wide(table, pages, seed):
    """The same table as the first columns, and rows, of a wider one whose other entries are pages too."""
    import torch
    g = np.random.default_rng(seed)
    B, n = table.shape
    wide = _int(g.integers(0, pages, (B + 2, n + 5)).tolist())
    wide[:B, :n] = table
    view = wide[:B, :n]
    assert view.stride(0) == n + 5 and torch.equal(view, table)
    return view


def _bits(t):
    import torch
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


ATTN = [
    dict(B=3, T=1, Hq=6, Hkv=2, kv_len=[127, 0, 300], page=32),                                  # joined in a cluster
    dict(B=24, T=1, Hq=16, Hkv=8, kv_len=[61 * i for i in range(24)], page=16),                  # pieces, few rows
    dict(B=40, T=9, Hq=16, Hkv=4, kv_len=[9 + 17 * i for i in range(40)], page=64),              # pieces, up to 128 rows
    dict(B=6, T=400, Hq=16, Hkv=4, kv_len=[1500, 400, 777, 1000, 401, 1200], page=16, q_len=[400, 1, 0, 399, 400, 7]),
    dict(B=3, T=400, Hq=32, Hkv=4, kv_len=[3000, 3000, 3000], page=128),                         # units
    dict(B=1, T=1, Hq=8, Hkv=2, kv_len=[3000], page=64),
]
NAME = lambda c: "-".join(f"{n}{c[n]}" for n in ("B", "T", "Hq", "Hkv", "page"))


@pytest.mark.parametrize("case", ATTN, ids=NAME)
def test_attention_by_a_part_of_a_wider_table(qi, case):  # noqa: F811
    import torch
    args, *_ = _paged_case(qi, seed=3, **case)
    want = qi.paged_attention(**args)
    assert want.any()
    args["table"] = _wide(args["table"], args["cache"].k.shape[0], 4)
    assert torch.equal(_bits(qi.paged_attention(**args)), _bits(want))


def _rope_case(seed, B, T, Hq, Hkv, dtype, layout):
    """q, k, v as three tensors, or as the heads of one, each in `layout` of test_gpu_paged.py."""
    if layout == "packed":
        p = _normal(seed, B, T, Hq + 2 * Hkv, 128, std=1.7, dtype=dtype)
        return p[:, :, :Hq], p[:, :, Hq:Hq + Hkv], p[:, :, Hq + Hkv:]
    return tuple(_spread(_normal(seed + i, B, T, h, 128, std=1.7, dtype=dtype), layout) for i, h in enumerate((Hq, Hkv, Hkv)))


@pytest.mark.parametrize("B,T,lens", [(1, 3, None), (3, 40, None), (3, 40, [40, 17, 0])])
def test_rotation_into_pages_by_a_part_of_a_wider_table(qi, B, T, lens):  # noqa: F811
    import torch
    page, need = 16, 6
    q, k, v = _rope_case(5, B, T, 5, 2, "bf16", "packed")
    table = _int(np.random.default_rng(6).permutation(B * need + 4)[:B * need].reshape(B, need).tolist())
    kw = dict(rope=qi.rope((64, 32)), start=_int([0, 9, 31][:B]), lens=None if lens is None else _int(lens))
    caches = []
    for t in (table, _wide(table, B * need + 4, 7)):
        cache = qi.PagedKV(*(_normal(8 + i, B * need + 4, page, 2, 128, dtype="bf16") for i in range(2)))
        before = [c.clone() for c in cache]
        rows = qi.qk_norm_rope(q, k, v, cache=cache, table=t, **kw)[0]
        assert all((c != b).any() for c, b in zip(cache, before))
        caches.append((rows, *cache))
    assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip(*caches))


@pytest.mark.parametrize("layout", ["packed", "plain", "heads first", "wide"])
@pytest.mark.parametrize("halves", [False, True], ids=["neighbours", "halves"])
@pytest.mark.parametrize("lens", [None, [50, 3, 0]], ids=["all", "padded"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rotation_of_all_three_in_place(qi, dtype, lens, halves, layout):  # noqa: F811
    import torch
    B, T = 3, 50
    ins = _rope_case(11, B, T, 6, 3, dtype, layout)
    kw = dict(rope=qi.rope((64, 32), halves=halves), lens=None if lens is None else _int(lens), start=_int([0, 7, 100]),
              q_w=_normal(14, 128, dtype="bf16"), k_w=_normal(15, 128, dtype="bf16"))
    before = [t.clone() for t in ins]
    want = qi.qk_norm_rope(*ins, **kw)
    assert all(torch.equal(_bits(t), _bits(b)) for t, b in zip(ins, before))
    got = qi.qk_norm_rope(*ins, out=ins, **kw)
    for g, t, w, b in zip(got, ins, want, before):
        assert g.data_ptr() == t.data_ptr()
        for i in range(B):
            n = T if lens is None else lens[i]
            assert torch.equal(_bits(t[i, :n]), _bits(w[i, :n])) and torch.equal(_bits(t[i, n:]), _bits(b[i, n:]))
    # what stands between and behind the rows is as it was
    if layout == "wide":
        for t, h in zip(ins, (6, 3, 3)):
            whole = torch.as_strided(t, (B, T, h + 3, 128), t.stride(), t.storage_offset() - 128)
            assert whole[:, :, 0].isnan().all() and whole[:, :, -2:].isnan().all()


# (chunk lengths, what the cache holds of each sequence with them)
MIXED = [
    dict(B=24, T=300, Hq=16, Hkv=4, page=16, q_len=[1] * 23 + [300], kv_len=[1 + 67 * i for i in range(23)] + [1500]),
    dict(B=24, T=300, Hq=16, Hkv=4, page=64, q_len=[300] + [1] * 22 + [0], kv_len=[300, *[1 + 67 * i for i in range(23)]]),
    dict(B=33, T=512, Hq=8, Hkv=2, page=32, q_len=[1] * 16 + [512] + [1] * 16, kv_len=[1000 - 29 * i for i in range(16)] + [2000] + [129] * 16),
    dict(B=40, T=257, Hq=12, Hkv=4, page=128, q_len=[1 if i % 5 else 257 - i for i in range(40)], kv_len=[300 + (37 * i) % 700 for i in range(40)]),
    dict(B=16, T=200, Hq=32, Hkv=32, page=16, q_len=[1, 200, 5, 1] * 4, kv_len=[400, 200, 5, 1] * 4),
    dict(B=9, T=130, Hq=40, Hkv=20, page=256, q_len=[1] * 8 + [130], kv_len=[0, 1, 127, 128, 129, 255, 256, 257, 700]),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", MIXED, ids=NAME)
def test_tokens_and_chunks_in_one_step(qi, case, dtype):  # noqa: F811
    import torch
    args, (q, k, v, table, kv_len, q_len), most = _paged_case(qi, seed=21, dtype=dtype, **case)
    for b, n in enumerate(q_len):  # rows of q behind a chunk may hold anything
        args["q"][b, n:] = float("nan")
    out = torch.full_like(args["q"], 7.0)
    qi.paged_attention(out=out, **args)
    ref, A, mag, vmax, live = op.paged_attention(q, k, v, table, kv_len, q_len, True, 1 / math.sqrt(128), most)
    got = _np(out)
    assert (got[~live] == 7).all()
    err, tol = np.abs(got - ref), _attn_tol(q, ref, A, mag, vmax, max(kv_len), dtype)
    assert (err[live] <= tol[live]).all(), f"{np.nanmax(err[live] / tol[live]):.2f} of the bound"
    # a single token of the step is what a call of it alone makes of it: the same sums, cut elsewhere
    one = [b for b, n in enumerate(q_len) if n == 1]
    alone = qi.paged_attention(args["q"][one, :1].contiguous(), args["cache"], args["table"][one].contiguous(),
                               args["kv_len"][one].contiguous())
    err = np.abs(_np(alone) - ref[one, :1])
    assert (err <= _attn_tol(q, ref, A, mag, vmax, max(kv_len), dtype)[one, :1]).all()
