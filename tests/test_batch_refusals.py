"""Refusals of the batch operators. Arguments are checked before any device work, so this runs without a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def qi():
    import diffusion_transformer_text_gb300 as q
    q.build()
    q.lib()
    return q


A = 4096  # an aligned address; nothing here is ever followed


def _attn(qi, **kw):
    """(status, message) of qi_prefix_attention on arguments that are right but for `kw`."""
    B, T, Hq, Hkv, P, S = (kw.pop(n, d) for n, d in (("B", 2), ("T", 3), ("Hq", 4), ("Hkv", 2), ("P", 5), ("S", 6)))
    f = dict(dtype=0, causal=0, scale=1.0, q=(A, T * Hq * 128, Hq * 128, 128), k=(A, S * Hkv * 128, Hkv * 128, 128),
             v=(A, S * Hkv * 128, Hkv * 128, 128), o=(A, T * Hq * 128, Hq * 128, 128), pk=(A, 0, Hkv * 128, 128),
             pv=(A, 0, Hkv * 128, 128), pk8=0, pv8=0, pk_sf=0, pv_sf=0, own_len=0, ws=0, ws_bytes=0, status=0)
    assert set(kw) <= set(f)
    f.update(kw)
    t = [f[n] for n in ("q", "k", "v", "o", "pk", "pv")]
    buf = qi._ATTN_HEAD.pack(*[x[0] for x in t], f["pk8"], f["pv8"], f["pk_sf"], f["pv_sf"], f["own_len"], f["ws"],
                             f["status"], f["causal"], f["scale"])
    buf += qi._ATTN_TAIL.pack(f["ws_bytes"], *[s for x in t for s in x[1:]], f["dtype"], B, T, Hq, Hkv, P, S)
    st = qi.lib().qi_prefix_attention(buf, None)
    return qi.STATUS[st], qi.lib().qi_last_error().decode()


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(B=65536), dict(T=0), dict(T=2 ** 24 + 1), dict(Hkv=0), dict(Hq=3), dict(Hq=1), dict(Hq=258, Hkv=2),
    dict(P=-1), dict(S=-1), dict(P=0, S=0), dict(P=2 ** 24 + 1), dict(S=2 ** 24 + 1), dict(B=65535, T=2 ** 20),
    dict(P=2 ** 20, Hkv=64, Hq=64, pk=(0, 0, 0, 0), pv=(0, 0, 0, 0), pk8=A, pv8=A, pk_sf=A, pv_sf=A),
])
def test_attention_shapes(qi, kw):
    st, msg = _attn(qi, **kw)
    assert st == "QI_ERR_SHAPE" and "qi_prefix_attention" in msg


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(dtype=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(q=(0, 512, 512, 128)), dict(o=(0, 512, 512, 128)), dict(k=(0, 512, 512, 128)), dict(v=(0, 512, 512, 128)),
    dict(pk=(0, 0, 256, 128)), dict(pv=(0, 0, 256, 128)),
    dict(q=(A + 8, 1536, 512, 128)), dict(k=(A, 1536, 260, 128)), dict(v=(A, 1536, 0, 128)), dict(o=(A, 1536, -512, 128)),
    dict(q=(A, 2 ** 38, 512, 128)), dict(pv=(A, 0, 256, 4)),
    dict(pk8=A), dict(pk8=A, pv8=A, pk_sf=A, pv_sf=A), dict(pk=(0, 0, 0, 0), pv=(0, 0, 0, 0), pk8=A, pv8=A, pk_sf=A),
    dict(pk=(0, 0, 0, 0), pv=(0, 0, 0, 0), pk8=A + 8, pv8=A, pk_sf=A, pv_sf=A),
    dict(pk=(0, 0, 0, 0), pv=(0, 0, 0, 0), pk8=A, pv8=A, pk_sf=A, pv_sf=A + 2), dict(own_len=A + 1), dict(status=A + 2),
])
def test_attention_arguments(qi, kw):
    assert _attn(qi, **kw)[0] == "QI_ERR_INVALID_ARG"


def test_null_structs(qi):
    assert qi.STATUS[qi.lib().qi_prefix_attention(None, None)] == "QI_ERR_INVALID_ARG"
    assert qi.lib().qi_prefix_attention_workspace(None) == 0
    assert qi.STATUS[qi.lib().qi_add_rmsnorm_mxfp8(None, None)] == "QI_ERR_INVALID_ARG"
    assert qi.STATUS[qi.lib().qi_kv8_write(None, None)] == qi.STATUS[qi.lib().qi_kv8_read(None, None)] == "QI_ERR_INVALID_ARG"


def _kv8(qi, name, **kw):
    f = dict(dtype=0, B=2, T=3, S=8, H=4, k=(A, 1536, 512, 128), v=(A, 1536, 512, 128), k8=A, v8=A, k_sf=A, v_sf=A,
             pos=0, lens=0)
    f.update(kw)
    k, v = (f[n] or (0, 8, 8, 8) for n in "kv")
    buf = qi._KV8_HEAD.pack(k[0], v[0], f["k8"], f["v8"], f["k_sf"], f["v_sf"], f["pos"], f["lens"])
    buf += qi._KV8_TAIL.pack(*k[1:], *v[1:], f["dtype"], f["B"], f["T"], f["S"], f["H"])
    return qi.STATUS[getattr(qi.lib(), "qi_kv8_" + name)(buf, None)]


@pytest.mark.parametrize("name", ["write", "read"])
@pytest.mark.parametrize("kw,want", [
    (dict(B=0), "SHAPE"), (dict(T=0), "SHAPE"), (dict(S=0), "SHAPE"), (dict(H=0), "SHAPE"), (dict(B=65536), "SHAPE"),
    (dict(T=2 ** 24 + 1), "SHAPE"), (dict(T=2 ** 16, H=2 ** 10), "SHAPE"), (dict(dtype=2), "INVALID_ARG"),
    (dict(k=None), "INVALID_ARG"), (dict(v=(0, 1536, 512, 128)), "INVALID_ARG"), (dict(k8=0), "INVALID_ARG"),
    (dict(v_sf=0), "INVALID_ARG"), (dict(k=(A + 2, 1536, 512, 128)), "INVALID_ARG"),
    (dict(v=(A, 1536, 516, 128)), "INVALID_ARG"), (dict(v8=A + 8), "INVALID_ARG"), (dict(k_sf=A + 1), "INVALID_ARG"),
    (dict(pos=A + 2), "INVALID_ARG"),
])
def test_kv8(qi, name, kw, want):
    assert _kv8(qi, name, **kw) == "QI_ERR_" + want


def _norm(qi, **kw):
    f = dict(xd=2, dd=0, rows=3, K=256, w32=0, plus=0, eps=1e-6, x=A, xs=256, d=A, ds=256, o=A, os=256, w=A, q=A, sf=A)
    f.update(kw)
    buf = qi._NORM_HEAD.pack(f["x"], f["d"], f["o"], f["w"], f["q"], f["sf"], f["plus"], f["eps"])
    buf += qi._NORM_TAIL.pack(f["xs"], f["ds"], f["os"], f["xd"], f["dd"], f["rows"], f["K"], f["w32"])
    return qi.STATUS[qi.lib().qi_add_rmsnorm_mxfp8(buf, None)]


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=192), "SHAPE"), (dict(K=16512), "SHAPE"),
    (dict(xd=3), "INVALID_ARG"), (dict(dd=-1), "INVALID_ARG"), (dict(x=0), "INVALID_ARG"), (dict(q=0), "INVALID_ARG"),
    (dict(sf=0), "INVALID_ARG"), (dict(x=A + 8), "INVALID_ARG"), (dict(d=A + 8), "INVALID_ARG"),
    (dict(o=A + 4), "INVALID_ARG"), (dict(w=A + 8), "INVALID_ARG"), (dict(q=A + 8), "INVALID_ARG"),
    (dict(xs=128), "INVALID_ARG"), (dict(xs=258), "INVALID_ARG"), (dict(ds=260), "INVALID_ARG"),
    (dict(os=-256), "INVALID_ARG"), (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG"),
    (dict(sf=A + 2), "INVALID_ARG"),
])
def test_norm(qi, kw, want):
    assert _norm(qi, **kw) == "QI_ERR_" + want


def test_python_checks(qi):
    import torch
    z = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt)
    with pytest.raises(ValueError, match="CUDA tensors"):
        qi.prefix_attention(z(1, 1, 2, 128), z(1, 1, 2, 128), z(1, 1, 2, 128))
    with pytest.raises(ValueError, match="CUDA tensors"):
        qi.kv8_write(qi.kv8_cache(1, 4, 2, device="cpu"), z(1, 1, 2, 128), z(1, 1, 2, 128))
    with pytest.raises(ValueError, match="CUDA tensors"):
        qi.add_rmsnorm_mxfp8(z(1, 128))
    cache = qi.kv8_cache(2, 4, 3, device="cpu")
    assert [tuple(t.shape) for t in cache.prefix(1, 2)] == [(2, 3, 128), (2, 3, 128), (2, 3, 4), (2, 3, 4)]
    for bad in ((2, 1), (-1, 1), (0, 0), (0, 5)):
        with pytest.raises(ValueError):
            cache.prefix(*bad)
