"""Refusals of the paged operators. Arguments are checked before any device work, so this runs without a GPU."""
import math
import struct

import pytest


@pytest.fixture(scope="module")
def qi():
    import diffusion_transformer_text_gb300 as q
    q.build()
    q.lib()
    return q


A = 4096  # an aligned address; nothing here is ever followed


def _rope(qi, **kw):
    """Status of qi_qk_norm_rope on arguments that are right but for `kw`."""
    f = dict(q=A, k=A, v=A, qo=A, ko=A, vo=A, q_w=A, k_w=A, pos=A, turns=A, start=0, lens=0, table=A, plus=0, eps=1e-6,
             qs=(1536, 512, 128), ks=(1536, 512, 128), vs=(1536, 512, 128), qos=(1536, 512, 128), kos=(8192, 256, 128),
             vos=(8192, 256, 128), ts=4, ind=0, d=0, wf=0, B=2, T=3, Hq=4, Hkv=2, axes=3, pairs=(8, 28, 28, 0), halves=0,
             pages=5, rows=32, width=4)
    assert set(kw) <= set(f)
    f.update(kw)
    buf = struct.pack("@13P", *[f[n] for n in ("q", "k", "v", "qo", "ko", "vo", "q_w", "k_w", "pos", "turns", "start",
                                               "lens", "table")]) + qi._ROPE_HEAD.pack(f["plus"], f["eps"])
    buf += qi._ROPE_TAIL.pack(*[x for n in ("qs", "ks", "vs", "qos", "kos", "vos") for x in f[n]], f["ts"], f["ind"],
                              f["d"], f["wf"], f["B"], f["T"], f["Hq"], f["Hkv"], f["axes"], *f["pairs"], f["halves"],
                              f["pages"], f["rows"], f["width"])
    st = qi.lib().qi_qk_norm_rope(buf, None)
    msg = qi.lib().qi_last_error().decode()
    assert "qi_qk_norm_rope" in msg
    return qi.STATUS[st]


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), "SHAPE"), (dict(B=65536), "SHAPE"), (dict(T=0), "SHAPE"), (dict(T=2 ** 24 + 1), "SHAPE"),
    (dict(Hq=-1), "SHAPE"), (dict(Hkv=65536), "SHAPE"), (dict(B=65535, T=2 ** 16), "SHAPE"), (dict(axes=5), "SHAPE"),
    (dict(axes=-1), "SHAPE"), (dict(pairs=(8, 29, 28, 0)), "SHAPE"), (dict(pairs=(65, 0, 0, 0)), "SHAPE"),
    (dict(pairs=(-1, 0, 0, 0)), "SHAPE"), (dict(halves=1, pairs=(8, 20, 27, 0)), "SHAPE"), (dict(rows=8), "SHAPE"),
    (dict(rows=48), "SHAPE"), (dict(rows=2 ** 17), "SHAPE"), (dict(pages=0), "SHAPE"), (dict(width=0), "SHAPE"),
    (dict(d=2), "INVALID_ARG"), (dict(d=-1), "INVALID_ARG"), (dict(ind=1), "INVALID_ARG"), (dict(ind=3), "INVALID_ARG"),
    (dict(q=0, k=0, v=0), "INVALID_ARG"), (dict(turns=0), "INVALID_ARG"), (dict(qo=0), "INVALID_ARG"),
    (dict(ko=0), "INVALID_ARG"), (dict(vo=0), "INVALID_ARG"), (dict(Hq=0), "INVALID_ARG"), (dict(Hkv=0), "INVALID_ARG"),
    (dict(k=0, v=0), "INVALID_ARG"), (dict(ts=3), "INVALID_ARG"), (dict(eps=-1.0), "INVALID_ARG"),
    (dict(eps=math.nan), "INVALID_ARG"), (dict(eps=math.inf), "INVALID_ARG"), (dict(q=A + 8), "INVALID_ARG"),
    (dict(ko=A + 8), "INVALID_ARG"), (dict(qs=(1536, 516, 128)), "INVALID_ARG"), (dict(vs=(0, 512, 128)), "INVALID_ARG"),
    (dict(kos=(8192, -256, 128)), "INVALID_ARG"), (dict(qos=(2 ** 38, 512, 128)), "INVALID_ARG"),
    (dict(ind=2, qs=(1536, 514, 128)), "INVALID_ARG"), (dict(q_w=A + 8), "INVALID_ARG"), (dict(turns=A + 4), "INVALID_ARG"),
    (dict(pos=A + 2), "INVALID_ARG"), (dict(start=A + 1), "INVALID_ARG"), (dict(lens=A + 2), "INVALID_ARG"),
    (dict(table=A + 2), "INVALID_ARG"),
])
def test_rope(qi, kw, want):
    assert _rope(qi, **kw) == "QI_ERR_" + want


def _attn(qi, **kw):
    f = dict(q=A, k=A, v=A, o=A, table=A, kv_len=A, q_len=0, ws=0, status=0, causal=1, scale=1.0, ws_bytes=0,
             qs=(1536, 512, 128), ks=(8192, 256, 128), vs=(8192, 256, 128), os=(1536, 512, 128), ts=4, d=0, B=2, T=3, Hq=4,
             Hkv=2, pages=5, rows=32, width=4, most=128)
    assert set(kw) <= set(f)
    f.update(kw)
    buf = struct.pack("@9P", *[f[n] for n in ("q", "k", "v", "o", "table", "kv_len", "q_len", "ws", "status")])
    buf += qi._PAGED_HEAD.pack(f["causal"], f["scale"])
    buf += qi._PAGED_TAIL.pack(f["ws_bytes"], *[x for n in ("qs", "ks", "vs", "os") for x in f[n]],
                               *[f[n] for n in ("ts", "d", "B", "T", "Hq", "Hkv", "pages", "rows", "width", "most")])
    st = qi.lib().qi_paged_attention(buf, None)
    assert "qi_paged_attention" in qi.lib().qi_last_error().decode()
    return qi.STATUS[st]


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), "SHAPE"), (dict(B=65536), "SHAPE"), (dict(T=0), "SHAPE"), (dict(T=2 ** 24 + 1), "SHAPE"),
    (dict(Hkv=0), "SHAPE"), (dict(Hq=3), "SHAPE"), (dict(Hq=1), "SHAPE"), (dict(Hq=258), "SHAPE"),
    (dict(B=65535, T=2 ** 20), "SHAPE"), (dict(rows=8), "SHAPE"), (dict(rows=24), "SHAPE"), (dict(rows=2 ** 17), "SHAPE"),
    (dict(pages=0), "SHAPE"), (dict(width=0), "SHAPE"), (dict(most=0), "SHAPE"), (dict(most=129), "SHAPE"),
    (dict(rows=65536, width=1000, most=2 ** 24 + 1), "SHAPE"),
    (dict(d=2), "INVALID_ARG"), (dict(d=-1), "INVALID_ARG"), (dict(q=0), "INVALID_ARG"), (dict(k=0), "INVALID_ARG"),
    (dict(v=0), "INVALID_ARG"), (dict(o=0), "INVALID_ARG"), (dict(table=0), "INVALID_ARG"), (dict(kv_len=0), "INVALID_ARG"),
    (dict(scale=0.0), "INVALID_ARG"), (dict(scale=-1.0), "INVALID_ARG"), (dict(scale=math.nan), "INVALID_ARG"),
    (dict(scale=math.inf), "INVALID_ARG"), (dict(q=A + 8), "INVALID_ARG"), (dict(ks=(8192, 260, 128)), "INVALID_ARG"),
    (dict(vs=(8192, 0, 128)), "INVALID_ARG"), (dict(os=(-1536, 512, 128)), "INVALID_ARG"),
    (dict(ks=(2 ** 38, 256, 128)), "INVALID_ARG"), (dict(ts=3), "INVALID_ARG"), (dict(table=A + 2), "INVALID_ARG"),
    (dict(kv_len=A + 1), "INVALID_ARG"), (dict(q_len=A + 2), "INVALID_ARG"), (dict(status=A + 2), "INVALID_ARG"),
])
def test_attention(qi, kw, want):
    assert _attn(qi, **kw) == "QI_ERR_" + want


def test_null_structs(qi):
    assert qi.STATUS[qi.lib().qi_qk_norm_rope(None, None)] == "QI_ERR_INVALID_ARG"
    assert qi.STATUS[qi.lib().qi_paged_attention(None, None)] == "QI_ERR_INVALID_ARG"
    assert qi.lib().qi_paged_attention_workspace(None) == 0


def test_python_checks(qi):
    import torch
    z = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    cache = qi.paged_kv(4, 16, 2, torch.float16, device="cpu")
    assert [tuple(t.shape) for t in cache] == [(4, 16, 2, 128)] * 2
    with pytest.raises(ValueError, match="CUDA tensors"):
        qi.qk_norm_rope(z(1, 1, 2, 128), None)
    with pytest.raises(ValueError, match="CUDA tensors"):
        qi.paged_attention(z(1, 1, 2, 128), cache, i(1, 4), i(1))
    with pytest.raises(ValueError, match="none of"):
        qi.qk_norm_rope(None, None)
    for rows in (0, 8, 24, -16):
        with pytest.raises(ValueError):
            qi.paged_kv(4, rows, 2, device="cpu")


def test_rope_handles(qi):
    r = qi.rope(device="cpu")
    assert r.pairs == (8, 28, 28) and r.turns.shape == (64,) and not r.halves
    # one position turns the first pair of each axis by one radian
    for at in (0, 8, 36):
        assert abs(int(r.turns[at]) / 2 ** 64 * 2 * math.pi - 1) < 2 ** -50
    f = [0.1 * k for k in range(8)]
    r = qi.rope((16,), freqs=f, halves=True, device="cpu")
    assert [round(int(t) / 2 ** 64 * 2 * math.pi, 12) for t in r.turns] == [round(x, 12) for x in f]
    # a frequency of more than half a circle a position is the same one modulo a circle
    r = qi.rope((2,), freqs=[2 * math.pi * 0.75], device="cpu")
    assert abs(int(r.turns[0]) / 2 ** 64 + 0.25) < 2 ** -50
    assert abs(int(qi.rope((2,), freqs=[-1.0], device="cpu").turns[0]) / 2 ** 64 * 2 * math.pi + 1) < 2 ** -50
    for bad in (dict(axes=()), dict(axes=(64, 66)), dict(axes=(3,)), dict(axes=(0, 64)), dict(axes=(8,) * 5),
                dict(axes=(24,), halves=True), dict(axes=(16,), freqs=[1.0]), dict(axes=(2,), freqs=[math.inf]),
                dict(theta=0.0), dict(theta=-2.0)):
        with pytest.raises(ValueError):
            qi.rope(device="cpu", **bad)


def test_descriptions_tell_layouts_apart(qi):
    """Equal bytes only for tensors of one type, device, shape and strides; addresses beside them."""
    import torch
    t = torch.zeros(4, 6, 8)
    same = qi._describe(t)[0]
    assert qi._describe(torch.ones(4, 6, 8))[0] == same
    others = [t.half(), t.int(), t[:3], t.transpose(0, 1), t[:, ::2], t.view(4, 48), t.view(2, 2, 6, 8), t[0], None,
              torch.zeros(4, 6, 8, device="meta")]
    keys = [qi._describe(x)[0] for x in others]
    assert len({same, *keys}) == len(others) + 1
    assert qi._describe(t, None)[0] != qi._describe(None, t)[0]
    assert struct.unpack("@3Q", qi._describe(t, None, t[1])[1]) == (t.data_ptr(), 0, t[1].data_ptr())
    for bad in (3, "x", [t]):
        with pytest.raises(TypeError):
            qi._describe(bad)
    with pytest.raises(ValueError):
        qi._describe(torch.eye(3).to_sparse())
    with pytest.raises(ValueError):
        qi._describe(*[t] * 25)
    with pytest.raises(ValueError):
        qi._describe(torch.zeros([1] * 9))


def test_longest_length_is_a_number(qi):
    """The plan is kept by max_len's value: what has none that holds, or could change, is no key."""
    import torch
    q, cache = torch.zeros(1, 1, 2, 128, dtype=torch.float16), qi.paged_kv(4, 16, 2, torch.float16, device="cpu")
    table, n = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for bad in (32.0, "32", [32]):
        with pytest.raises(TypeError):
            qi.paged_attention(q, cache, table, n, max_len=bad)


def test_library_without_torch(qi, monkeypatch, tmp_path):
    """The library is built and loaded without PyTorch; only what takes tensors wants the compiled reader."""
    import importlib
    import subprocess
    import sys
    code = "import sys, diffusion_transformer_text_gb300 as q; q.lib(); assert 'torch' not in sys.modules"
    subprocess.run([sys.executable, "-c", code], check=True, cwd=importlib.import_module("oracle").__path__[0] + "/..")
    b = importlib.import_module("diffusion_transformer_text_gb300.build")
    monkeypatch.setattr(b, "_torch_dir", lambda: None)
    monkeypatch.setattr(b, "TENSORS", str(tmp_path / "absent.so"))
    b._build_tensors()
    assert b._torch_version() == "" and not (tmp_path / "absent.so").exists()
