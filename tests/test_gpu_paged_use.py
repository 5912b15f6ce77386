"""The paged operators as a server uses them: one after the other, captured and replayed while sequences grow, on
several streams and threads at once, over caches of more than 2^31 elements, and when a wait in a kernel expires."""
import math
import threading

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


def _rand(seed, *shape, std=1.0, dtype=None):
    import torch
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype or torch.float16)


def _int(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _np(t):
    return t.detach().double().cpu().numpy()


# sizes that reach every way of cutting the work: clusters, even pieces (few rows and many), units of one length,
# with their chunks joined and without
KINDS = [
    dict(B=2, T=1, Hq=8, Hkv=2, S=300, page=16),                   # one launch, chunks joined in a cluster
    dict(B=3, T=5, Hq=6, Hkv=2, S=900, page=32),
    dict(B=2, T=40, Hq=4, Hkv=2, S=600, page=16),
    dict(B=24, T=1, Hq=16, Hkv=8, S=1500, page=16),                # even pieces, few rows
    dict(B=1, T=1, Hq=8, Hkv=2, S=20000, page=64),
    dict(B=40, T=9, Hq=16, Hkv=4, S=700, page=64),                 # even pieces, blocks of up to 128 rows
    dict(B=6, T=400, Hq=16, Hkv=4, S=1500, page=16, ragged=True),
    dict(B=3, T=400, Hq=32, Hkv=4, S=3000, page=128),              # units of one length
    dict(B=1, T=300, Hq=8, Hkv=8, S=9000, page=64),                # ... their chunks' parts merged
    dict(B=30, T=1, Hq=8, Hkv=8, S=31, page=16),                   # more units than SMs, a tile each
]
NAME = lambda c: "-".join(f"{n}{c[n]}" for n in ("B", "T", "Hq", "Hkv", "S"))


def _case(qi, B, T, Hq, Hkv, S, page, ragged=False, seed=0, dtype=None):
    import torch
    rng = np.random.default_rng(seed + 1)
    need = -(-S // page)
    table = rng.permutation(B * need + 1)[:B * need].reshape(B, need)
    k, v = (_rand(seed + i, B * need + 1, page, Hkv, 128, dtype=dtype) for i in (2, 3))
    kw = dict(q=_rand(seed + 4, B, T, Hq, 128, dtype=dtype), cache=qi.PagedKV(k, v), table=_int(table.tolist()),
              kv_len=_int([S] * B), q_len=_int([T] * B) if ragged else None)
    return kw


def _grow(kw, step, T, S):
    """Lengths of another step of the same sequences, in place."""
    B = kw["kv_len"].shape[0]
    kw["kv_len"].copy_(_int([max(0, S - (7 * step + 131 * b * step) % (S + 1)) for b in range(B)]))
    if kw["q_len"] is not None:
        kw["q_len"].copy_(_int([(T - 53 * step * b) % (T + 1) for b in range(B)]))


@pytest.mark.parametrize("kind", KINDS, ids=NAME)
def test_graph_follows_lengths(qi, kind):
    """Captured once, replayed while sequences grow, shrink and end: all lengths are read when the kernels run."""
    import torch
    kw = _case(qi, **kind)
    out = torch.zeros_like(kw["q"])
    qi.paged_attention(out=out, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qi.paged_attention(out=out, **kw)
    for step in range(4):
        _grow(kw, step, kind["T"], kind["S"])
        out.zero_()
        g.replay()
        want = torch.zeros_like(out)
        qi.paged_attention(out=want, **kw)
        assert torch.equal(out, want)
    if kw["kv_len"].sum():
        assert out.any()


@pytest.mark.parametrize("kind", KINDS[1::2], ids=NAME)
def test_the_bound_on_lengths_changes_only_roundings(qi, kind):
    """max_len cuts the work another way; a larger table than the sequences need too."""
    import torch
    kw = _case(qi, **kind)
    S = kind["S"]
    kw["kv_len"].copy_(_int([max(1, S // 3 - 11 * b) for b in range(kind["B"])]))
    a = qi.paged_attention(**kw)
    A = float(kw["cache"].v.abs().max())
    wide = torch.cat([kw["table"], torch.full_like(kw["table"], -1).repeat(1, 30)], 1)
    for b in (qi.paged_attention(max_len=S // 3 + 1, **kw), qi.paged_attention(**{**kw, "table": wide})):
        # both are within 2 u (1 + small) of the exact row (test_gpu_paged.py)
        assert (a.float() - b.float()).abs().max() <= 4.5 * U["fp16"] * A


def test_two_graphs_at_once(qi):
    """Two captured chains, each with workspaces of its own graph, replayed side by side."""
    import torch
    sets = [[_case(qi, seed=50 * i + j, **KINDS[j]) for j in (3, 6, 8)] for i in range(2)]
    want = [[qi.paged_attention(**kw) for kw in s] for s in sets]
    graphs, outs = [], []
    for s in sets:
        g, o = torch.cuda.CUDAGraph(), [torch.zeros_like(kw["q"]) for kw in s]
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            for kw, x in zip(s, o):
                qi.paged_attention(out=x, **kw)
        graphs.append(g), outs.append(o)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(15):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(o, w))


def test_streams_and_memory_that_is_freed(qi):
    """Calls on other streams than the current one; what they were given may be dropped at once."""
    import torch
    sets = [_case(qi, seed=i, **KINDS[3]) for i in range(2)]
    want = [qi.paged_attention(**kw) for kw in sets]
    rope = qi.rope((128,))
    q = _rand(7, 24, 1, 16, 128)
    turned = qi.qk_norm_rope(q, None, None, rope, start=_int(list(range(24))))[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got, rot = [[], []], []
    for _ in range(12):
        for i, st in enumerate(streams):
            kw = {**sets[i], "q": sets[i]["q"].clone()}
            st.wait_stream(torch.cuda.current_stream())
            got[i].append(qi.paged_attention(stream=st, **kw))
            del kw
            x = q.clone()
            st.wait_stream(torch.cuda.current_stream())
            rot.append(qi.qk_norm_rope(x, None, None, rope, start=_int(list(range(24))), stream=st)[0])
            del x
            torch.full((24, 1, 16, 128), float("nan"), device="cuda", dtype=torch.float16)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])
    assert all(torch.equal(o, turned) for o in rot)
    with pytest.raises(ValueError, match="stream of|CUDA"):
        qi.paged_attention(**{**sets[0], "q": sets[0]["q"].cpu()})


def test_threads(qi):
    import torch
    sets = [_case(qi, seed=i, **KINDS[i]) for i in range(len(KINDS))]
    rope = qi.rope((64, 64), halves=True)
    pos = _int(np.arange(2 * 50).reshape(2, 50, 1).repeat(2, 2).tolist())
    x = _rand(5, 2, 50, 6, 128)
    want = [qi.paged_attention(**kw) for kw in sets]
    turned = qi.qk_norm_rope(x, x[:, :, :2], None, rope, pos)
    torch.cuda.synchronize()
    bad = []

    def work(n):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in range(20):
                    j = (n + i) % len(sets)
                    if not torch.equal(qi.paged_attention(**sets[j]), want[j]):
                        bad.append((n, j))
                    r = qi.qk_norm_rope(x, x[:, :, :2], None, rope, pos)
                    if not (torch.equal(r[0], turned[0]) and torch.equal(r[1], turned[1])):
                        bad.append((n, "rope"))
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad, bad[:3]


@pytest.mark.parametrize("kind", [dict(B=2, T=1, Hq=8, Hkv=2, S=700, page=16), dict(B=40, T=1, Hq=8, Hkv=8, S=900, page=16),
                                  dict(B=2, T=100, Hq=8, Hkv=2, S=700, page=16), dict(B=40, T=40, Hq=8, Hkv=2, S=900, page=16),
                                  dict(B=4, T=200, Hq=16, Hkv=8, S=900, page=16)], ids=NAME)
def test_an_expired_wait_is_told(qi, kind):
    """A launch whose Q never comes winds down within its waits' limit and says so; the next one is right."""
    import torch
    kw = _case(qi, **kind)
    want = qi.paged_attention(**kw)
    qi.prefix_attention_check()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qi.debug_inject(3)
    qi.paged_attention(status=status, **kw)
    torch.cuda.synchronize()
    assert status.item() != 0
    qi.prefix_attention_check()
    qi.debug_inject(3)
    qi.paged_attention(**kw)
    with pytest.raises(qi.QiError) as e:
        qi.prefix_attention_check()
    assert e.value.status == 6
    assert torch.equal(qi.paged_attention(**kw), want)
    qi.prefix_attention_check()


def test_far_pages(qi):
    """A cache of more than 2^31 elements, its last pages in use: written, and read back by attention."""
    import torch
    page, H, pages = 256, 8, 8400                # 8400 x 256 x 8 x 128 = 2.2e9 elements of K, and of V
    far = qi.PagedKV(*(torch.empty(pages, page, H, 128, dtype=torch.float16, device="cuda") for _ in range(2)))
    near = qi.paged_kv(4, page, H, torch.float16)
    B, T = 2, 300
    p = _rand(1, B, T, 16 + 2 * H, 128)
    rope, start = qi.rope((64, 64)), _int([0, 100])
    ids = [[pages - 1, 3], [pages - 3, pages - 2]]
    outs = []
    for cache, table in ((far, ids), (near, [[0, 1], [2, 3]])):
        t = _int(table)
        q, _, _ = qi.qk_norm_rope(p[:, :, :16], p[:, :, 16:24], p[:, :, 24:], rope, cache=cache, table=t, start=start)
        outs.append((q, qi.paged_attention(q, cache, t, start + T), qi.paged_attention(q[:, -1:], cache, t, start + T)))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    for c, n in zip(far, near):
        assert torch.equal(c[ids[0][0]], n[0]) and torch.equal(c[ids[1][0], 100:], n[2, 100:])


@pytest.mark.parametrize("dtype,halves", [("bf16", True), ("fp16", False)])
def test_prompts_in_chunks_then_tokens(qi, dtype, halves):
    """What a server does: prompts of unlike lengths run through in padded chunks, then token by token, each step the
    projection's fp32 rows through qk_norm_rope into pages and paged_attention over them. Every step against the
    float64 attention of the rows as the cache holds them, those rows against float64 norm and rotation."""
    import torch
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    u = U[dtype]
    B, Hq, Hkv, page, axes = 3, 6, 2, 16, (32, 48, 48)
    freqs, pairs = op.frequencies(axes, 1e4), tuple(a // 2 for a in axes)
    rope = qi.rope(axes, halves=halves)
    prompts, new = [70, 33, 1], 4
    longest = max(prompts) + new
    need = -(-longest // page)
    cache = qi.paged_kv(B * need + 2, page, Hkv, dt)
    table = np.random.default_rng(3).permutation(B * need + 2)[:B * need].reshape(B, need)
    dev_table = _int(table.tolist())
    w = [(1 + _rand(i, 128, std=0.2)).float() for i in (20, 21)]
    done = [0] * B
    rows_k = [np.zeros((0, Hkv, 128))] * B
    rows_v = [np.zeros((0, Hkv, 128))] * B
    step = 0
    while min(d - p for d, p in zip(done, prompts)) < new:
        T = 32 if any(d < p for d, p in zip(done, prompts)) else 1
        n = [min(T, p - d) if d < p else min(1, p + new - d) for d, p in zip(done, prompts)]
        x = _rand(100 + step, B, T, Hq + 2 * Hkv, 128, std=1.5, dtype=torch.float32)
        pos = np.stack([np.array([[d + t, 3 * (d + t) % 17, -(d + t)] for t in range(T)]) for d in done])
        start, lens = _int(done), _int(n)
        q, _, _ = qi.qk_norm_rope(x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], rope, _int(pos.tolist()), w[0], w[1],
                                  cache=cache, table=dev_table, start=start, lens=lens)
        kv = [d + m for d, m in zip(done, n)]
        o = qi.paged_attention(q, cache, dev_table, _int(kv), q_len=lens)
        a = op.angles(pos, freqs, pairs)
        xs = _np(x)
        ref_q, mq = op.norm_rope(xs[:, :, :Hq], _np(w[0]), 1e-6, a, halves)
        ref_k, mk = op.norm_rope(xs[:, :, Hq:Hq + Hkv], _np(w[1]), 1e-6, a, halves)
        pk, pv = _np(cache.k), _np(cache.v)
        for b in range(B):
            live = slice(0, n[b])
            # (bounds of test_gpu_paged.py, whose angle term is below 2^-40 here)
            tol = lambda y, m: u * np.abs(y) + m * 2.0 ** -19 + 2.0 ** -25
            assert (np.abs(_np(q)[b, live] - ref_q[b, live]) <= tol(ref_q[b, live], mq[b, live])).all()
            got_k, got_v = op.rows_of(pk, table[b], kv[b]), op.rows_of(pv, table[b], kv[b])
            assert (np.abs(got_k[done[b]:] - ref_k[b, live]) <= tol(ref_k[b, live], mk[b, live])).all()
            v = xs[b, live, Hq + Hkv:]
            assert (np.abs(got_v[done[b]:] - v) <= u * np.abs(v) + 2.0 ** -25).all()
            # rows of earlier steps are as they were
            assert (got_k[:done[b]] == rows_k[b]).all() and (got_v[:done[b]] == rows_v[b]).all()
            rows_k[b], rows_v[b] = got_k, got_v
        ref, A, mag, vmax, alive = op.paged_attention(_np(q), pk, pv, table, kv, n, True, 1 / math.sqrt(128), need * page)
        ds = mag[..., None] * (128 * 2.0 ** -23 + 3 * 2.0 ** -24) + 2.0 ** -22
        bound = (u * (A + np.abs(ref)) * (1 + 2.0 ** -8) + 2 * ds * A + (2 * longest * 2.0 ** -23 + 8 * 2.0 ** -22) * A
                 + (longest * 2.0 ** -25 * vmax[:, None, :, None] if dtype == "fp16" else 0.0) + 2.0 ** -25)
        got = _np(o)
        assert (np.abs(got - ref)[alive] <= bound[alive]).all()
        assert (got[~alive] == 0).all()
        done = kv
        step += 1
    assert step >= 6 and done == [p + new for p in prompts]


def test_images_from_one_prompt(qi):
    """Image rows of the fp32 projection to the shared-prefix attention: three axes, k and v to tensors. The cosines are
    those of the DiT's own tables up to their fp32 angles."""
    import torch
    L, h, w, H, n = 9, 6, 8, 4, 2
    N = h * w
    x = _rand(1, n, N, 3 * H, 128, dtype=torch.float32)
    pos = np.array([[L, y - (h - h // 2), z - (w - w // 2)] for y in range(h) for z in range(w)])
    q, k, v = qi.qk_norm_rope(x[:, :, :H], x[:, :, H:2 * H], x[:, :, 2 * H:], qi.rope(), _int(np.stack([pos] * n).tolist()),
                              dtype=torch.float16)
    _, _, ic, is_ = qi.rope_tables(L, h, w)
    c, s = (t.double().cpu().numpy()[None, :, None, :] for t in (ic, is_))
    for got, src in ((q, x[:, :, :H]), (k, x[:, :, H:2 * H])):
        y = _np(src)
        want = np.empty_like(y)
        want[..., 0::2] = y[..., 0::2] * c - y[..., 1::2] * s
        want[..., 1::2] = y[..., 1::2] * c + y[..., 0::2] * s
        m = np.repeat(np.abs(y[..., 0::2]) + np.abs(y[..., 1::2]), 2, -1)
        # the kernel's own bound, and the tables' angles: positions up to 9, off by 9 x 2^-23
        assert (np.abs(_np(got) - want) <= U["fp16"] * np.abs(want) + m * (2.0 ** -19 + 9 * 2.0 ** -23) + 2.0 ** -25).all()
    pk, pv = _rand(2, L, H, 128), _rand(3, L, H, 128)
    o = qi.prefix_attention(q, k, v, pk, pv)
    # the same rows in pages: the prompt's in each sequence's own
    rows = [torch.cat([torch.stack([p] * n), t], 1) for p, t in ((pk, k), (pv, v))]
    need = -(-(L + N) // 16)
    cache = qi.paged_kv(n * need, 16, H, torch.float16)
    for i in range(n):
        for t, r in zip(cache, rows):
            t[i * need:(i + 1) * need].view(-1, H, 128)[:L + N] = r[i]
    table = _int(np.arange(n * need).reshape(n, need).tolist())
    b = qi.paged_attention(q, cache, table, _int([L + N] * n), causal=False)
    A = float(max(t.abs().max() for t in (pv, v)))
    assert (o.float() - b.float()).abs().max() <= 4.5 * U["fp16"] * A


def test_captured_step(qi):
    """A decode step captured as one graph, rotation, store and attention, its positions kept on the device."""
    import torch
    B, Hq, Hkv, page, need = 4, 8, 2, 16, 6
    cache = qi.paged_kv(B * need, page, Hkv, torch.float16)
    table = _int(np.random.default_rng(1).permutation(B * need).reshape(B, need).tolist())
    rope = qi.rope((128,), halves=True)
    at, n = _int([0, 3, 15, 40]), _int([1, 4, 16, 41])
    for t in cache:
        t.normal_()
    start_cache = [t.clone() for t in cache]
    x = torch.empty(B, 1, Hq + 2 * Hkv, 128, dtype=torch.float16, device="cuda")
    q, o = (torch.empty(B, 1, Hq, 128, dtype=torch.float16, device="cuda") for _ in range(2))

    def step():
        qi.qk_norm_rope(x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], rope, out=(q, None, None), cache=cache,
                        table=table, start=at)
        qi.paged_attention(q, cache, table, n, out=o)
        at.add_(1), n.add_(1)

    xs = [_rand(i, *x.shape) for i in range(20)]
    want = []
    for s in xs:
        x.copy_(s)
        step()
        want.append(o.clone())
    final = [t.clone() for t in cache]
    for t, s in zip(cache, start_cache):
        t.copy_(s)
    at.copy_(_int([0, 3, 15, 40])), n.copy_(_int([1, 4, 16, 41]))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i, s in enumerate(xs):
        x.copy_(s)
        g.replay()
        assert torch.equal(o, want[i])
    assert all(torch.equal(a, b) for a, b in zip(cache, final))


@pytest.mark.parametrize("G", [4, 17])
def test_bound_far_above_the_lengths(qi, G):
    """So many sequences, and so long ones by max_len, that their tiles are not told in 32 bits; all on one page."""
    import torch
    B, page, width = 4200, 65536, 256
    q = _rand(1, B, 1, G, 128)
    k, v = _rand(2, 1, page, 1, 128), _rand(3, 1, page, 1, 128)
    n = np.random.default_rng(4).integers(0, 300, B)
    n[7], n[8] = 0, 1
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    o = qi.paged_attention(q, qi.PagedKV(k, v), table, _int(n.tolist()), max_len=width * page)
    s = torch.einsum("bhd,kd->bhk", q[:, 0].double(), k[0, :300, 0].double()) / math.sqrt(128)
    seen = torch.arange(300, device="cuda")[None, None] < _int(n.tolist())[:, None, None]
    w = torch.where(seen, torch.exp(s - s.amax(-1, keepdim=True)), 0.0)
    w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    want, size = w @ v[0, :300, 0].double(), w @ v[0, :300, 0].double().abs()
    # P and the output rounded to fp16, each by half a step of what it is part of; scores, sums and parts in fp32
    mag = torch.einsum("bhd,kd->bhk", q[:, 0].double().abs(), k[0, :300, 0].double().abs()).amax(-1, keepdim=True) / math.sqrt(128)
    ds = mag * (128 * 2.0 ** -23 + 3 * 2.0 ** -24) + 2.0 ** -22
    tol = (U["fp16"] * (size + want.abs()) * (1 + 2.0 ** -8) + (2 * ds + 2 * 300 * 2.0 ** -23 + 8 * 2.0 ** -22) * size
           + 300 * 2.0 ** -25 * v[0, :300, 0].double().abs().max() + 2.0 ** -25)
    err = (o[:, 0].double() - want).abs()
    assert (o[7] == 0).all()
    assert (err <= tol).all(), f"{(err / tol).max().item():.2f} of the bound"


@pytest.mark.parametrize("B,T,Hkv,causal", [(4, 260, 4, True), (8, 100, 8, True), (8, 100, 8, False)])
def test_pieces_in_several_rounds(qi, B, T, Hkv, causal):
    """More keys than the L2 holds, shared by several row blocks: the rows of some tokens against 64 bits."""
    import torch
    G, S, page = 4, 30000, 64
    kw = _case(qi, B, T, G * Hkv, Hkv, S, page, ragged=True, seed=5, dtype=torch.bfloat16)
    rng = np.random.default_rng(6)
    n, r = rng.integers(S // 3, S + 1, B), rng.integers(1, T + 1, B)
    n[1], r[2], r[0] = 5, 0, T
    kw["kv_len"].copy_(_int(n.tolist())), kw["q_len"].copy_(_int(r.tolist()))
    o = qi.paged_attention(causal=causal, **kw)
    again = qi.paged_attention(causal=causal, **kw)
    assert torch.equal(o, again)
    for b in range(B):
        assert (o[b, r[b]:] == 0).all()
        if r[b] == 0:
            continue
        rows = sorted({0, r[b] - 1, *(int(x) for x in rng.integers(0, r[b], 4))})
        pages = kw["table"][b, :-(-n[b] // page)].long()
        for h in range(Hkv):
            k, v = (kw["cache"][i][pages, :, h].flatten(0, 1)[:n[b]].double() for i in (0, 1))
            q = kw["q"][b, rows, h * G:(h + 1) * G].double()
            s = q @ k.T / math.sqrt(128)
            lim = torch.tensor([n[b] - r[b] + t + 1 if causal else n[b] for t in rows], device="cuda")
            s.masked_fill_(torch.arange(n[b], device="cuda") >= lim[:, None, None], -math.inf)
            w = torch.nan_to_num(torch.softmax(s, -1))  # (a row without a key)
            want, size = w @ v, w @ v.abs()
            # P and the output rounded to bf16, each by half a step of what it is part of; scores, sums, parts in fp32
            mag = (q.abs() @ k.abs().T).amax(-1, keepdim=True) / math.sqrt(128)
            ds = mag * (128 * 2.0 ** -23 + 3 * 2.0 ** -24) + 2.0 ** -22
            tol = (U["bf16"] * (size + want.abs()) * (1 + 2.0 ** -8) + (2 * ds + 2 * n[b] * 2.0 ** -23 + 8 * 2.0 ** -22) * size
                   + 2.0 ** -25)
            err = (o[b, rows, h * G:(h + 1) * G].double() - want).abs()
            assert (err <= tol).all(), f"{b} {h}: {(err / tol).max().item():.2f} of the bound"
