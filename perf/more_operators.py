"""Cases of the operators between the projection and attention, and of attention over a cache in pages:
what a server that makes images, or continues sequences, of prompts that come and go runs beside the DiT pass.

* qk_norm_rope: RMSNorm of every head of q and k and the rotation by positions of several axes, in one pass
  over what the projection left; K and V go to tensors, or into the pages of a cache.
* paged_attention: attention of a chunk of new tokens (one token in decoding, a whole image, a piece of a
  prompt) over each sequence's keys and values, which lie in pages behind a table.

`run` computes an operator in elementary torch operations, or, with `own`, calls the library's kernel.
`exact` evaluates the definition in 64 bits.
"""
import math

import torch

own = False

D = 128      # head dimension
EPS = 1e-6
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}


def listed():
    return [
        # one token of one sequence on its way into the cache: latency alone
        {"name": "rotate one token into pages", "op": "rope", "x": "bf16", "dtype": "bf16", "B": 1, "T": 1, "Hq": 32,
         "Hkv": 8, "norm": True, "axes": "128", "theta": 1e6, "halves": True, "page": 16, "far": 100000,
         "ragged": False, "layout": "packed"},
        # a decode batch: single tokens of many sequences, each at its own place, one slot idle
        {"name": "rotate 64 tokens into pages", "op": "rope", "x": "bf16", "dtype": "bf16", "B": 64, "T": 1, "Hq": 32,
         "Hkv": 8, "norm": True, "axes": "128", "theta": 1e6, "halves": True, "page": 16, "far": 8192, "ragged": True,
         "layout": "packed"},
        # a padded batch of prompts stored as they are run through, a part of each head not rotated
        {"name": "rotate padded prompts into pages", "op": "rope", "x": "fp16", "dtype": "fp16", "B": 15, "T": 1499,
         "Hq": 24, "Hkv": 8, "norm": False, "axes": "64", "theta": 1e4, "halves": False, "page": 64, "far": 512,
         "ragged": True, "layout": "bshd"},
        # 1024^2 image rows as the fp32 product leaves them, three axes, to the attention's type
        {"name": "rotate 4096 image rows", "op": "rope", "x": "fp32", "dtype": "fp16", "B": 1, "T": 4096, "Hq": 32,
         "Hkv": 32, "norm": True, "axes": "16+56+56", "theta": 1e4, "halves": False, "page": 0, "far": 512,
         "ragged": False, "layout": "packed"},
        # 13 frames of 30 x 52 tokens: time, height and width
        {"name": "rotate a video", "op": "rope", "x": "bf16", "dtype": "bf16", "B": 1, "T": 20280, "Hq": 32, "Hkv": 32,
         "norm": True, "axes": "44+42+42", "theta": 1e4, "halves": False, "page": 0, "far": 1024, "ragged": False,
         "layout": "packed"},
        # the first token behind a short prompt: latency alone
        {"name": "attend one token in pages", "op": "attn", "dtype": "bf16", "B": 1, "T": 1, "Hq": 32, "Hkv": 8,
         "S": 23, "page": 16, "causal": True, "ragged": False, "layout": "pshd"},
        # a decode batch of sequences of unlike lengths, one slot idle
        {"name": "decode 64 sequences", "op": "attn", "dtype": "bf16", "B": 64, "T": 1, "Hq": 32, "Hkv": 8, "S": 4096,
         "page": 16, "causal": True, "ragged": True, "layout": "pshd"},
        # one sequence with a long past
        {"name": "decode one long sequence", "op": "attn", "dtype": "fp16", "B": 1, "T": 1, "Hq": 32, "Hkv": 8,
         "S": 131071, "page": 64, "causal": True, "ragged": False, "layout": "pshd"},
        # drafted tokens checked at once: odd batch, group and lengths
        {"name": "drafted tokens in pages", "op": "attn", "dtype": "fp16", "B": 7, "T": 5, "Hq": 24, "Hkv": 8,
         "S": 1861, "page": 32, "causal": True, "ragged": True, "layout": "phsd"},
        # a piece of a long prompt run through while it is filled in
        {"name": "a chunk of a long prompt", "op": "attn", "dtype": "bf16", "B": 1, "T": 1024, "Hq": 32, "Hkv": 8,
         "S": 16384, "page": 64, "causal": True, "ragged": False, "layout": "pshd"},
        # pieces of several prompts, unlike in length and past, padded to the longest
        {"name": "padded chunks", "op": "attn", "dtype": "bf16", "B": 6, "T": 777, "Hq": 32, "Hkv": 4, "S": 3001,
         "page": 16, "causal": True, "ragged": True, "layout": "pshd"},
        # four 1024^2 images, each behind a prompt of its own: the largest
        {"name": "4 images at 1024^2, own prompts", "op": "attn", "dtype": "fp16", "B": 4, "T": 4096, "Hq": 32,
         "Hkv": 32, "S": 4590, "page": 128, "causal": False, "ragged": True, "layout": "pshd"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    Hkv = rng.choice([1, 2, 4, 8, 16, 32])
    if rng.random() < 0.4:
        Hq = Hkv * rng.choice([g for g in (1, 2, 3, 4, 7, 8) if g * Hkv <= 40])
        B, T = _log(rng, 1, 64), _log(rng, 1, 20000)
        while B * T * (Hq + 2 * Hkv) > 20280 * 96:  # at most the largest listed case
            B, T = max(1, B * 2 // 3), max(1, T * 2 // 3)
        axes = rng.choice(["128", "64", "16+56+56", "44+42+42", "64+64", "32+32+32", "8+24+48+48"])
        dtype = rng.choice(["fp16", "bf16"])
        return {"op": "rope", "x": rng.choice([dtype, dtype, "fp32"]), "dtype": dtype, "B": B, "T": T, "Hq": Hq,
                "Hkv": Hkv, "norm": rng.random() < 0.7, "axes": axes, "theta": rng.choice([1e4, 5e5, 1e6]),
                "halves": rng.random() < 0.5, "page": rng.choice([0, 0, 16, 32, 64, 128, 256]),
                "far": _log(rng, 100, 1000000), "ragged": rng.random() < 0.5, "layout": rng.choice(["packed", "bshd"])}
    Hq = Hkv * rng.choice([g for g in (1, 2, 3, 4, 5, 8) if g * Hkv <= 40])
    B, T = _log(rng, 1, 128), _log(rng, 1, 4096) if rng.random() < 0.6 else 1
    S = max(T, _log(rng, 1, 131072))
    while B * T * Hq * S > 2e9 or B * S * Hkv > 4e6:  # at most the largest listed case
        B, T = max(1, B * 2 // 3), max(1, T * 3 // 4)
        S = max(T, S * 3 // 4)
    return {"op": "attn", "dtype": rng.choice(["fp16", "bf16"]), "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "S": S,
            "page": rng.choice([16, 32, 64, 128, 256]), "causal": rng.random() < 0.7, "ragged": rng.random() < 0.7,
            "layout": rng.choice(["pshd", "phsd"])}


def _axes(c):
    """Dims of each axis."""
    return [int(d) for d in c["axes"].split("+")]


def _rows(c):
    """New tokens of each sequence: all T, or from half of them up, the last of three or more single tokens none."""
    if not c["ragged"]:
        return [c["T"]] * c["B"]
    n = [max(1, c["T"] - (i * 3 % 8) * c["T"] // 14) for i in range(c["B"])]
    if c["B"] >= 3 and c["T"] == 1:
        n[-1] = 0
    return n


def _lens(c):
    """Rows of each sequence in the cache, the new ones among them: S, or spread between an eighth of it and all."""
    if not c["ragged"]:
        return [c["S"]] * c["B"]
    if not c["causal"]:  # whole images behind prompts: the prompts differ
        return [c["S"] - (i * 5 % 8) * (c["S"] - c["T"]) // 8 for i in range(c["B"])]
    return [0 if n == 0 else max(n, c["S"] - (i * 5 % 8) * c["S"] // 8) for i, n in enumerate(_rows(c))]


def _starts(c):
    """Where a sequence's new rows begin in the cache (its first position), for the rotation."""
    return [c["far"] // (1 + i % 5) for i in range(c["B"])] if c["ragged"] else [c["far"]] * c["B"]


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(lens, page, g):
    """int32 [B, M]: pages dealt out at random, -1 behind a sequence's last one; and the number of pages."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + 2
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _freqs(c):
    """Radians a position for each pair, float64, and the axis of each pair."""
    f, a = [], []
    for i, d in enumerate(_axes(c)):
        f += [c["theta"] ** (-2.0 * k / d) for k in range(d // 2)]
        a += [i] * (d // 2)
    return f, a


def _positions(c, g):
    """int32 [B, T, axes] of a sequence's tokens, or None for plain counting from its start."""
    A = len(_axes(c))
    if A == 1:
        return None
    if A == 3:  # (time, height, width) of frames, or of one image behind a prompt
        w = max(1, int(math.isqrt(c["T"])))
        t = torch.arange(c["T"], device="cuda")
        per = w * max(1, c["T"] // (w * 8))
        p = torch.stack([t // per + c["far"], t % per // w - 11, t % w - w // 2], -1)
        return p.expand(c["B"], -1, -1).to(torch.int32).contiguous()
    return torch.randint(-c["far"], c["far"], (c["B"], c["T"], A), generator=g, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        x = torch.empty(shape, dtype=dtype, device="cuda")
        return x.normal_(0.0, std, generator=g)

    s = {"case": c}
    B, T, Hq, Hkv, dt = c["B"], c["T"], c["Hq"], c["Hkv"], DT[c["dtype"]]
    if c["op"] == "rope":
        x = DT[c["x"]]
        if c["layout"] == "packed":  # the projection's output as it stands: q, k and v side by side
            p = normal(B, T, Hq + 2 * Hkv, D, std=1.7, dtype=x)
            s["q"], s["k"], s["v"] = p[:, :, :Hq], p[:, :, Hq:Hq + Hkv], p[:, :, Hq + Hkv:]
        else:
            s["q"], s["k"], s["v"] = (normal(B, T, h, D, std=1.7, dtype=x) for h in (Hq, Hkv, Hkv))
        if c["norm"]:
            s["q_w"], s["k_w"] = (1 + normal(D, std=0.2)).to(torch.bfloat16), (1 + normal(D, std=0.2)).to(torch.bfloat16)
        else:
            s["q_w"] = s["k_w"] = None
        s["pos"] = _positions(c, g)
        s["lens"] = _int32(_rows(c)) if c["ragged"] else None
        s["start"] = _int32(_starts(c))
        f, a = _freqs(c)
        s["freqs"], s["axis"] = torch.tensor(f, dtype=torch.float64, device="cuda"), torch.tensor(a, device="cuda")
        s["q_out"] = torch.zeros(B, T, Hq, D, dtype=dt, device="cuda")
        if c["page"]:
            # (the rows before the new ones are other calls': their part of the table holds one page that nobody has)
            first = [st // c["page"] for st in _starts(c)]
            last = [-(-(st + n) // c["page"]) for st, n in zip(_starts(c), _rows(c))]
            need = [max(0, e - f0) for f0, e in zip(first, last)]
            order = torch.randperm(sum(need) + 2, generator=g, device="cuda").to(torch.int32)
            table = torch.full((B, max(1, max(last))), -1, dtype=torch.int32, device="cuda")
            at = 0
            for b in range(B):
                table[b, first[b]:last[b]] = order[at:at + need[b]]
                at += need[b]
            s["table"] = table
            s["ck"], s["cv"] = (normal(sum(need) + 2, c["page"], Hkv, D, dtype=dt) for _ in range(2))
        else:
            s["ck"], s["cv"] = (torch.zeros(B, T, Hkv, D, dtype=dt, device="cuda") for _ in range(2))
        if own:
            import diffusion_transformer_text_gb300 as qi
            s["rope"] = qi.rope(tuple(_axes(c)), theta=c["theta"], halves=c["halves"])
        return s
    lens = _lens(c)
    s["table"], pages = _table(lens, c["page"], g)
    for n in "kv":
        if c["layout"] == "phsd":
            s["c" + n] = normal(pages, Hkv, c["page"], D, std=1.3 if n == "k" else 1.0, dtype=dt).transpose(1, 2)
        else:
            s["c" + n] = normal(pages, c["page"], Hkv, D, std=1.3 if n == "k" else 1.0, dtype=dt)
    s["q"] = normal(B, T, Hq, D, std=1.3, dtype=dt)
    s["lens"] = _int32(lens)
    s["rows"] = _int32(_rows(c)) if c["ragged"] and c["causal"] else None
    s["out"] = torch.zeros(B, T, Hq, D, dtype=dt, device="cuda")
    return s


def run(state):
    return _run_rope(state) if state["case"]["op"] == "rope" else _run_attn(state)


def _norm_rotate(x, w, cos, sin, C, halves):
    """[B, T, H, 128] of any type: norm if w is given, rotation by cos, sin [B, T, 1, C], in 32 bits."""
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
    if halves:
        a, b = y[..., :C], y[..., C:2 * C]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, y[..., 2 * C:]], -1)
    a, b = y[..., 0:2 * C:2], y[..., 1:2 * C:2]
    r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([r, y[..., 2 * C:]], -1)


def _run_rope(s):
    c = s["case"]
    if own:
        import diffusion_transformer_text_gb300 as qi
        if c["page"]:
            qi.qk_norm_rope(s["q"], s["k"], s["v"], s["rope"], pos=s["pos"], q_w=s["q_w"], k_w=s["k_w"], eps=EPS,
                            out=(s["q_out"], None, None), cache=qi.PagedKV(s["ck"], s["cv"]), table=s["table"],
                            start=s["start"], lens=s["lens"])
        else:
            qi.qk_norm_rope(s["q"], s["k"], s["v"], s["rope"], pos=s["pos"], q_w=s["q_w"], k_w=s["k_w"], eps=EPS,
                            out=(s["q_out"], s["ck"], s["cv"]), start=s["start"], lens=s["lens"])
        return s["q_out"], s["ck"], s["cv"]
    B, T, dt, C = c["B"], c["T"], s["q_out"].dtype, len(s["freqs"])
    t = torch.arange(T, device="cuda").view(1, -1)
    row = s["start"].view(-1, 1) + t  # [B, T]
    pos = row.unsqueeze(-1) if s["pos"] is None else s["pos"][..., s["axis"]]
    angle = pos.double() * s["freqs"]
    cos, sin = angle.cos().float().unsqueeze(2), angle.sin().float().unsqueeze(2)
    q = _norm_rotate(s["q"], s["q_w"], cos, sin, C, c["halves"]).to(dt)
    k = _norm_rotate(s["k"], s["k_w"], cos, sin, C, c["halves"]).to(dt)
    v = s["v"].to(dt)
    use = (t < s["lens"].view(-1, 1)) if s["lens"] is not None else (t >= 0).expand(B, -1)
    s["q_out"][use] = q[use]
    if c["page"]:
        page = s["table"].gather(1, (row // c["page"]).clamp(max=s["table"].shape[1] - 1).long())
        at = (page[use].long(), (row % c["page"])[use])
        s["ck"][at], s["cv"][at] = k[use], v[use]
    else:
        s["ck"][use], s["cv"][use] = k[use], v[use]
    return s["q_out"], s["ck"], s["cv"]


def _run_attn(s):
    c = s["case"]
    if own:
        import diffusion_transformer_text_gb300 as qi
        return qi.paged_attention(s["q"], qi.PagedKV(s["ck"], s["cv"]), s["table"], s["lens"], q_len=s["rows"],
                                  causal=c["causal"], out=s["out"])
    B, T, Hkv, G = c["B"], c["T"], c["Hkv"], c["Hq"] // c["Hkv"]
    n = s["lens"].view(B, 1, 1)
    ids = s["table"].clamp(min=0).long()
    S = ids.shape[1] * c["page"]
    k = s["ck"][ids].float().flatten(1, 2).permute(0, 2, 1, 3)  # [B, Hkv, S, D]
    q = s["q"].float().unflatten(2, (-1, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hkv, G T, D]
    w = torch.matmul(q, k.transpose(-1, -2)).unflatten(2, (G, T))
    del k
    t = torch.arange(T, device="cuda").view(1, T, 1)
    rows = s["rows"].view(B, 1, 1) if s["rows"] is not None else T
    last = n - rows + t + 1 if c["causal"] else n + 0 * t
    last = torch.minimum(last, n)
    seen = torch.arange(S, device="cuda").view(1, 1, S) < last  # [B, T, S]
    w *= 1 / math.sqrt(D)
    w.masked_fill_(~seen.unsqueeze(1).unsqueeze(1), -math.inf)
    top = w.amax(-1, keepdim=True)
    w -= top.masked_fill(top == -math.inf, 0.0)
    w = w.exp_()
    w /= w.sum(-1, keepdim=True).clamp(min=1e-30)  # a row without a key is zero
    v = s["cv"][ids].float().flatten(1, 2).permute(0, 2, 1, 3)
    o = torch.matmul(w.flatten(2, 3), v).unflatten(2, (G, T)).permute(0, 3, 1, 2, 4).flatten(2, 3).to(s["q"].dtype)
    if s["rows"] is None:
        s["out"].copy_(o)
    else:
        use = torch.arange(T, device="cuda").view(1, T) < s["rows"].view(B, 1)
        s["out"][use] = o[use]
    return s["out"]


def work(case):
    c = case
    if c["op"] == "rope":
        n = sum(_rows(c))
        values = n * (c["Hq"] + 2 * c["Hkv"]) * D
        A = 0 if len(_axes(c)) == 1 else 4 * len(_axes(c))
        return {"bytes": values * (SIZE[c["x"]] + SIZE[c["dtype"]]) + n * A,
                "flops": n * (c["Hq"] + c["Hkv"]) * D * (7 if c["norm"] else 3)}
    lens, rows = _lens(c), _rows(c) if c["causal"] else [c["T"]] * c["B"]
    if c["causal"]:
        pairs = sum(max(0, n - r + t + 1) for n, r in zip(lens, rows) for t in range(r))
    else:
        pairs = c["T"] * sum(lens)
    return {"bytes": sum(lens) * 4 * D * c["Hkv"] + 4 * D * sum(rows) * c["Hq"] + 4 * sum(-(-n // c["page"]) for n in lens),
            "flops": 4 * D * c["Hq"] * pairs}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    return _exact_rope(s, c) if c["op"] == "rope" else _exact_attn(s, c)


def _exact_rope(s, c):
    out, ck, cv = (s[n].double() for n in ("q_out", "ck", "cv"))
    C = sum(_axes(c)) // 2
    first = [C and sum(_axes(c)[:i]) // 2 for i in range(len(_axes(c)))]
    starts = _starts(c)
    for b, n in enumerate(_rows(c)):
        if n == 0:
            continue
        turn = torch.empty(n, C, dtype=torch.float64, device="cuda")
        for i, d in enumerate(_axes(c)):
            if s["pos"] is None:
                p = torch.arange(starts[b], starts[b] + n, dtype=torch.float64, device="cuda")
            else:
                p = s["pos"][b, :n, i].double()
            e = torch.arange(d // 2, dtype=torch.float64, device="cuda") * (-2.0 / d)
            turn[:, first[i]:first[i] + d // 2] = p[:, None] * torch.pow(torch.tensor(c["theta"], dtype=torch.float64, device="cuda"), e)[None]
        z = torch.polar(torch.ones_like(turn), turn)[:, None]  # [n, 1, C]
        for name, w in (("q", s["q_w"]), ("k", s["k_w"])):
            y = s[name][b, :n].double()
            if w is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + EPS) * w.double()
            if c["halves"]:
                r = torch.complex(y[..., :C].contiguous(), y[..., C:2 * C].contiguous()) * z
                y = torch.cat([r.real, r.imag, y[..., 2 * C:]], -1)
            else:
                r = torch.view_as_complex(y[..., :2 * C].unflatten(-1, (C, 2)).contiguous()) * z
                y = torch.cat([torch.view_as_real(r).flatten(-2), y[..., 2 * C:]], -1)
            if name == "q":
                out[b, :n] = y
            else:
                k = y
        v = s["v"][b, :n].double()
        if c["page"]:
            row = torch.arange(starts[b], starts[b] + n, device="cuda")
            page = s["table"][b][row // c["page"]].long()
            ck[page, row % c["page"]], cv[page, row % c["page"]] = k, v
        else:
            ck[b, :n], cv[b, :n] = k, v
    return out, ck, cv


def _exact_attn(s, c):
    G, T = c["Hq"] // c["Hkv"], c["T"]
    out = s["out"].double()
    rows = _rows(c) if c["causal"] else [T] * c["B"]
    for b, (n, r) in enumerate(zip(_lens(c), rows)):
        if n == 0 or r == 0:
            continue
        pages = s["table"][b, :-(-n // c["page"])].long()
        for h in range(c["Hkv"]):
            keys = s["ck"][pages, :, h].flatten(0, 1)[:n].double()
            vals = s["cv"][pages, :, h].flatten(0, 1)[:n].double()
            per = max(1, int(6e8) // n // r)  # heads at a time
            for j in range(0, G, per):
                x = s["q"][b, :r, h * G + j:min(h * G + j + per, (h + 1) * G)].double()  # [r, heads, D]
                m = x.shape[1]
                a = x.transpose(0, 1).reshape(m * r, D) @ keys.T / math.sqrt(D)
                if c["causal"]:
                    tok = torch.arange(r, device="cuda").repeat(m)
                    a[torch.arange(n, device="cuda")[None, :] > tok[:, None] + (n - r)] = -math.inf
                a = torch.exp(a - a.max(1, keepdim=True).values)
                o = a @ vals / a.sum(1, keepdim=True)
                out[b, :r, h * G + j:h * G + j + m] = o.reshape(m, r, D).transpose(0, 1)
    return out
