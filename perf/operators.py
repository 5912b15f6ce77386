"""Cases of the batch-serving operators: what a server that makes many images, or
continues many sequences, from one prompt runs beside the DiT pass.

* prefix_attention: attention of a batch whose sequences share one prompt's K/V (the
  prefix, in 16 bits or as the 8-bit cache holds it) and have keys of their own.
* kv8_write / kv8_read: K/V rows quantised to MXFP8 as they enter a cache (E4M3 codes,
  one power-of-two scale per 32 values), and read back in 16 bits.
* add_rmsnorm_mxfp8: the residual's addition, RMSNorm and the MXFP8 operand of the next
  block-scaled GEMM.

`run` computes an operator in elementary torch operations, or, with `own`, calls the
library's kernel. `exact` evaluates the definition in 64 bits.
"""
import math

import torch

own = False

D = 128   # head dimension
BLK = 32  # values that share a scale
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one image's first tokens against a short prompt: the smallest call, latency alone
        {"name": "attend one token", "op": "attn", "dtype": "fp16", "B": 1, "T": 1, "Hq": 32, "Hkv": 32, "P": 22,
         "S": 17, "causal": False, "ragged": False, "layout": "bshd", "bits": 16},
        # a batch of sequences continued token by token from one long shared prompt, grouped heads
        {"name": "decode, long shared prefix", "op": "attn", "dtype": "bf16", "B": 32, "T": 1, "Hq": 32, "Hkv": 8,
         "P": 8192, "S": 512, "causal": True, "ragged": True, "layout": "bshd", "bits": 16},
        # the same with the prompt held in 8 bits, a head of keys for each head of queries
        {"name": "decode, 8-bit prefix", "op": "attn", "dtype": "fp16", "B": 16, "T": 1, "Hq": 32, "Hkv": 32,
         "P": 8192, "S": 256, "causal": True, "ragged": True, "layout": "bhsd", "bits": 8},
        # a few drafted tokens per sequence checked at once: odd batch, group and lengths
        {"name": "drafted tokens, odd sizes", "op": "attn", "dtype": "bf16", "B": 7, "T": 5, "Hq": 24, "Hkv": 8,
         "P": 1531, "S": 333, "causal": True, "ragged": True, "layout": "bhsd", "bits": 16},
        # prompts that continue a shared one, run through in one pass
        {"name": "causal continuation", "op": "attn", "dtype": "bf16", "B": 3, "T": 777, "Hq": 32, "Hkv": 4,
         "P": 2048, "S": 1201, "causal": True, "ragged": True, "layout": "bshd", "bits": 16},
        # eight 384^2 images from one prompt of 494 text rows in the 8-bit cache
        {"name": "8 images at 384^2, 8-bit text", "op": "attn", "dtype": "fp16", "B": 8, "T": 576, "Hq": 32,
         "Hkv": 32, "P": 494, "S": 576, "causal": False, "ragged": False, "layout": "packed", "bits": 8},
        # four 1024^2 images from one prompt of 407 text rows: the largest
        {"name": "4 images at 1024^2", "op": "attn", "dtype": "fp16", "B": 4, "T": 4096, "Hq": 32, "Hkv": 32,
         "P": 407, "S": 4096, "causal": False, "ragged": False, "layout": "packed", "bits": 16},
        # one block's text K/V of a 407-row prompt stored after its capture
        {"name": "store 407 text rows", "op": "write", "dtype": "fp16", "B": 1, "T": 407, "H": 32, "S": 512,
         "ragged": False, "layout": "packed"},
        # a padded batch of prompts stored at once, each behind what its slot holds
        {"name": "store a padded batch", "op": "write", "dtype": "bf16", "B": 16, "T": 2048, "H": 8, "S": 4096,
         "ragged": True, "layout": "bshd"},
        # stored prompts brought back in 16 bits
        {"name": "read 4 prompts back", "op": "read", "dtype": "fp16", "B": 4, "T": 1999, "H": 32, "S": 2048,
         "ragged": True},
        # the residual stream of a 1024^2 joint pass into the next GEMM's operand
        {"name": "norm 4503 rows", "op": "norm", "x": "fp32", "delta": "fp16", "R": 4503, "K": 4096},
        # a handful of tokens
        {"name": "norm 3 rows", "op": "norm", "x": "bf16", "delta": "bf16", "R": 3, "K": 4096},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "write", "read", "norm"])
    if op == "attn":
        Hkv = rng.choice([1, 2, 4, 8, 16, 32])
        Hq = Hkv * rng.choice([g for g in (1, 2, 3, 4, 5, 8) if g * Hkv <= 40])
        T = _log(rng, 1, 4096)
        B = _log(rng, 1, 64)
        P = _log(rng, 1, 16384)
        S = max(T, _log(rng, 1, 4096))
        while B * T * Hq * (P + S) > 2e9:  # at most the largest listed case
            B, T, P = max(1, B // 2), max(1, T // 2), max(1, P * 3 // 4)
            S = max(T, S * 3 // 4)
        return {"op": op, "dtype": rng.choice(["fp16", "bf16"]), "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "P": P, "S": S,
                "causal": rng.random() < 0.6, "ragged": rng.random() < 0.6, "layout": rng.choice(["bshd", "bhsd"]),
                "bits": rng.choice([16, 16, 8])}
    if op == "norm":
        return {"op": op, "x": rng.choice(["fp32", "bf16", "fp16"]), "delta": rng.choice(["fp32", "bf16", "fp16"]),
                "R": _log(rng, 1, 9000), "K": 128 * _log(rng, 1, 96)}
    T = _log(rng, 1, 2500)
    case = {"op": op, "dtype": rng.choice(["fp16", "bf16"]), "B": _log(rng, 1, 16), "T": T,
            "H": rng.choice([1, 3, 4, 8, 32]), "S": T + _log(rng, 1, 1000), "ragged": rng.random() < 0.7}
    if op == "write":
        case["layout"] = rng.choice(["packed", "bshd"])
    return case


def _own_lens(c):
    """Own keys of each sequence: all of them, or spread over the upper half, the last sequence of three or more empty."""
    if not c["ragged"]:
        return [c["S"]] * c["B"]
    n = [max(1, c["S"] - (i * 5 % c["B"]) * c["S"] // (2 * c["B"])) for i in range(c["B"])]
    if c["B"] >= 3 and c["T"] == 1:
        n[-1] = 0
    return n


def _rows(c):
    """(first row, number of rows) of each sequence of a write or a read."""
    if not c["ragged"]:
        return [0] * c["B"], [c["T"]] * c["B"]
    room = c["S"] - c["T"]
    return ([(i * 7919) % (room + 1) for i in range(c["B"])], [max(1, c["T"] - (i * 3 % 8) * c["T"] // 8) for i in range(c["B"])])


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _quantise(v):
    """Codes [..., n] and scale bytes [..., n / 32] of 32-bit values, along the last axis."""
    b = v.unflatten(-1, (-1, BLK))
    top = b.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1] - 9, -127).clamp(-127, 127)
    q = torch.ldexp(b, -e.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.flatten(-2), (e + 127).to(torch.uint8)


def _values(q, s):
    """What codes (as bytes) and scale bytes stand for, in 32 bits."""
    b = q.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, BLK))
    return torch.ldexp(b, s.to(torch.int32).unsqueeze(-1) - 127).flatten(-2)


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    s = {"case": c}
    if c["op"] == "attn":
        dt, B, T, S, Hq, Hkv = DT[c["dtype"]], c["B"], c["T"], c["S"], c["Hq"], c["Hkv"]
        if c["layout"] == "packed":  # the projection's output as it stands: q, k and v side by side
            p = normal(B, T, Hq + 2 * Hkv, D, std=1.3, dtype=dt)
            s["q"], s["k"], s["v"] = p[:, :, :Hq], p[:, :, Hq:Hq + Hkv], p[:, :, Hq + Hkv:]
        else:
            s["q"] = normal(B, T, Hq, D, std=1.3, dtype=dt)
            for n in "kv":
                t = normal(B, Hkv, S, D, dtype=dt) if c["layout"] == "bhsd" else normal(B, S, Hkv, D, dtype=dt)
                s[n] = t.transpose(1, 2) if c["layout"] == "bhsd" else t
        s["pk"], s["pv"] = normal(c["P"], Hkv, D, std=1.3, dtype=dt), normal(c["P"], Hkv, D, dtype=dt)
        if c["bits"] == 8:  # the prompt as the 8-bit cache holds it
            for n in ("pk", "pv"):
                q, e = _quantise(s.pop(n).float())
                s[n + "8"], s[n + "_sf"] = q.view(torch.uint8), e
        s["lens"] = _int32(_own_lens(c)) if c["ragged"] else None
    elif c["op"] == "norm":
        # a residual stream with a few large channels, as trained models have
        big = 1.0 + 20.0 * (torch.rand(c["K"], generator=g, device="cuda") > 0.99)
        s["x"] = (normal(c["R"], c["K"], std=2.0) * big).to(DT[c["x"]])
        s["delta"] = normal(c["R"], c["K"], std=0.5, dtype=DT[c["delta"]])
        s["w"] = normal(c["K"], std=0.2, dtype=torch.bfloat16)
        s["x_out"] = torch.empty_like(s["x"])
        s["codes"] = torch.empty(c["R"], c["K"], dtype=torch.uint8, device="cuda")
        s["sf"] = torch.zeros(-(-c["R"] // 128) * (c["K"] // 128) * 512, dtype=torch.uint8, device="cuda")
    else:
        B, T, H, S, dt = c["B"], c["T"], c["H"], c["S"], DT[c["dtype"]]
        pos, n = _rows(c)
        s["pos"], s["lens"] = (_int32(pos), _int32(n)) if c["ragged"] else (None, None)
        scale = 2.0 ** torch.randint(-3, 4, (H, D), generator=g, device="cuda")  # channels of unlike size
        if c["op"] == "write":
            if c["layout"] == "packed":
                p = (normal(B, T, 3, H, D) * scale).to(dt)
                s["k"], s["v"] = p[:, :, 1], p[:, :, 2]
            else:
                s["k"], s["v"] = (normal(B, T, H, D) * scale).to(dt), (normal(B, T, H, D) * scale).to(dt)
            s["cache"] = [torch.zeros(B, S, H, n, dtype=torch.uint8, device="cuda") for n in (D, D, D // BLK, D // BLK)]
        else:
            kq, ke = _quantise((normal(B, S, H, D) * scale).to(dt).float())
            vq, ve = _quantise((normal(B, S, H, D) * scale).to(dt).float())
            s["cache"] = [kq.view(torch.uint8), vq.view(torch.uint8), ke, ve]
            s["out"] = [torch.zeros(B, T, H, D, dtype=dt, device="cuda") for _ in range(2)]
    return s


def run(state):
    s = state
    op = s["case"]["op"]
    return {"attn": _run_attn, "write": _run_write, "read": _run_read, "norm": _run_norm}[op](s)


def _run_attn(s):
    c = s["case"]
    if own:
        import diffusion_transformer_text_gb300 as qi
        if c["bits"] == 8:
            cache = qi.KV8Cache(s["pk8"], s["pv8"], s["pk_sf"], s["pv_sf"])
            return qi.prefix_attention(s["q"], s["k"], s["v"], prefix8=cache, own_len=s["lens"], causal=c["causal"])
        return qi.prefix_attention(s["q"], s["k"], s["v"], s["pk"], s["pv"], own_len=s["lens"], causal=c["causal"])
    B, T, S, G = c["B"], c["T"], c["S"], c["Hq"] // c["Hkv"]
    if c["bits"] == 8:
        pk, pv = _values(s["pk8"], s["pk_sf"]), _values(s["pv8"], s["pv_sf"])
    else:
        pk, pv = s["pk"].float(), s["pv"].float()
    q = s["q"].float().unflatten(2, (-1, G)).permute(0, 2, 3, 1, 4)  # [B, Hkv, G, T, D]
    k, v = s["k"].float().permute(0, 2, 1, 3), s["v"].float().permute(0, 2, 1, 3)  # [B, Hkv, S, D]
    shared = torch.einsum("bhgtd,phd->bhgtp", q, pk)
    mine = torch.einsum("bhgtd,bhsd->bhgts", q, k)
    n = s["lens"].view(B, 1, 1) if s["lens"] is not None else torch.full((1, 1, 1), S, device="cuda")
    last = n - T + 1 + torch.arange(T, device="cuda").view(1, T, 1) if c["causal"] else n
    seen = torch.arange(S, device="cuda").view(1, 1, S) < last  # [B or 1, T or 1, S]
    mine = mine.masked_fill(~seen.unsqueeze(1).unsqueeze(1), -math.inf)
    w = torch.cat([shared, mine], -1)
    del shared, mine
    w *= 1 / math.sqrt(D)
    w -= w.amax(-1, keepdim=True)  # the prefix is never empty here
    w = w.exp_()
    w /= w.sum(-1, keepdim=True)
    P = c["P"]
    o = torch.einsum("bhgtp,phd->bthgd", w[..., :P], pv) + torch.einsum("bhgts,bhsd->bthgd", w[..., P:], v)
    return o.flatten(2, 3).to(s["q"].dtype)


def _picked(s):
    """Which rows of the batch count, and the cache row of each."""
    c = s["case"]
    t = torch.arange(c["T"], device="cuda").view(1, -1)
    if s["pos"] is None:
        return t.expand(c["B"], -1) >= 0, t.expand(c["B"], -1)
    return t < s["lens"].view(-1, 1), t + s["pos"].view(-1, 1)


def _run_write(s):
    if own:
        import diffusion_transformer_text_gb300 as qi
        qi.kv8_write(qi.KV8Cache(*s["cache"]), s["k"], s["v"], pos=s["pos"], lens=s["lens"])
    else:
        use, row = _picked(s)
        b = torch.arange(s["case"]["B"], device="cuda").view(-1, 1).expand_as(row)
        at = (b[use], row[use])
        for x, codes, sf in ((s["k"], 0, 2), (s["v"], 1, 3)):
            q, e = _quantise(x[use].float())
            s["cache"][codes][at] = q.view(torch.uint8)
            s["cache"][sf][at] = e
    k, v, k_sf, v_sf = s["cache"]
    return {"k": k.view(torch.float8_e4m3fn), "v": v.view(torch.float8_e4m3fn), "k_sf": k_sf, "v_sf": v_sf}


def _run_read(s):
    c = s["case"]
    if own:
        import diffusion_transformer_text_gb300 as qi
        return qi.kv8_read(qi.KV8Cache(*s["cache"]), c["T"], DT[c["dtype"]], pos=s["pos"], lens=s["lens"], out=s["out"])
    use, row = _picked(s)
    b = torch.arange(c["B"], device="cuda").view(-1, 1).expand_as(row)
    at = (b[use], row[use])
    k, v, k_sf, v_sf = s["cache"]
    s["out"][0][use] = _values(k[at], k_sf[at]).to(DT[c["dtype"]])
    s["out"][1][use] = _values(v[at], v_sf[at]).to(DT[c["dtype"]])
    return s["out"][0], s["out"][1]


def _chunks(e, R, K):
    """Scale bytes [R, K / 32] in the GEMM's order: 512-byte chunks of 128 rows x 4 scales."""
    G = -(-R // 128)
    full = torch.zeros(G * 128, K // 32, dtype=e.dtype, device=e.device)
    full[:R] = e
    return full.view(G, 4, 32, K // 128, 4).permute(3, 0, 2, 1, 4).reshape(-1)


def _run_norm(s):
    c = s["case"]
    if own:
        import diffusion_transformer_text_gb300 as qi
        x, q, sf = qi.add_rmsnorm_mxfp8(s["x"], s["delta"], s["w"], plus_one=True, x_out=s["x_out"], q=s["codes"],
                                        sf=s["sf"])
    else:
        x = (s["x"].float() + s["delta"].float()).to(s["x"].dtype)
        f = x.float()
        y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6) * (1 + s["w"].float())
        q, e = _quantise(y)
        sf = _chunks(e, c["R"], c["K"])
    return {"x": x, "q": q.view(torch.float8_e4m3fn), "sf": sf.view(torch.float8_e8m0fnu)}


def work(case):
    c = case
    if c["op"] == "attn":
        lens = _own_lens(c)
        own_keys = sum(lens)
        if c["causal"]:
            pairs = sum(max(0, n - t) for n in lens for t in range(c["T"]))
        else:
            pairs = c["T"] * own_keys
        pairs += c["B"] * c["T"] * c["P"]
        row = 2 * c["Hkv"] * (D + D // BLK if c["bits"] == 8 else 2 * D)
        return {"bytes": c["P"] * row + own_keys * 4 * D * c["Hkv"] + 4 * D * c["B"] * c["T"] * c["Hq"],
                "flops": 4 * D * c["Hq"] * pairs}
    if c["op"] == "norm":
        size = {"fp32": 4, "fp16": 2, "bf16": 2}
        return {"bytes": c["R"] * (c["K"] * (2 * size[c["x"]] + size[c["delta"]] + 1) + c["K"] // 32) + 2 * c["K"],
                "flops": 7 * c["R"] * c["K"]}
    n = sum(_rows(c)[1]) * c["H"] * D * 2
    return {"bytes": 3 * n + n // 32, "flops": 3 * n}


# ---------------------------------------------------------------- the definitions in 64 bits


def _e4m3_64(v):
    """The nearest E4M3 values of 64-bit ones, ties to even, at most 448."""
    step = torch.exp2((torch.frexp(v.abs())[1] - 1).clamp(min=-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _blocks_64(v):
    """(codes' values, exponents) of 64-bit values in blocks of 32 along the last axis."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // BLK, BLK)
    top = b.abs().max(-1).values
    e = torch.where(top == 0, torch.full_like(top, -127), torch.frexp(top)[1].double() - 9)
    return _e4m3_64(b * torch.exp2(-e)[..., None]).reshape(v.shape), e


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "attn":
        if c["bits"] == 8:
            kv = []
            for n in ("pk", "pv"):
                e = s[n + "_sf"].double() - 127
                kv.append(s[n + "8"].view(torch.float8_e4m3fn).double() * torch.exp2(e).repeat_interleave(BLK, -1))
            pk, pv = kv
        else:
            pk, pv = s["pk"].double(), s["pv"].double()
        G, T = c["Hq"] // c["Hkv"], c["T"]
        o = torch.empty(c["B"], T, c["Hq"], D, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_own_lens(c)):
            for h in range(c["Hkv"]):
                keys = torch.cat([pk[:, h], s["k"][b, :n, h].double()])
                vals = torch.cat([pv[:, h], s["v"][b, :n, h].double()])
                for j in range(G):
                    a = s["q"][b, :, h * G + j].double() @ keys.T / math.sqrt(D)
                    if c["causal"]:
                        key = torch.arange(n, device="cuda")
                        tok = torch.arange(T, device="cuda")
                        a[:, c["P"]:][key[None, :] > tok[:, None] + (n - T)] = -math.inf
                    a = torch.exp(a - a.max(1, keepdim=True).values)
                    o[b, :, h * G + j] = a @ vals / a.sum(1, keepdim=True)
        return o
    if c["op"] == "norm":
        x = (s["x"].double() + s["delta"].double()).to(s["x"].dtype).double()  # the stream is stored in its type
        y = x / torch.sqrt((x * x).sum(1, keepdim=True) / c["K"] + 1e-6) * (1 + s["w"].double())
        q, e = _blocks_64(y)
        G = -(-c["R"] // 128)
        sf = torch.full((c["K"] // 128, G, 32, 4, 4), 2.0 ** -127, dtype=torch.float64, device="cuda")
        r = torch.arange(c["R"], device="cuda")[:, None]
        kb = torch.arange(c["K"] // 32, device="cuda")[None, :]
        sf[kb // 4, r // 128, r % 32, r % 128 // 32, kb % 4] = torch.exp2(e)
        return {"x": x, "q": q, "sf": sf.reshape(-1)}
    pos, lens = _rows(c)
    if c["op"] == "write":
        got = {}
        for n in "kv":
            z = torch.zeros(c["B"], c["S"], c["H"], D, dtype=torch.float64, device="cuda")
            for b in range(c["B"]):
                z[b, pos[b]:pos[b] + lens[b]] = _blocks_64(s[n][b, :lens[b]].double())[0]
            got[n], got[n + "_sf"] = z, None
        return got
    out = []
    for i in range(2):
        z = torch.zeros(c["B"], c["T"], c["H"], D, dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            at = slice(pos[b], pos[b] + lens[b])
            e = s["cache"][i + 2][b, at].double() - 127
            z[b, :lens[b]] = s["cache"][i][b, at].view(torch.float8_e4m3fn).double() * torch.exp2(e).repeat_interleave(BLK, -1)
        out.append(z)
    return tuple(out)
