"""Benchmark cases of the operators around a paged key-value cache: per-head norms of queries
and keys with the rotation by their positions, the same pass writing keys and values into the
pages (16 bits or e4m3), reading sequences back from their pages, and attention of new tokens
over them.

Each operator has a plain form (elementary torch operations in fp32, angles in fp64) and the
library's call; `own` selects the second. `exact` is the definition in fp64.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
ESIZE = {"f16": 2, "bf16": 2, "e4m3": 1}


def listed():
    return [
        # one token's queries and keys between the QKV product and the attention (launch latency)
        dict(name="rotary_token", op="rotary", T=1, Hq=20, Hkv=4, D=64, R=64, dtype="f16", interleaved=False,
             norm=False, far=4096, stretch=1.0),
        # heads of 80 channels, half of them rotated, positions of a long context (stretched frequencies)
        dict(name="rotary_ragged", op="rotary", T=1031, Hq=12, Hkv=12, D=80, R=40, dtype="bf16", interleaved=True,
             norm=True, far=1000000, stretch=8.0),
        # images and text of the DiT: queries and keys of 24 heads normed and rotated
        dict(name="rotary_dit", op="rotary", T=4608, Hq=24, Hkv=24, D=128, R=128, dtype="f16", interleaved=True,
             norm=True, far=4608, stretch=1.0),
        # one token for each of 8 sequences into an 8-bit cache
        dict(name="write_tokens", op="write", T=8, Hq=32, Hkv=8, D=128, R=128, dtype="bf16", cache="e4m3", page=64,
             interleaved=False, norm=True, far=8191, stretch=1.0, skip=0, rotate=True),
        # keys and values as they are into 16-bit pages, padding among the tokens
        dict(name="write_ragged", op="write", T=777, Hq=0, Hkv=5, D=72, R=0, dtype="f16", cache="f16", page=16,
             interleaved=False, norm=False, far=777, stretch=1.0, skip=9, rotate=False),
        # a long prompt into an 8-bit cache
        dict(name="write_prompt", op="write", T=8191, Hq=32, Hkv=8, D=128, R=128, dtype="bf16", cache="e4m3", page=64,
             interleaved=False, norm=True, far=8191, stretch=1.0, skip=0, rotate=True),
        # three short sequences out of small pages
        dict(name="read_short", op="read", B=3, L=129, Hkv=4, D=64, dtype="f16", cache="f16", page=16),
        # 8 sequences of unequal lengths out of an 8-bit cache
        dict(name="read_long", op="read", B=8, L=8191, Hkv=8, D=128, dtype="bf16", cache="e4m3", page=64),
        # one token over a short text in 16-bit pages (latency), scores capped
        dict(name="attn_token", op="attn", B=1, n=1, chunks=0, L=333, Hq=20, Hkv=4, D=64, dtype="f16", cache="f16",
             page=16, cap=20.0, slopes=False),
        # one new token for each of 8 sequences of unequal lengths over the 8-bit cache
        dict(name="attn_tokens", op="attn", B=8, n=1, chunks=0, L=8191, Hq=32, Hkv=8, D=128, dtype="bf16",
             cache="e4m3", page=64, cap=0.0, slopes=False),
        # single tokens of most sequences beside chunks of prompts of the others, distance bias
        dict(name="attn_mixed", op="attn", B=16, n=1, chunks=3, L=4500, Hq=24, Hkv=8, D=128, dtype="f16",
             cache="e4m3", page=32, cap=0.0, slopes=True),
        # the last chunk of a long prompt
        dict(name="attn_prompt", op="attn", B=1, n=4095, chunks=0, L=16383, Hq=32, Hkv=8, D=128, dtype="bf16",
             cache="e4m3", page=64, cap=0.0, slopes=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "write", "read", "attn", "attn"])
    D = rng.choice([64, 128, 128, 72, 80, 40, 96])
    Hkv = rng.choice([1, 2, 4, 5, 8, 12])
    dtype = rng.choice(["f16", "bf16"])
    cache = rng.choice(["e4m3", dtype])
    page = rng.choice([16, 32, 64, 128])
    if op in ("rotary", "write"):
        Hq = Hkv * rng.choice([1, 1, 2, 4, 5])
        rotate = op == "rotary" or rng.random() < 0.7
        while True:
            T = _log(rng, 1, 8191)
            if T * (Hq + 2 * Hkv) * D <= 8191 * 48 * 128:
                break
        c = dict(op=op, T=T, Hq=Hq if rotate else 0, Hkv=Hkv, D=D, R=rng.choice([D, D, D // 2, 32]) if rotate else 0,
                 dtype=dtype, interleaved=rng.random() < 0.5, norm=rotate and rng.random() < 0.6,
                 far=_log(rng, 16, 1000000), stretch=rng.choice([1.0, 1.0, 4.0, 8.0]))
        return c if op == "rotary" else dict(c, cache=cache, page=page, skip=rng.randint(0, min(9, T - 1)), rotate=rotate)
    if op == "read":
        while True:
            B, L = _log(rng, 1, 32), _log(rng, 1, 16383)
            if B * L * Hkv * D <= 8 * 8191 * 8 * 128:
                break
        return dict(op="read", B=B, L=L, Hkv=Hkv, D=D, dtype=dtype, cache=cache, page=page)
    Hq = Hkv * rng.choice([1, 1, 2, 4, 5])
    while True:
        B, L = _log(rng, 1, 32), _log(rng, 1, 16383)
        kind = rng.choice(["tokens", "mixed", "prompt"])
        n = _log(rng, 1, min(L, 8)) if kind == "tokens" else _log(rng, 1, min(L, 4095)) if kind == "prompt" else 1
        c = dict(op="attn", B=B, n=n, chunks=rng.randint(1, 3) if kind == "mixed" else 0, L=L, Hq=Hq, Hkv=Hkv, D=D,
                 dtype=dtype, cache=cache, page=page, cap=rng.choice([0.0, 0.0, 0.0, 20.0]), slopes=rng.random() < 0.25)
        w = work(c)
        if w["flops"] <= 4 * 128 * 32 * 4095 * 12000 and w["bytes"] <= 8 * 8191 * 8 * 256 and max(
                k * s for k, s in zip(*_sequences(c))) * Hq <= 32 * 4095 * 16383:
            return c


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _lengths(B, L):
    """From the whole length down to half of it."""
    return [max(1, L - (L // 2) * b // B) for b in range(B)]


def _sequences(c):
    """(new tokens, tokens in the cache with them) of each sequence: n new ones each, but chunks
    of 1/8, 2/8 and 3/8 of the whole sequence for the last `chunks` of them."""
    held = _lengths(c["B"], c["L"])
    new = [min(c["n"], h) for h in held]
    for i in range(min(c["chunks"], c["B"])):
        new[-1 - i] = max(1, held[-1 - i] * (i + 1) // 8)
    return new, held


def _frequencies(R, stretch):
    """Radians per position, fp64. Stretched for a context longer than the trained one: the pairs
    that turn less than once in 4096 positions are slowed down by the factor, those that turn more
    than 32 times are kept, those between in part."""
    f = 10000.0 ** (-np.arange(0, R, 2, dtype=np.float64) / max(R, 1))
    if stretch != 1.0:
        turns = 4096 * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / 31.0, 0.0, 1.0)
        f = f * keep + f / stretch * (1.0 - keep)
    return torch.from_numpy(f).to(DEV)


def _heads(g, T, Hq, Hkv, D, t):
    """Slices of one QKV product; a few channels of the keys are far larger than the rest."""
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV)
    x[:, Hq:Hq + Hkv, torch.randperm(D, generator=g, device=DEV)[:max(1, D // 64)]] *= 8.0
    x = x.to(t)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _pool(g, pages, c):
    """Pages as another sequence left them, and the scales of an 8-bit cache's heads."""
    shape = (pages, c["Hkv"], c["page"], c["D"])
    k = torch.randn(shape, generator=g, device=DEV)
    v = torch.randn(shape, generator=g, device=DEV)
    if c["cache"] != "e4m3":
        return k.to(DTYPES[c["dtype"]]), v.to(DTYPES[c["dtype"]]), None, None
    # the largest |k| is about 30 before and after the norm, the largest |v| about 5
    ks = 0.08 * (1.0 + 0.5 * torch.rand(c["Hkv"], generator=g, device=DEV))
    vs = 0.012 * (1.0 + 0.5 * torch.rand(c["Hkv"], generator=g, device=DEV))
    s = (1, -1, 1, 1)
    return _codes(k, ks.view(s)), _codes(v, vs.view(s)), ks, vs


def _codes(x, scale):
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _tables(g, lengths, page):
    """int32 sequences x most pages: every sequence's pages, scattered over the pool; -1 behind
    its end. And the pages of the pool (an eighth of them is free)."""
    need = [-(-n // page) for n in lengths]
    total = sum(need) + max(1, sum(need) // 8)
    order = torch.randperm(total, generator=g, device=DEV).cpu().numpy().astype(np.int32)
    t = np.full((len(need), max(need)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t, total


def prepare(case, seed):
    c, g = case, _gen(seed)
    t = DTYPES[c["dtype"]]
    if c["op"] in ("rotary", "write"):
        T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
        q, k, v = _heads(g, T, Hq, Hkv, D, t)
        first = int(torch.randint(0, max(1, c["far"] - T + 1), (1,), generator=g, device=DEV))
        rotary = c["op"] == "rotary" or c["rotate"]
        s = dict(op=c["op"], q=q, k=k, v=v, interleaved=c["interleaved"], rotary=rotary,
                 positions=torch.arange(first, first + T, device=DEV, dtype=torch.int32) if rotary else None,
                 freqs=_frequencies(c["R"], c["stretch"]) if rotary else None,
                 factor=1.0 if c["stretch"] == 1.0 else 0.1 * math.log(c["stretch"]) + 1.0,
                 q_gain=1.0 + 0.2 * torch.randn(D, generator=g, device=DEV) if c["norm"] else None,
                 k_gain=1.0 + 0.2 * torch.randn(D, generator=g, device=DEV) if c["norm"] else None,
                 eps=EPS if c["norm"] else None,
                 q_out=torch.empty(T, Hq, D, device=DEV, dtype=t))
        if c["op"] == "rotary":
            s["k_out"] = torch.empty(T, Hkv, D, device=DEV, dtype=t)
            return s
        table, pages = _tables(g, [T], c["page"])
        at = np.arange(T)
        slots = table[0, at // c["page"]].astype(np.int64) * c["page"] + at % c["page"]
        if c["skip"]:
            slots[-c["skip"]:] = -1                          # padding: stored nowhere
        s["slots"] = torch.from_numpy(slots.astype(np.int32)).to(DEV)
        s["kept"] = (slots >= 0).nonzero()[0]
        s["k_pages"], s["v_pages"], s["ks"], s["vs"] = _pool(g, pages, c)
        return s
    if c["op"] == "read":
        held = _lengths(c["B"], c["L"])
        table, pages = _tables(g, held, c["page"])
        k, v, ks, vs = _pool(g, pages, c)
        shape = (c["B"], c["L"], c["Hkv"], c["D"])
        return dict(op="read", k_pages=k, v_pages=v, ks=ks, vs=vs, tables=torch.from_numpy(table).to(DEV), held=held,
                    lengths=torch.tensor(held, device=DEV, dtype=torch.int32),
                    k_out=torch.zeros(shape, device=DEV, dtype=t), v_out=torch.zeros(shape, device=DEV, dtype=t))
    new, held = _sequences(c)
    table, pages = _tables(g, held, c["page"])
    k, v, ks, vs = _pool(g, pages, c)
    T, Hq, D = sum(new), c["Hq"], c["D"]
    s = dict(op="attn", q=torch.randn(T, Hq, D, generator=g, device=DEV).to(t), k_pages=k, v_pages=v, ks=ks, vs=vs,
             tables=torch.from_numpy(table).to(DEV), new=new, held=held,
             lengths=torch.tensor(held, device=DEV, dtype=torch.int32),
             starts=torch.tensor([0] + list(np.cumsum(new)), device=DEV, dtype=torch.int32),
             out=torch.empty(T, Hq, D, device=DEV, dtype=t), scale=D ** -0.5, cap=c["cap"],
             slopes=torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=DEV) / Hq) if c["slopes"] else None, ws=None)
    if own:
        import bit_post_quantized_smooth_amd as sq
        need = sq.paged_attention_workspace_bytes(T, c["B"], table.shape[1] * c["page"], Hq, c["Hkv"], D)
        s["ws"] = torch.empty(need, device=DEV, dtype=torch.uint8)
    return s


# ---------------------------------------------------------------------------- one pass

def run(state):
    return _library(state) if own else _plain(state)


def _outputs(s):
    if s["op"] == "rotary":
        return dict(q=s["q_out"], k=s["k_out"])
    if s["op"] == "write":
        return dict(q=s["q_out"] if s["rotary"] else None, k_pages=s["k_pages"], v_pages=s["v_pages"])
    if s["op"] == "read":
        return dict(k=s["k_out"], v=s["v_out"])
    return s["out"]


def _library(s):
    import bit_post_quantized_smooth_amd as sq
    if s["op"] == "rotary":
        sq.norm_rotary(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["freqs"], factor=s["factor"],
                       interleaved=s["interleaved"], q_gain=s["q_gain"], k_gain=s["k_gain"], eps=s["eps"])
    elif s["op"] == "write" and s["rotary"]:
        sq.norm_rotary_write(s["q"], s["k"], s["v"], s["q_out"], s["slots"], s["k_pages"], s["v_pages"], s["ks"],
                             s["vs"], s["positions"], s["freqs"], factor=s["factor"], interleaved=s["interleaved"],
                             q_gain=s["q_gain"], k_gain=s["k_gain"], eps=s["eps"])
    elif s["op"] == "write":
        sq.paged_write(s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"], s["ks"], s["vs"])
    elif s["op"] == "read":
        sq.paged_read(s["k_pages"], s["v_pages"], s["tables"], s["lengths"], s["k_out"], s["v_out"], s["ks"], s["vs"])
    else:
        sq.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["tables"], s["lengths"], s["starts"], s["out"],
                           s["ks"], s["vs"], scale=s["scale"], softcap=s["cap"], slopes=s["slopes"], ws=s["ws"])
    return _outputs(s)


def _plain_heads(s, x, gain):
    """Normed and rotated heads in fp32."""
    x = x.float()
    if s["eps"] is not None:
        x = x * torch.rsqrt(x.square().mean(2, keepdim=True) + s["eps"]) * gain
    n = s["freqs"].shape[0]
    angle = (s["positions"].double()[:, None] * s["freqs"])[:, None]
    cos, sin = torch.cos(angle).float() * s["factor"], torch.sin(angle).float() * s["factor"]
    if s["interleaved"]:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _plain_store(s, x, pages, scales):
    page = pages.shape[2]
    slots = s["slots"].long()
    keep = slots >= 0
    slots, x = slots[keep], x[keep].float()
    x = x.to(pages.dtype) if scales is None else _codes(x, scales[:, None])
    as_bytes = torch.uint8 if scales is not None else pages.dtype
    pages.view(as_bytes)[slots // page, :, slots % page] = x.view(as_bytes)


def _plain_dense(s, name, b, n):
    """n tokens x heads x channels of sequence b in fp32."""
    pages = s[name + "_pages"]
    page = pages.shape[2]
    x = pages[s["tables"][b, :-(-n // page)].long()].float()
    if s[name + "s"] is not None:
        x = x * s[name + "s"][:, None, None]
    return x.transpose(1, 2).flatten(0, 1)[:n]


def _plain(s):
    if s["op"] == "rotary":
        s["q_out"].copy_(_plain_heads(s, s["q"], s["q_gain"]))
        s["k_out"].copy_(_plain_heads(s, s["k"], s["k_gain"]))
    elif s["op"] == "write":
        k = s["k"]
        if s["rotary"]:
            s["q_out"].copy_(_plain_heads(s, s["q"], s["q_gain"]))
            k = _plain_heads(s, k, s["k_gain"])
        _plain_store(s, k, s["k_pages"], s["ks"])
        _plain_store(s, s["v"], s["v_pages"], s["vs"])
    elif s["op"] == "read":
        for b, n in enumerate(s["held"]):
            s["k_out"][b, :n] = _plain_dense(s, "k", b, n).to(s["k_out"].dtype)
            s["v_out"][b, :n] = _plain_dense(s, "v", b, n).to(s["v_out"].dtype)
    else:
        at = 0
        for b, (n, held) in enumerate(zip(s["new"], s["held"])):
            k, v = (_plain_dense(s, name, b, held).permute(1, 0, 2) for name in "kv")
            Hkv, D = k.shape[0], k.shape[2]
            q = s["q"][at:at + n].float()
            Hq = q.shape[1]
            q = q.view(n, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
            x = torch.bmm(q, k.transpose(1, 2).contiguous()).view(Hq, n, held) * s["scale"]
            if s["cap"]:
                x = s["cap"] * torch.tanh(x / s["cap"])
            pos = torch.arange(held - n, held, device=x.device)[:, None]
            key = torch.arange(held, device=x.device)[None]
            if s["slopes"] is not None:
                x = x - s["slopes"][:, None, None] * (pos - key)
            x = x.masked_fill(key > pos, -math.inf)
            p = torch.exp(x - x.amax(2, keepdim=True))
            p = p / p.sum(2, keepdim=True)
            o = torch.bmm(p.view(Hkv, -1, held), v.contiguous()).view(Hq, n, D)
            s["out"][at:at + n] = o.transpose(0, 1).to(s["out"].dtype)
            at += n
    return _outputs(s)


# ---------------------------------------------------------------------------- costs and exact values

def work(case):
    c = case
    e = ESIZE[c["dtype"]]
    if c["op"] in ("rotary", "write"):
        T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
        flops = T * (Hq + Hkv) * (3 * c["R"] + (4 * D if c["norm"] else 0))
        if c["op"] == "rotary":
            return dict(bytes=2 * T * (Hq + Hkv) * D * e, flops=flops)
        kept = T - c["skip"]
        return dict(bytes=2 * T * Hq * D * e + 2 * kept * Hkv * D * (e + ESIZE[c["cache"]]) + 4 * T,
                    flops=flops + 2 * T * Hkv * D)
    if c["op"] == "read":
        n = sum(_lengths(c["B"], c["L"])) * 2 * c["Hkv"] * c["D"]
        return dict(bytes=n * (e + ESIZE[c["cache"]]), flops=n)
    new, held = _sequences(c)
    seen = sum(n * h - n * (n - 1) // 2 for n, h in zip(new, held))
    return dict(bytes=sum(held) * 2 * c["Hkv"] * c["D"] * ESIZE[c["cache"]] + 2 * sum(new) * c["Hq"] * c["D"] * e,
                flops=4 * c["D"] * c["Hq"] * seen)


def _exact_heads(c, s, x, gain):
    f64 = torch.float64
    y = x.to(f64)
    if c["norm"]:
        rms = (torch.linalg.vector_norm(y, dim=2) ** 2 / c["D"] + EPS).sqrt()
        y = y / rms[:, :, None] * gain.to(f64)
    out = y.clone()
    turn = s["positions"].to(f64)
    for i, f in enumerate(s["freqs"].tolist()):
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + len(s["freqs"]))
        z = torch.complex(y[:, :, a], y[:, :, b]) * torch.polar(
            torch.full_like(turn, s["factor"]), turn * f)[:, None]
        out[:, :, a], out[:, :, b] = z.real, z.imag
    return out


def _exact_store(s, x, pages, scales):
    out = pages.to(torch.float64)
    size = pages.shape[2]
    where = s["slots"].cpu().numpy()[s["kept"]]
    page, row = torch.from_numpy(where // size).to(DEV), torch.from_numpy(where % size).to(DEV)
    x = x.to(torch.float64)[torch.from_numpy(s["kept"]).to(DEV)]
    if scales is not None:
        x = torch.clamp(x / scales.to(torch.float64)[None, :, None], -E4M3_MAX, E4M3_MAX)
    out[page.long(), :, row.long()] = x
    return out


def _exact_sequence(s, name, b):
    """heads x tokens x channels in fp64, page by page."""
    pages, n = s[name + "_pages"], s["held"][b]
    ids = s["tables"][b].tolist()
    size = pages.shape[2]
    rows = torch.cat([pages[ids[i]].to(torch.float64) for i in range(-(-n // size))], dim=1)[:, :n]
    return rows if s[name + "s"] is None else rows * s[name + "s"].to(torch.float64).view(-1, 1, 1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rotary":
        return dict(q=_exact_heads(c, s, s["q"], s["q_gain"]), k=_exact_heads(c, s, s["k"], s["k_gain"]))
    if c["op"] == "write":
        k = _exact_heads(c, s, s["k"], s["k_gain"]) if c["rotate"] else s["k"]
        return dict(q=_exact_heads(c, s, s["q"], s["q_gain"]) if c["rotate"] else None,
                    k_pages=_exact_store(s, k, s["k_pages"], s["ks"]),
                    v_pages=_exact_store(s, s["v"], s["v_pages"], s["vs"]))
    if c["op"] == "read":
        out = dict(k=torch.zeros(s["k_out"].shape, dtype=torch.float64, device=DEV),
                   v=torch.zeros(s["v_out"].shape, dtype=torch.float64, device=DEV))
        for b, n in enumerate(s["held"]):
            for name in "kv":
                out[name][b, :n] = _exact_sequence(s, name, b).transpose(0, 1)
        return out
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, held) in enumerate(zip(s["new"], s["held"])):
        keys, values = _exact_sequence(s, "k", b), _exact_sequence(s, "v", b)
        age = (torch.arange(held - n, held, device=DEV, dtype=torch.float64)[:, None]
               - torch.arange(held, device=DEV, dtype=torch.float64)[None])
        for h in range(c["Hq"]):
            kv = h // (c["Hq"] // c["Hkv"])
            x = torch.mm(s["q"][at:at + n, h].to(torch.float64), keys[kv].t().contiguous()) / math.sqrt(c["D"])
            if c["cap"]:
                x = torch.tanh(x / c["cap"]) * c["cap"]
            if s["slopes"] is not None:
                x = x - float(s["slopes"][h]) * age
            x[age < 0] = -math.inf
            w = torch.exp(x - torch.logsumexp(x, dim=1, keepdim=True))
            out[at:at + n, h] = torch.mm(w, values[kv].contiguous())
        at += n
    return out
