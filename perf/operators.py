"""Benchmark cases of the 8-bit attention block's operators: the residual's addition with RMS
norm and 8-bit quantization, the 8-bit block-scaled matrix product, and masked attention.

Each operator has a plain form (elementary torch operations in fp32) and the library's call; `own`
selects the second. `exact` is the definition in fp64.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128            # channels per scale
E4M3_MAX = 448.0
TINY = 2.0 ** -126     # smallest scale
DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # residual + norm + quantize: one token of a UNet-width model (launch latency)
        dict(name="norm_token", op="norm", M=1, K=1280, dtype="bf16", residual=True),
        # fp32 activations of an odd width: rows that are neither 16-byte nor block aligned
        dict(name="norm_ragged_f32", op="norm", M=1031, K=1001, dtype="f32", residual=False),
        # the wide side of the DiT MLP pair, whole prompt
        dict(name="norm_mlp", op="norm", M=4608, K=12288, dtype="bf16", residual=True),
        # one token through the UNet's widest projection: weights read once
        dict(name="gemm_token", op="gemm", M=1, N=10240, K=1280, out="bf16", bias=True, act=False),
        # a small batch through the MLP's down-projection: long K, few rows
        dict(name="gemm_few_rows", op="gemm", M=24, N=3072, K=12288, out="f16", bias=True, act=False),
        # ragged in every size, with the MLP's activation and fp32 output
        dict(name="gemm_ragged_f32", op="gemm", M=1023, N=1283, K=1272, out="f32", bias=True, act=True),
        # the DiT's fused QKV projection
        dict(name="gemm_dit_qkv", op="gemm", M=4608, N=9216, K=3072, out="f16", bias=True, act=False),
        # a text encoder's prompt: causal, scores capped
        dict(name="attn_text", op="attn", B=2, Lq=77, Lk=77, Hq=12, Hkv=12, D=64, dtype="f16",
             causal=True, prefix=0, docs=0, lens=False, cap=20.0, slopes=False, fused=True),
        # one new token for each of 8 sequences of unequal lengths, grouped heads, distance bias
        dict(name="attn_token", op="attn", B=8, Lq=1, Lk=8191, Hq=32, Hkv=8, D=128, dtype="bf16",
             causal=False, prefix=0, docs=0, lens=True, cap=0.0, slopes=True, fused=False),
        # images and text of the DiT in one sequence, every token sees every token
        dict(name="attn_dit", op="attn", B=1, Lq=4608, Lk=4608, Hq=24, Hkv=24, D=128, dtype="f16",
             causal=False, prefix=0, docs=0, lens=False, cap=0.0, slopes=False, fused=True),
        # the same with three prompts packed into the sequence and padding behind them
        dict(name="attn_dit_packed", op="attn", B=1, Lq=4608, Lk=4608, Hq=24, Hkv=24, D=128,
             dtype="f16", causal=False, prefix=0, docs=3, lens=False, cap=0.0, slopes=False, fused=True),
        # a long prompt with a bidirectional prefix, grouped heads and capped scores
        dict(name="attn_prefix", op="attn", B=1, Lq=8191, Lk=8191, Hq=16, Hkv=4, D=128, dtype="bf16",
             causal=True, prefix=1000, docs=0, lens=False, cap=30.0, slopes=False, fused=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gemm", "attn"])
    if op == "norm":
        while True:
            M, K = _log(rng, 1, 16384), _log(rng, 64, 12288)
            if M * K <= 4608 * 12288:
                break
        if rng.random() < 0.6:
            K = -(-K // 8) * 8
        return dict(op="norm", M=M, K=K, dtype=rng.choice(["f16", "bf16", "f32"]), residual=rng.random() < 0.6)
    if op == "gemm":
        while True:
            M, N, K = _log(rng, 1, 9216), _log(rng, 64, 12288), _log(rng, 64, 12288)
            if M * N * K <= 4608 * 3072 * 9216:
                break
        return dict(op="gemm", M=M, N=N, K=K, out=rng.choice(["f16", "bf16", "f32"]),
                    bias=rng.random() < 0.7, act=rng.random() < 0.2)
    D = rng.choice([64, 128, 128, 72, 80, 40])
    Hkv = rng.choice([1, 2, 4, 8, 12, 16])
    Hq = Hkv * rng.choice([1, 1, 2, 4, 8])
    kind = rng.choice(["prompt", "token", "causal", "packed", "cross"])
    while True:
        B, Lk = _log(rng, 1, 8), _log(rng, 16, 16384)
        Lq = _log(rng, 1, 8) if kind == "token" else _log(rng, 16, 4608) if kind == "cross" else Lk
        if Lq <= Lk and B * Hq * Lq * Lk <= 16 * 8191 * 8191 and B * Hkv * Lk * D <= 8 * 8 * 8191 * 128:
            break
    return dict(op="attn", B=B, Lq=Lq, Lk=Lk, Hq=Hq, Hkv=Hkv, D=D, dtype=rng.choice(["f16", "bf16"]),
                causal=kind == "causal" or (kind == "token" and Lq > 1),
                prefix=rng.randint(1, Lk) if kind == "causal" and rng.random() < 0.5 else 0,
                docs=rng.randint(2, 6) if kind == "packed" else 0,
                lens=kind == "token" and Lq == 1,
                cap=rng.choice([0.0, 0.0, 20.0, 50.0]), slopes=rng.random() < 0.3,
                fused=Lq == Lk)


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _activation(g, M, K):
    """N(0, 1) with 1% of the channels times 20: a transformer's outlier channels."""
    x = torch.randn(M, K, generator=g, device=DEV)
    hot = torch.randperm(K, generator=g, device=DEV)[:max(1, K // 100)]
    x[:, hot] *= 20.0
    return x


def _pad(K):
    return -(-K // BLOCK) * BLOCK


def _ranges(c):
    """int32 (B or 1) x Lq x 2: the keys [begin, end) each query may see, or None."""
    if c["docs"]:
        # documents of unequal lengths over the first 31/32 of the sequence, then padding
        L, n = c["Lk"], c["docs"]
        used = L - L // 32
        ends = [used * (i + 1) * (i + 2) // (n * (n + 1)) for i in range(n)]
        r = np.zeros((1, L, 2), np.int32)
        for b, e in zip([0] + ends, ends):
            r[0, b:e] = (b, e)
        return r
    if c["lens"]:
        # caches filled from half to the whole of their length
        r = np.zeros((c["B"], c["Lq"], 2), np.int32)
        for b in range(c["B"]):
            r[b, :, 1] = c["Lk"] - (c["Lk"] // 2) * b // c["B"]
        return r
    return None


def _seen(c):
    """Pairs (query, key) that the masks leave, over the batch, for one head."""
    r = _ranges(c)
    lo, hi = (np.zeros((1, c["Lq"]), np.int64), np.full((1, c["Lq"]), c["Lk"], np.int64)) if r is None else (
        r[..., 0].astype(np.int64), r[..., 1].astype(np.int64))
    if c["causal"]:
        pos = np.arange(c["Lq"], dtype=np.int64)[None] + c["Lk"] - c["Lq"]
        hi = np.minimum(hi, np.maximum(pos + 1, c["prefix"]))
    n = int(np.maximum(hi - lo, 0).sum())
    return n * (c["B"] if lo.shape[0] == 1 else 1)


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "norm":
        t = DTYPES[c["dtype"]]
        M, K, G = c["M"], c["K"], _pad(c["K"]) // BLOCK
        return dict(
            op="norm", X=_activation(g, M, K).to(t),
            residual=torch.randn(M, K, generator=g, device=DEV).mul_(4.0).to(t) if c["residual"] else None,
            gain=1.0 + 0.2 * torch.randn(K, generator=g, device=DEV), eps=1e-6,
            codes=torch.empty(M, _pad(K), device=DEV, dtype=torch.float8_e4m3fn),
            scales=torch.empty(M, G, device=DEV), out=torch.empty(M, K, device=DEV, dtype=t) if c["residual"] else None)
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        Kp = _pad(K)
        x = torch.zeros(M, Kp, device=DEV)
        x[:, :K] = _activation(g, M, K)
        xg = x.view(M, Kp // BLOCK, BLOCK)
        sa = (xg.abs().amax(2) / E4M3_MAX).clamp_min(TINY)
        a = (xg / sa[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(M, Kp)
        Np = _pad(N)
        w = torch.zeros(Np, Kp, device=DEV)
        w[:N, :K] = 0.02 * torch.randn(N, K, generator=g, device=DEV)
        w[:, torch.randperm(K, generator=g, device=DEV)[:max(1, K // 100)]] *= 10.0
        wg = w.view(Np // BLOCK, BLOCK, Kp // BLOCK, BLOCK)
        sw = (wg.abs().amax((1, 3)) / E4M3_MAX).clamp_min(TINY)
        q = (wg / sw[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s = dict(op="gemm", a=a, sa=sa, w=q.view(Np, Kp)[:N].contiguous(), sw=sw,
                 bias=0.1 * torch.randn(N, generator=g, device=DEV) if c["bias"] else None,
                 act="gelu_tanh" if c["act"] else None, Y=torch.empty(M, N, device=DEV, dtype=DTYPES[c["out"]]), ws=None)
        if own:
            import bit_post_quantized_smooth_amd as sq
            s["ws"] = torch.empty(sq.gemm_fp8_workspace_bytes(M, N, Kp), device=DEV, dtype=torch.uint8)
        return s
    B, Lq, Lk, Hq, Hkv, D = (c[k] for k in ("B", "Lq", "Lk", "Hq", "Hkv", "D"))
    t = DTYPES[c["dtype"]]
    if c["fused"]:   # slices of the QKV projection's output
        x = torch.randn(B, Lk, (Hq + 2 * Hkv) * D, generator=g, device=DEV).to(t)
        q, k, v = x.split([Hq * D, Hkv * D, Hkv * D], dim=2)
        q, k, v = q.unflatten(2, (Hq, D)), k.unflatten(2, (Hkv, D)), v.unflatten(2, (Hkv, D))
    else:
        q = torch.randn(B, Lq, Hq, D, generator=g, device=DEV).to(t)
        k = torch.randn(B, Lk, Hkv, D, generator=g, device=DEV).to(t)
        v = torch.randn(B, Lk, Hkv, D, generator=g, device=DEV).to(t)
    r = _ranges(c)
    s = dict(op="attn", q=q, k=k, v=v, scale=D ** -0.5, cap=c["cap"], causal=c["causal"],
             slopes=torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=DEV) / Hq) if c["slopes"] else None,
             prefix=torch.full((B,), c["prefix"], device=DEV, dtype=torch.int32) if c["prefix"] else None,
             ranges=None if r is None else torch.from_numpy(r).to(DEV),
             out=torch.empty(B, Lq, Hq, D, device=DEV, dtype=t), ws=None)
    if own:
        import bit_post_quantized_smooth_amd as sq
        s["ws"] = torch.empty(sq.attention_workspace_bytes(B, Lq, Lk, Hq, Hkv, D), device=DEV, dtype=torch.uint8)
    return s


# ---------------------------------------------------------------------------- one pass

def run(state):
    return _library(state) if own else _plain(state)


def _library(s):
    import bit_post_quantized_smooth_amd as sq
    if s["op"] == "norm":
        sq.rmsnorm_quantize_fp8(s["X"], s["residual"], s["gain"], s["eps"], s["codes"], s["scales"], s["out"])
        return dict(codes=s["codes"], scales=s["scales"], residual=s["out"])
    if s["op"] == "gemm":
        sq.gemm_fp8(s["a"], s["sa"], s["w"], s["sw"], s["bias"], s["Y"], ws=s["ws"], activation=s["act"])
        return s["Y"]
    sq.attention(s["q"], s["k"], s["v"], s["out"], scale=s["scale"], softcap=s["cap"], slopes=s["slopes"],
                 causal=s["causal"], prefix=s["prefix"], key_ranges=s["ranges"], ws=s["ws"])
    return s["out"]


def _plain(s):
    if s["op"] == "norm":
        X = s["X"]
        M, K = X.shape
        h = X.float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
        u = h * torch.rsqrt(h.square().mean(1, keepdim=True) + s["eps"]) * s["gain"]
        p = torch.nn.functional.pad(u, (0, _pad(K) - K)).view(M, -1, BLOCK)
        sc = (p.abs().amax(2) / E4M3_MAX).clamp_min(TINY)
        q = (p * (1.0 / sc)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return dict(codes=q.view(M, -1), scales=sc, residual=h.to(X.dtype) if s["residual"] is not None else None)
    if s["op"] == "gemm":
        a = s["a"].float() * s["sa"].repeat_interleave(BLOCK, 1)
        N = s["w"].shape[0]
        w = s["w"].float() * s["sw"].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)
        y = a @ w.t()
        if s["bias"] is not None:
            y = y + s["bias"]
        if s["act"]:
            y = y * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y))
        return y.to(s["Y"].dtype)
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    B, Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[1:3]
    q = q.view(B, Lq, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = (q @ k.permute(0, 2, 3, 1)).view(B, Hq, Lq, Lk) * s["scale"]
    if s["cap"]:
        x = s["cap"] * torch.tanh(x / s["cap"])
    pos = torch.arange(Lq, device=x.device)[:, None] + Lk - Lq
    j = torch.arange(Lk, device=x.device)[None, :]
    if s["slopes"] is not None:
        x = x - s["slopes"][:, None, None] * (pos - j).abs()
    see = torch.ones(1, Lq, Lk, dtype=torch.bool, device=x.device)
    if s["ranges"] is not None:
        see = see & (j >= s["ranges"][..., :1]) & (j < s["ranges"][..., 1:])
    if s["causal"]:
        first = j <= pos
        see = see & (first if s["prefix"] is None else first | (j < s["prefix"][:, None, None]))
    x = x.masked_fill(~see[:, None], -math.inf)
    top = x.amax(3, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    n = p.sum(3, keepdim=True)
    p = p / torch.where(n == 0, 1.0, n)
    o = p.view(B, Hkv, -1, Lk) @ v.permute(0, 2, 1, 3)
    return o.view(B, Hq, Lq, D).transpose(1, 2).contiguous().to(s["out"].dtype)


# ---------------------------------------------------------------------------- costs and exact values

def work(case):
    c = case
    if c["op"] == "norm":
        M, K, Kp, e = c["M"], c["K"], _pad(c["K"]), ESIZE[c["dtype"]]
        return dict(bytes=M * K * e * (3 if c["residual"] else 1) + M * Kp + 4 * M * Kp // BLOCK + 4 * K, flops=10 * M * K)
    if c["op"] == "gemm":
        M, N, Kp = c["M"], c["N"], _pad(c["K"])
        scales = 4 * (M + _pad(N) // BLOCK) * Kp // BLOCK
        return dict(bytes=(M + N) * Kp + scales + M * N * ESIZE[c["out"]] + (4 * N if c["bias"] else 0), flops=2 * M * N * Kp)
    B, Lq, Hq, Hkv, D = (c[k] for k in ("B", "Lq", "Hq", "Hkv", "D"))
    r = _ranges(c)
    keys = B * c["Lk"] if not c["lens"] else int(r[:, 0, 1].sum())
    return dict(bytes=2 * D * (2 * B * Lq * Hq + 2 * keys * Hkv), flops=4 * D * Hq * _seen(c))


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if s["op"] == "norm":
        M, K = s["X"].shape
        h = s["X"].to(f64)
        if s["residual"] is not None:
            h = h + s["residual"].to(f64)
        rms = (torch.linalg.vector_norm(h, dim=1) ** 2 / K + s["eps"]).sqrt()
        u = h / rms[:, None] * s["gain"].to(f64)
        G = _pad(K) // BLOCK
        codes = torch.zeros(M, G * BLOCK, dtype=f64, device=h.device)
        scales = torch.zeros(M, G, dtype=f64, device=h.device)
        for i in range(G):
            blk = u[:, i * BLOCK:(i + 1) * BLOCK]
            scales[:, i] = torch.clamp(blk.abs().max(dim=1).values / E4M3_MAX, min=TINY)
            codes[:, i * BLOCK:i * BLOCK + blk.shape[1]] = blk / scales[:, i:i + 1]
        return dict(codes=codes, scales=scales, residual=h if s["residual"] is not None else None)
    if s["op"] == "gemm":
        N, Kp = s["w"].shape
        y = torch.zeros(s["a"].shape[0], N, dtype=f64, device=s["w"].device)
        col = torch.arange(N, device=y.device) // BLOCK
        for i in range(Kp // BLOCK):
            b = slice(i * BLOCK, (i + 1) * BLOCK)
            part = torch.mm(s["a"][:, b].to(f64), s["w"][:, b].to(f64).t().contiguous())
            y += part * s["sa"][:, i].to(f64)[:, None] * s["sw"][:, i].to(f64)[col][None, :]
        if s["bias"] is not None:
            y += s["bias"].to(f64)
        if s["act"]:
            y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3)))
        return y
    c = case
    out = torch.zeros(s["out"].shape, dtype=f64, device=s["out"].device)
    pos = torch.arange(c["Lq"], device=out.device, dtype=f64) + (c["Lk"] - c["Lq"])
    key = torch.arange(c["Lk"], device=out.device, dtype=f64)
    for b in range(c["B"]):
        hide = torch.zeros(c["Lq"], c["Lk"], dtype=torch.bool, device=out.device)
        if s["ranges"] is not None:
            lim = s["ranges"][min(b, s["ranges"].shape[0] - 1)].to(f64)
            hide |= (key[None] < lim[:, :1]) | (key[None] >= lim[:, 1:])
        if c["causal"]:
            hide |= (key[None] > pos[:, None]) & (key[None] >= c["prefix"])
        for h in range(c["Hq"]):
            kv = h // (c["Hq"] // c["Hkv"])
            x = torch.mm(s["q"][b, :, h].to(f64), s["k"][b, :, kv].to(f64).t().contiguous()) / math.sqrt(c["D"])
            if c["cap"]:
                x = torch.tanh(x / c["cap"]) * c["cap"]
            if s["slopes"] is not None:
                x = x - float(s["slopes"][h]) * torch.abs(pos[:, None] - key[None])
            x[hide] = -math.inf
            z = torch.logsumexp(x, dim=1, keepdim=True)
            w = torch.where(hide, 0.0, torch.exp(x - z))
            out[b, :, h] = torch.mm(w, s["v"][b, :, kv].to(f64).contiguous())
    return out
