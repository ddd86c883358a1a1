"""Plain fp64 implementations of the 8-bit attention block's operators and the
error bounds their tests hold the kernels to. CPU only; nothing here uses the
library."""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -126
F64 = torch.float64


def padded(K: int) -> int:
    return -(-K // BLOCK) * BLOCK


def e4m3_values() -> np.ndarray:
    """The value of every e4m3 code (NaN for 0x7F and 0xFF)."""
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = math.ldexp(8 + f, e - 10) if e else math.ldexp(f, -9)
        v[c] = math.nan if e == 15 and f == 7 else x
        if c & 128:
            v[c] = -v[c]
    return v


def decode(codes) -> torch.Tensor:
    """fp64 values of e4m3 codes (uint8 or float8 tensor, on the CPU)."""
    b = codes.cpu().contiguous().view(torch.uint8).numpy()
    return torch.from_numpy(e4m3_values()[b])


def nearest_distance(v: torch.Tensor) -> torch.Tensor:
    """Distance from each value to the nearest finite e4m3 value."""
    t = e4m3_values()
    t = torch.from_numpy(np.unique(t[np.isfinite(t)]))
    i = torch.searchsorted(t, v.contiguous()).clamp(1, len(t) - 1)
    return torch.minimum((v - t[i - 1]).abs(), (v - t[i]).abs())


def norm(X, residual, gain, eps):
    """(h, u) in fp64."""
    h = X.to(F64)
    if residual is not None:
        h = h + residual.to(F64)
    u = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h, u if gain is None else u * gain.to(F64)


def check_quantized(codes, scales, u, rel):
    """Codes (M x Kp) and scales (M x G) against the fp64 values u (M x K), whose
    fp32 computation is good to `rel`: the scale to that and two roundings, each
    code a nearest one of u / s up to the same error (an exact tie or a value
    within the error of one may go either way), zeros past K."""
    M, K = u.shape
    Kp = padded(K)
    assert tuple(codes.shape) == (M, Kp) and tuple(scales.shape) == (M, Kp // BLOCK)
    up = torch.zeros(M, Kp, dtype=F64)
    up[:, :K] = u
    g = up.view(M, -1, BLOCK)
    s = (g.abs().amax(2) / E4M3_MAX).clamp_min(TINY)
    got = scales.cpu().to(F64)
    assert bool(((got - s).abs() <= (rel + 2.0 ** -23) * s).all()), float(((got - s).abs() / s).max())
    q = decode(codes).view(M, -1, BLOCK)
    v = g / s[:, :, None]
    err = (q - v).abs() - nearest_distance(v)
    assert bool((err <= (4 * rel + 2.0 ** -21) * v.abs()).all()), float(err.max())
    assert bool((q.reshape(M, Kp)[:, K:] == 0).all())


def gemm(a, sa, w, sw, bias, gelu):
    """(y, envelope, peak) in fp64 from codes and scales: envelope = sum of the
    absolute terms, peak = per group the largest |a w| term, summed over groups."""
    M, Kp = a.shape
    N = w.shape[0]
    A, W = decode(a), decode(w)
    sa, sw = sa.cpu().to(F64), sw.cpu().to(F64)
    col = torch.arange(N) // BLOCK
    y = torch.zeros(M, N, dtype=F64)
    env = torch.zeros(M, N, dtype=F64)
    peak = torch.zeros(M, N, dtype=F64)
    for g in range(Kp // BLOCK):
        b = slice(g * BLOCK, (g + 1) * BLOCK)
        s = sa[:, g, None] * sw[col, g][None]
        y += (A[:, b] @ W[:, b].t().contiguous()) * s
        env += (A[:, b].abs() @ W[:, b].abs().t().contiguous()) * s
        peak += A[:, b].abs().amax(1)[:, None] * W[:, b].abs().amax(1)[None] * s
    if bias is not None:
        y = y + bias.cpu().to(F64)
        env = env + bias.cpu().to(F64).abs()
    if gelu:
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    return y, env, peak


def gemm_bound(y, env, peak, Kp, dtype):
    """Error a correct kernel stays below. fp32: 128 + 2 G roundings of partial sums,
    each at most 2^-24 of the envelope. 16 bits: besides, what the 8-bit matrix
    instruction loses by aligning a group's products to their largest, at most
    2^-13 of it in a probe of 60000 sums (2^-11 allowed here), and the rounding of
    the output. GELU's slope is at most 1.13."""
    G = Kp // BLOCK
    t = 1.2 * (128 + 2 * G) * 2.0 ** -24 * env + 2.0 ** -22 * y.abs()
    if dtype == torch.float32:
        return t + 2.0 ** -126
    ulp = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    return t + 1.2 * 2.0 ** -11 * peak + ulp * y.abs() + (2.0 ** -25 if dtype == torch.float16 else 0)


def attention(Q, K, V, scale, softcap=0.0, slopes=None, causal=False, prefix=None, ranges=None):
    """(out, bound) in fp64, (B, Lq, Hq, D). bound: the error a correct kernel stays
    below, from its roundings: P to 16 bits (relative eps, or the step 2^-25 of a
    subnormal fp16), the output to 16 bits, and a logit error dx that moves a
    softmax average by at most 2 dx times the average of |v|."""
    B, Lq, Hq, D = Q.shape
    Lk, Hkv = K.shape[1:3]
    eps = 2.0 ** -11 if Q.dtype == torch.float16 else 2.0 ** -8
    q, k, v = (t.cpu().to(F64) for t in (Q, K, V))
    out = torch.zeros(B, Lq, Hq, D, dtype=F64)
    bound = torch.zeros(B, Lq, Hq, D, dtype=F64)
    pos = torch.arange(Lq) + Lk - Lq
    key = torch.arange(Lk)
    for b in range(B):
        see = torch.ones(Lq, Lk, dtype=torch.bool)
        if ranges is not None:
            r = ranges.cpu()[min(b, ranges.shape[0] - 1)]
            see &= (key[None] >= r[:, :1]) & (key[None] < r[:, 1:])
        if causal:
            c = key[None] <= pos[:, None]
            if prefix is not None:
                c = c | (key[None] < int(prefix[b]))
            see &= c
        for h in range(Hq):
            kk, vv = k[b, :, h // (Hq // Hkv)], v[b, :, h // (Hq // Hkv)]
            x = (q[b, :, h] @ kk.t().contiguous()) * scale
            dx = (D + 4) * 2.0 ** -24 * abs(scale) * (
                q[b, :, h].nan_to_num(0, 0, 0).norm(dim=1, keepdim=True)
                * (kk.nan_to_num(0, 0, 0).norm(dim=1).max() if Lk else 0.0))
            if softcap:
                x = softcap * torch.tanh(x / softcap)
                dx = dx + 8 * softcap * 2.0 ** -24
            if slopes is not None:
                s = float(slopes[h])
                x = x - s * (pos[:, None] - key[None]).abs()
                dx = dx + 4 * s * (Lk + Lq) * 2.0 ** -24
            x = torch.where(see, x, -math.inf)
            top = x.max(1, keepdim=True).values if Lk else torch.full((Lq, 1), -math.inf, dtype=F64)
            dx = dx + 4 * 2.0 ** -24 * (2 + top.abs().nan_to_num(0, 0, 0))
            e = torch.where(see, torch.exp(x - torch.where(top == -math.inf, 0.0, top)), 0.0)
            n = e.sum(1, keepdim=True)
            n = torch.where(n == 0, 1.0, n)
            # a hidden key takes no part, whatever its v holds
            bad = ~torch.isfinite(vv)
            fin = torch.where(bad, 0.0, vv)
            o = (e @ fin) / n
            if bool(bad.any()):
                for j in torch.nonzero(bad.any(1)).flatten().tolist():
                    hit = see[:, j, None] & bad[j][None]
                    o = torch.where(hit, o + vv[j][None], o)
            a = (e @ fin.abs()) / n
            out[b, :, h] = o
            sub = 2.0 ** -25 if Q.dtype == torch.float16 else 0.0
            tail = see.sum(1, keepdim=True) * sub * (fin.abs().max() if Lk else 0.0) / n
            bound[b, :, h] = eps * (a + o.abs().nan_to_num(0, 0, 0)) + (2 * dx + 2.0 ** -20) * a + tail + sub
    return out, bound


def assert_within(got, ref, bound):
    got = got.cpu().to(F64)
    fine = torch.isfinite(ref)
    assert torch.equal(fine, torch.isfinite(got)), "finite values differ"
    assert torch.equal(torch.isnan(ref), torch.isnan(got)), "NaN differ"
    assert bool((got[~fine & ~torch.isnan(ref)] == ref[~fine & ~torch.isnan(ref)]).all())
    ratio = ((got - ref).abs() / bound.clamp_min(1e-300))[fine]
    if ratio.numel():
        assert float(ratio.max()) <= 1.0, (int((ratio > 1).sum()), float(ratio.max()))
