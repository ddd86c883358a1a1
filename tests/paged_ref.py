"""Plain fp64 implementations of the paged cache's operators, the error bounds their tests
hold the kernels to, and pools to run them on. CPU only; nothing here uses the library."""
from __future__ import annotations

import math

import torch

import block_ref as R

F64 = R.F64
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E4M3 = torch.float8_e4m3fn
VALUES = torch.from_numpy(R.e4m3_values())


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the step of a subnormal number of 16 bits (0 where fp64 does not see it)."""
    return 2.0 ** -25 if dtype == F16 else 2.0 ** -134


def heads(x, positions=None, freqs=None, factor=1.0, interleaved=False, gain=None, eps=None):
    """(out, error) in fp64 of x (T x H x D): the definition, and what an fp32 computation of it
    may be off by before its rounding to 16 bits.

    The norm: 8 squares in a chain and 4 additions across lanes are 12 roundings of positive
    terms, halved by the root; division by D, the root and the reciprocal 3 more, the two products
    2 more: 12 of 2^-24, 16 allowed. A cosine: 2^-22 (its polynomial and factor 4 roundings
    of values up to 1). The rotation: 3 roundings of |a c| + |b s|."""
    u = x.cpu().to(F64)
    rel = 0.0
    if eps is not None:
        u = u / torch.sqrt((u * u).mean(2, keepdim=True) + eps)
        u = u if gain is None else u * gain.cpu().to(F64)
        rel = 16 * 2.0 ** -24
    out, err = u.clone(), rel * u.abs()
    if freqs is not None:
        n = freqs.numel()
        ang = positions.cpu().to(F64)[:, None, None] * freqs.cpu().to(F64)
        c, s = factor * torch.cos(ang), factor * torch.sin(ang)
        a = (slice(0, 2 * n, 2) if interleaved else slice(0, n))
        b = (slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n))
        out[..., a] = u[..., a] * c - u[..., b] * s
        out[..., b] = u[..., a] * s + u[..., b] * c
        both = u[..., a].abs() + u[..., b].abs()
        err[..., a] = err[..., b] = abs(factor) * both * (rel + 2.0 ** -22 + 3 * 2.0 ** -24)
    return out, err


def assert_rounded(got, ref, err, dtype):
    """got: ref, computed to err, rounded once to dtype. Values that dtype does not reach may come
    out as the infinity."""
    got = got.cpu().to(F64)
    fine = torch.isfinite(ref)
    most = torch.finfo(dtype).max
    assert torch.equal(torch.isnan(ref), torch.isnan(got)), "NaN differ"
    over = ref.abs() * (1 + half_step(dtype)) + err >= most
    bound = err + half_step(dtype) * (ref.abs() + err) + tiny(dtype)
    ok = ((got - ref).abs() <= bound) | over | ~fine
    assert bool(ok.all()), (int((~ok).sum()), float(((got - ref).abs() / bound)[~ok].max()))


def assert_codes(codes, ref, err, scale):
    """codes: e4m3_rne(clamp(ref / scale)) of a ref computed to err, times the rounded reciprocal
    of the scale (2 roundings)."""
    got = R.decode(codes)
    v = ref / scale
    d = err / scale + 2.0 ** -22 * v.abs()
    bad = ~torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), bad)
    v = v.clamp(-R.E4M3_MAX, R.E4M3_MAX)
    off = (got - v).abs() - R.nearest_distance(v)
    # a value off by d takes a code that is up to 2 d further away
    ok = (off <= 2 * d + 2.0 ** -40) | bad
    assert bool(ok.all()), float((off - 2 * d)[~ok].max())


class Pool:
    """A pool with tables of B sequences of the given lengths in scattered pages, -1 behind their
    ends, `spare` pages over, random values everywhere (NaN codes and infinities among what no
    sequence owns)."""

    def __init__(self, lengths, Hkv, D, dtype, coded, page=16, spare=2, seed=0, width=None, scales=True):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lengths]
        total = sum(need) + spare
        self.page, self.dtype, self.coded, self.lengths_list = page, dtype, coded, list(lengths)
        order = torch.randperm(total, generator=g).tolist()
        self.width = max([1, *need]) if width is None else width
        self.tables = torch.full((len(lengths), self.width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.k, self.v = (torch.randn(total, Hkv, page, D, generator=g) for _ in range(2))
        self.ks = self.vs = None
        if coded:
            if scales:
                self.ks, self.vs = (0.01 * (1 + torch.rand(Hkv, generator=g)) for _ in range(2))
            one = torch.ones(Hkv)
            self.k, self.v = ((x / (one if s is None else s).view(-1, 1, 1)).clamp(-448, 448).to(E4M3)
                              for x, s in ((self.k, self.ks), (self.v, self.vs)))
        else:
            self.k, self.v = self.k.to(dtype), self.v.to(dtype)
        self.lengths = torch.tensor(lengths, dtype=torch.int32)

    def cuda(self):
        for name in ("k", "v", "ks", "vs", "tables", "lengths"):
            t = getattr(self, name)
            if t is not None:
                setattr(self, name, t.cuda())
        return self

    @staticmethod
    def poison(t):
        """All of t's elements not a number."""
        if t.element_size() == 1:
            t.view(torch.uint8).fill_(0x7F)
        else:
            t.fill_(float("nan"))

    def poison_free(self):
        """NaN in every page no table names and in every row behind its sequence's end."""
        used = set(self.tables.flatten().tolist())
        for x in (self.k, self.v):
            for p in range(x.shape[0]):
                if p not in used:
                    self.poison(x[p])
            for b, n in enumerate(self.lengths_list):
                for i in range(self.width):
                    p = int(self.tables[b, i])
                    first = n - i * self.page
                    if p >= 0 and first < self.page:
                        self.poison(x[p, :, max(first, 0):])
        return self

    def dense(self, b, n=None):
        """(k, v, there): the first n tokens of sequence b, n x Hkv x D in fp64, and whether each
        lies in a page of the pool."""
        n = self.lengths_list[b] if n is None else n
        n = max(0, min(n, self.width * self.page))
        out = []
        ids = self.tables[b].cpu()[torch.arange(n) // self.page].long()
        there = (ids >= 0) & (ids < self.k.shape[0])
        ids = torch.where(there, ids, 0)
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            if x.shape[0] == 0:
                out.append(torch.zeros(n, x.shape[1], x.shape[3], dtype=F64))
                continue
            # the sequence's pages first: pools are large
            used, where = torch.unique(ids, return_inverse=True)
            x = (x.view(torch.uint8) if self.coded else x)[used.to(x.device)]
            x = VALUES[x.cpu().long()] if self.coded else x.cpu().to(F64)
            if s is not None:
                x = x * s.cpu().to(F64).view(-1, 1, 1)
            out.append(x[where, :, torch.arange(n) % self.page])
        return (*out, there)


def attention(Q, pool, starts, lengths, scale, softcap=0.0, slopes=None, causal=True):
    """(out, bound, owned) in fp64, (T, Hq, D). bound as in block_ref.attention: weights rounded
    to 16 bits, the output's rounding and a logit error dx that moves an average by up to 2 dx of
    the average |v|. owned: rows of a sequence."""
    T, Hq, D = Q.shape
    half = half_step(Q.dtype)
    q = Q.cpu().to(F64)
    out = torch.zeros(T, Hq, D, dtype=F64)
    bound = torch.zeros(T, Hq, D, dtype=F64)
    owned = torch.zeros(T, dtype=torch.bool)
    for b in range(len(starts) - 1):
        at, n = starts[b], starts[b + 1] - starts[b]
        owned[at:at + n] = True
        k, v, there = pool.dense(b, lengths[b])
        held = k.shape[0]
        pos = torch.arange(n)[:, None] + held - n
        key = torch.arange(held)[None]
        see = there[None] & (key <= pos) if causal else there[None].expand(n, held)
        G = Hq // k.shape[1]
        for h in range(Hq):
            kk, vv = k[:, h // G], v[:, h // G]
            kf = kk.nan_to_num(0, 0, 0)
            x = (q[at:at + n, h] @ kk.t().contiguous()) * scale
            dx = (D + 4) * 2.0 ** -24 * abs(scale) * (
                q[at:at + n, h].nan_to_num(0, 0, 0).norm(dim=1, keepdim=True) * (kf.norm(dim=1).max() if held else 0.0))
            if softcap:
                x = softcap * torch.tanh(x / softcap)
                dx = dx + 8 * softcap * 2.0 ** -24
            if slopes is not None:
                s = float(slopes[h])
                x = x - s * (pos - key).abs()
                dx = dx + 4 * s * (held + n) * 2.0 ** -24
            x = torch.where(see, x, -math.inf)
            top = x.max(1, keepdim=True).values if held else torch.full((n, 1), -math.inf, dtype=F64)
            dx = dx + 4 * 2.0 ** -24 * (2 + top.abs().nan_to_num(0, 0, 0))
            e = torch.where(see, torch.exp(x - torch.where(top == -math.inf, 0.0, top)), 0.0)
            z = e.sum(1, keepdim=True)
            z = torch.where(z == 0, 1.0, z)
            bad = ~torch.isfinite(vv)
            fin = torch.where(bad, 0.0, vv)
            o = (e @ fin) / z
            for j in torch.nonzero(bad.any(1)).flatten().tolist():
                o = torch.where(see[:, j, None] & bad[j][None], o + vv[j][None], o)
            a = (e @ fin.abs()) / z
            out[at:at + n, h] = o
            sub = tiny(Q.dtype)
            tail = see.sum(1, keepdim=True) * sub * (fin.abs().max() if held else 0.0) / z
            bound[at:at + n, h] = half * (a + o.abs().nan_to_num(0, 0, 0)) + (2 * dx + 2.0 ** -20) * a + tail + sub
    return out, bound, owned
