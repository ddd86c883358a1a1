"""A pre-norm attention block with 8-bit linears: the operators in the order a
transformer runs them.

    h = X + residual
    a = quantize(rms_norm(h) * gain)             rmsnorm_quantize_fp8
    q, k, v = a Wqkv^T + b                       gemm_fp8
    o = attention(q, keys, values)               attention
    Y = quantize(o) Wout^T + b                   quantize_act_fp8, gemm_fp8

Five launches (more where a product or the attention is split, and two copies where
there is a cache). The normalized activation exists only as codes and scales, the
residual addition costs no pass of its own, and q, k and v are read in place as strided
views of one product. What a model does to q and k in between (rotary embedding, norms)
has no place here: such a model calls the operators one by one.
"""
from __future__ import annotations

import math

import numpy as np

from . import api


class KeyValueCache:
    """Keys and values of up to ``capacity`` tokens for each of ``batch``
    sequences; ``length`` tokens are held. The length is a number of the host's: a graph
    captured from a call with the cache writes, in every replay, to the slots of its
    capture and sees as many keys as it did then. A graph for each length, or eager
    calls, generate token after token."""

    def __init__(self, batch: int, capacity: int, kv_heads: int, head_dim: int, dtype, device="cuda"):
        torch = api._torch()
        shape = (batch, capacity, kv_heads, head_dim)
        self.k = torch.empty(shape, dtype=dtype, device=device)
        self.v = torch.empty(shape, dtype=dtype, device=device)
        self.capacity = capacity
        self.length = 0

    def _refuse(self, k, v):
        """Raises for the first of k and v that the cache does not take."""
        for name, t in (("k", k), ("v", v)):
            if not isinstance(t, api._torch().Tensor):
                raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
            want = (self.k.shape[0], k.shape[1] if k.dim() == 4 else None, *self.k.shape[2:])
            if tuple(t.shape) != want:
                raise ValueError(f"{name}: shape {tuple(t.shape)}, the cache takes {want}")
            if t.dtype != self.k.dtype or t.device != self.k.device:
                raise ValueError(f"{name}: {t.dtype} on {t.device}, the cache holds {self.k.dtype} "
                                 f"on {self.k.device}")

    def append(self, k, v):
        """Take in k and v (batch x tokens x kv_heads x head_dim, the cache's type); the
        views of all tokens held. What does not fit is refused before anything changes."""
        held = self.k
        try:
            b, n, h, d = k.shape
            good = ((b, self.capacity, h, d) == held.shape and v.shape == k.shape
                    and k.dtype is held.dtype and v.dtype is held.dtype
                    and k.device == held.device and v.device == held.device)
        except (AttributeError, TypeError, ValueError):
            good = False
        if not good:
            self._refuse(k, v)
        end = self.length + n
        if end > self.capacity:
            raise ValueError(f"cache of {self.capacity} tokens: {end} needed")
        self.k[:, self.length:end].copy_(k)
        self.v[:, self.length:end].copy_(v)
        self.length = end
        return self.k[:, :end], self.v[:, :end]


class AttentionBlock:
    """One block resident on a device.

    ``qkv`` and ``out`` are prepare_weights_fp8 of (K x (heads + 2 kv_heads)
    head_dim) and (heads head_dim x K) weights, ``gain`` the norm's K values.
    ``block(X, residual)`` takes batch x tokens x K and returns (Y, h): the
    block's output and X + residual, which are the next block's X and residual.
    With a KeyValueCache the tokens are appended to it and attend to all that it
    holds; a call that raises leaves the cache's length as it was. Buffers are kept between calls and grown when more tokens arrive, so
    one block serves one stream at a time (the smaller ones stay, for graphs captured
    with them), and Y and h are new tensors."""

    def __init__(self, gain, qkv, out, heads: int, kv_heads: int, head_dim: int,
                 qkv_bias=None, out_bias=None, eps: float = 1e-6, softcap: float = 0.0,
                 slopes=None, device="cuda"):
        torch = api._torch()
        self.K = qkv.K
        if qkv.fmt != "fp8" or out.fmt != "fp8":
            raise ValueError("qkv and out must come from prepare_weights_fp8")
        if qkv.rank or out.rank:
            raise ValueError("8-bit layers have no low-rank branch: qkv's or out's would not be "
                             "applied")
        if qkv.N != (heads + 2 * kv_heads) * head_dim or out.K != heads * head_dim or out.N != qkv.K:
            raise ValueError(f"qkv is {qkv.K} x {qkv.N} and out {out.K} x {out.N}: they do not fit "
                             f"{heads} + 2 x {kv_heads} heads of {head_dim}")
        if (min(heads, kv_heads, head_dim) < 1 or heads % kv_heads or head_dim % 8
                or head_dim > 128):
            raise ValueError(f"{heads} heads over {kv_heads} of {head_dim}: attention takes whole "
                             "groups of heads, each a multiple of 8 up to 128")
        for name, x, n in (("gain", gain, qkv.K), ("qkv_bias", qkv_bias, qkv.N),
                           ("out_bias", out_bias, out.N), ("slopes", slopes, heads)):
            if x is not None and math.prod(np.shape(x)) != n:
                raise ValueError(f"{name}: shape {tuple(np.shape(x))}, expected {n} values")
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.eps, self.softcap = float(eps), float(softcap)
        dev = self.device = torch.device(device)

        def put(x):
            return None if x is None else torch.from_numpy(api._c(x, np.float32)).to(dev)

        self.gain, self.slopes = put(gain), put(slopes)
        self.qkv = (torch.from_numpy(qkv.w_codes).to(dev), put(qkv.w_scales), put(qkv_bias))
        self.out = (torch.from_numpy(out.w_codes).to(dev), put(out.w_scales), put(out_bias))
        self._buffers = api._Buffers(dev)
        self._kept = self._buffers.kept

    def _buffer(self, name, shape, dtype):
        """The buffer kept under `name`, as a tensor of this shape."""
        count = math.prod(shape)
        t = self._kept.get((name, dtype))
        if t is None or t.numel() < count:
            t = self._buffers.larger(name, count, dtype)
        return t[:count].view(shape)

    def _codes(self, name, M, K):
        torch = api._torch()
        Kp = api.fp8_padded(K)
        return (self._buffer(name, (M, Kp), torch.uint8),
                self._buffer(name, (M, Kp // api.FP8_BLOCK), torch.float32))

    def _product(self, codes, scales, weights, Y):
        M, N = Y.shape
        need = api.gemm_fp8_workspace_bytes(M, N, codes.shape[1])
        ws = self._buffer("split", (need,), api._torch().uint8) if need else None
        api.gemm_fp8(codes, scales, *weights, Y, ws=ws)

    def __call__(self, X, residual=None, cache=None, causal: bool = True, prefix=None,
                 key_ranges=None):
        """(Y, h) of X (batch x tokens x K, fp16 or bf16), on the current stream. Masks
        as in attention(): ``causal``, ``prefix`` tokens per sequence that all see,
        ``key_ranges``."""
        torch = api._torch()
        if not isinstance(X, torch.Tensor):
            raise TypeError(f"X: expected a torch tensor, got {type(X).__name__}")
        if X.dtype not in (torch.float16, torch.bfloat16):
            raise ValueError(f"X: dtype {X.dtype}, expected float16 or bfloat16")
        if X.dim() != 3 or X.shape[2] != self.K:
            raise ValueError(f"X: shape {tuple(X.shape)}, expected (batch, tokens, {self.K})")
        if residual is not None and residual.shape != X.shape:
            raise ValueError(f"residual: shape {tuple(residual.shape)}, X has {tuple(X.shape)}")
        held = None if cache is None else cache.length
        try:
            return self._run(X, residual, cache, causal, prefix, key_ranges)
        except BaseException:
            if cache is not None:
                cache.length = held      # tokens behind it are not seen and written again
            raise

    def _run(self, X, residual, cache, causal, prefix, key_ranges):
        torch = api._torch()
        B, L, K = X.shape
        M, D, Hq, Hkv = B * L, self.head_dim, self.heads, self.kv_heads
        h = torch.empty_like(X, memory_format=torch.contiguous_format)
        Y = torch.empty_like(h)

        codes = self._codes("a", M, K)
        api.rmsnorm_quantize_fp8(X.reshape(M, K),
                                 None if residual is None else residual.reshape(M, K),
                                 self.gain, self.eps, *codes, h.view(M, K))
        t = self._buffer("qkv", (M, (Hq + 2 * Hkv) * D), X.dtype)
        self._product(*codes, self.qkv, t)
        t = t.view(B, L, Hq + 2 * Hkv, D)
        q, k, v = t[:, :, :Hq], t[:, :, Hq:Hq + Hkv], t[:, :, Hq + Hkv:]
        if cache is not None:
            k, v = cache.append(k, v)
        o = self._buffer("o", (B, L, Hq, D), X.dtype)
        need = api.attention_workspace_bytes(B, L, k.shape[1], Hq, Hkv, D)
        api.attention(q, k, v, o, softcap=self.softcap, slopes=self.slopes, causal=causal,
                      prefix=prefix, key_ranges=key_ranges,
                      ws=self._buffer("attention", (need,), torch.uint8) if need else None)
        codes = self._codes("c", M, Hq * D)
        api.quantize_act_fp8(o.view(M, Hq * D), *codes)
        self._product(*codes, self.out, Y.view(M, K))
        return Y, h
