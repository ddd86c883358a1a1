"""A pre-norm attention block with 8-bit linears: the operators in the order a
transformer runs them.

    h = X + residual
    a = quantize(rms_norm(h) * gain)             rmsnorm_quantize_fp8
    q, k, v = a Wqkv^T + b                       gemm_fp8
    q, k = rotate(norm(q)), rotate(norm(k))      norm_rotary (optional, in place)
    o = attention(q, keys, values)               attention
    Y = quantize(o) Wout^T + b                   quantize_act_fp8, gemm_fp8

Five launches, six with norms or rotation of the heads (more where a product or the
attention is split, and two copies where there is a KeyValueCache). The normalized
activation exists only as codes and scales, the residual addition costs no pass of its own,
and q, k and v are read in place as strided views of one product. With a
PagedKeyValueCache the pass over the heads writes keys and values into their pages
(norm_rotary_write) and the attention reads them there (paged_attention).
"""
from __future__ import annotations

import math

import numpy as np

from . import api, paged


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


class PageTable:
    """Where the tokens of up to ``batch`` sequences of up to ``capacity`` tokens lie: pages of
    ``page_size`` tokens out of ``pages`` (by default as many as all sequences at their
    longest need), handed out as sequences grow. One table serves the caches of all layers.

    ``begin(counts)`` before each step says how many tokens each sequence gets in it; the
    step's tokens, sequence after sequence, are then the rows of every layer's call. It
    writes tables, lengths, starts, slots and positions into tensors that stay where they are:
    a graph captured from a step of the layers is replayed for later steps, after
    ``begin``, with up to the tokens that it was captured with (rows behind the last
    sequence's belong to none). ``step_tokens``: most tokens of one step."""

    def __init__(self, batch: int, capacity: int, page_size: int = 64, pages: int | None = None,
                 step_tokens: int | None = None, device="cuda"):
        torch = api._torch()
        if batch < 1 or capacity < 1:
            raise ValueError(f"{batch} sequences of {capacity} tokens")
        if page_size < 16 or page_size > 1024 or page_size & (page_size - 1):
            raise ValueError(f"page_size: {page_size}, expected a power of two in 16 .. 1024")
        self.batch, self.capacity, self.page_size = batch, capacity, page_size
        self.width = -(-capacity // page_size)
        self.pages = batch * self.width if pages is None else pages
        self.step_tokens = batch * capacity if step_tokens is None else step_tokens
        if self.width * page_size > 2 ** 26:
            raise ValueError(f"capacity: {capacity}, attention takes up to 2^26 keys of a sequence")
        if self.pages < 0 or self.pages * page_size > 2 ** 31:
            raise ValueError(f"pages: {self.pages} of {page_size} tokens, expected up to 2^31 tokens")
        if self.step_tokens < 0:
            raise ValueError(f"step_tokens: {self.step_tokens}")
        self.tokens = 0                           # of the step that was begun last
        self.device = torch.device(device)
        sizes = [batch * self.width, batch, batch + 1, self.step_tokens, self.step_tokens]
        flat = torch.zeros(sum(sizes), dtype=torch.int32, device=device)
        self._flat, self._written = flat, 0
        tables, self.lengths, self.starts, self.slots, self.positions = flat.split(sizes)
        self.tables = tables.view(batch, self.width)
        tables.fill_(-1)
        self.slots.fill_(-1)
        self._tables = np.full((batch, self.width), -1, np.int32)
        self._lengths = np.zeros(batch, np.int64)
        self._free = list(range(self.pages - 1, -1, -1))

    def length(self, sequence: int) -> int:
        """Tokens of a sequence, those of the step that was begun among them."""
        return int(self._lengths[sequence])

    def release(self, sequence: int) -> None:
        """Ends a sequence: its pages are free again, its place in the batch is that of a new
        one. The tensors change with the next ``begin``."""
        row = self._tables[sequence]
        self._free.extend(int(p) for p in row[row >= 0][::-1])
        row[:] = -1
        self._lengths[sequence] = 0

    def begin(self, counts) -> None:
        """A step of counts[b] further tokens for sequence b (one number: for each). What
        does not fit is refused before anything changes. Copies on the current stream,
        without waiting for it."""
        torch = api._torch()
        n = np.asarray(counts)
        if n.dtype.kind not in "iu":
            raise TypeError("counts: expected integers")
        n = np.broadcast_to(n, (self.batch,)).astype(np.int64) if n.ndim == 0 else n.astype(np.int64)
        if n.shape != (self.batch,) or np.any(n < 0):
            raise ValueError(f"counts: expected {self.batch} numbers >= 0")
        if np.any(n > self.capacity):             # before sums that could wrap
            raise ValueError(f"sequences of up to {self.capacity} tokens: {int(n.max())} more needed")
        total, after = int(n.sum()), self._lengths + n
        if total > self.step_tokens:
            raise ValueError(f"{total} tokens in a step of up to {self.step_tokens}")
        if np.any(after > self.capacity):
            raise ValueError(f"sequences of up to {self.capacity} tokens: {int(after.max())} needed")
        size = self.page_size
        have, need = -(-self._lengths // size), -(-after // size)
        if int((need - have).sum()) > len(self._free):
            raise ValueError(f"{int((need - have).sum())} pages needed, {len(self._free)} are free")
        if self.device.type == "cuda" and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("begin: while a graph is captured; call it before each replay")
        # tables, lengths, starts and slots lie one behind the other: one copy, with -1 for
        # the slots that the step before used and this one does not
        used = max(total, self._written)
        fixed = self._tables.size + 2 * self.batch + 1
        host = torch.empty(fixed + used + total, dtype=torch.int32, pin_memory=self.device.type == "cuda")
        for b in np.nonzero(need > have)[0]:
            for i in range(have[b], need[b]):
                self._tables[b, i] = self._free.pop()
        starts = np.concatenate(([0], np.cumsum(n)))
        sequence = np.repeat(np.arange(self.batch), n)
        position = np.arange(total) - starts[sequence] + self._lengths[sequence]
        self._lengths = after
        self.tokens = total
        h = host.numpy()
        h[:self._tables.size] = self._tables.ravel()
        h[self._tables.size:fixed] = np.concatenate((after, starts))
        h[fixed:fixed + total] = self._tables[sequence, position // size] * size + position % size
        h[fixed + total:fixed + used] = -1
        h[fixed + used:] = position
        self._flat[:fixed + used].copy_(host[:fixed + used], non_blocking=True)
        self.positions[:total].copy_(host[fixed + used:], non_blocking=True)
        self._written = total


class PagedKeyValueCache:
    """One layer's keys and values in the pages of a PageTable, of the layer's 16-bit type or
    (``dtype`` torch.float8_e4m3fn) as e4m3 codes of one scale per head: ``k_scales``,
    ``v_scales``, fp32, kv_heads values in 2^-64 .. 2^64, by default 1. Values beyond 448 scales are
    clamped, those up to 2^-10 of one vanish."""

    def __init__(self, table: PageTable, kv_heads: int, head_dim: int, dtype, k_scales=None, v_scales=None):
        torch = api._torch()
        if dtype not in (torch.float16, torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError(f"dtype {dtype}, expected float16, bfloat16 or float8_e4m3fn")
        self.table = table
        shape = (table.pages, kv_heads, table.page_size, head_dim)
        self.k = torch.empty(shape, dtype=dtype, device=table.device)
        self.v = torch.empty(shape, dtype=dtype, device=table.device)
        for name, x in (("k_scales", k_scales), ("v_scales", v_scales)):
            if x is None:
                continue
            x = np.asarray(x, np.float32)
            if dtype is not torch.float8_e4m3fn:
                raise ValueError(f"{name}: 16-bit pages have none")
            # beyond, their reciprocals or their products with the scores' scale leave fp32
            if x.shape != (kv_heads,) or not np.all((x >= 2.0 ** -64) & (x <= 2.0 ** 64)):
                raise ValueError(f"{name}: expected {kv_heads} values in 2^-64 .. 2^64")
        put = lambda x: None if x is None else torch.from_numpy(api._c(x, np.float32)).to(table.device)  # noqa: E731
        self.k_scales, self.v_scales = put(k_scales), put(v_scales)


class AttentionBlock:
    """One block resident on a device.

    ``qkv`` and ``out`` are prepare_weights_fp8 of (K x (heads + 2 kv_heads)
    head_dim) and (heads head_dim x K) weights, ``gain`` the norm's K values.
    ``head_gains``: (query, key) gains of the RMS norm of each head, head_dim values each;
    ``rotary``: the (freqs, factor) of rotary_frequencies, ``interleaved`` its pairs.
    ``block(X, residual)`` takes batch x tokens x K and returns (Y, h): the
    block's output and X + residual, which are the next block's X and residual.
    With a KeyValueCache the tokens are appended to it and attend to all that it
    holds; a call that raises leaves the cache's length as it was. With a
    PagedKeyValueCache the rows of X are the tokens of the step that its table's
    ``begin`` was last called for, sequence after sequence whatever batch and tokens X
    has, and the rows of Y behind them are not specified. Buffers are kept between calls and grown when more tokens arrive, so
    one block serves one stream at a time (the smaller ones stay, for graphs captured
    with them), and Y and h are new tensors. Over a paged cache the attention's parts
    take up to 68 MB of them in every block (heads of 128 channels)."""

    def __init__(self, gain, qkv, out, heads: int, kv_heads: int, head_dim: int,
                 qkv_bias=None, out_bias=None, eps: float = 1e-6, softcap: float = 0.0,
                 slopes=None, device="cuda", head_gains=None, rotary=None, interleaved: bool = False):
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
        q_gain, k_gain = (None, None) if head_gains is None else head_gains
        for name, x, n in (("gain", gain, qkv.K), ("qkv_bias", qkv_bias, qkv.N),
                           ("out_bias", out_bias, out.N), ("slopes", slopes, heads),
                           ("head_gains", q_gain, head_dim), ("head_gains", k_gain, head_dim)):
            if x is not None and math.prod(np.shape(x)) != n:
                raise ValueError(f"{name}: shape {tuple(np.shape(x))}, expected {n} values")
        # as norm_rotary takes it, in fp32
        if head_gains is not None and not (eps == 0 or (2.0 ** -126 <= np.float32(eps) < math.inf)):
            raise ValueError(f"eps: {eps}, norms of heads take 0 or a finite value from 2^-126 on")
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.eps, self.softcap = float(eps), float(softcap)
        dev = self.device = torch.device(device)

        def put(x):
            return None if x is None else torch.from_numpy(api._c(x, np.float32)).to(dev)

        self.gain, self.slopes = put(gain), put(slopes)
        # what norm_rotary takes; None: heads stay as the product gives them
        self.turn = None
        if head_gains is not None or rotary is not None:
            freqs, factor = (None, 1.0) if rotary is None else rotary
            if freqs is not None:
                freqs = api._c(freqs, np.float64)
                if freqs.ndim != 1 or 2 * len(freqs) > head_dim:
                    raise ValueError(f"rotary: {freqs.shape} pairs in heads of {head_dim}")
                freqs = torch.from_numpy(freqs).to(dev)
            self.turn = dict(freqs=freqs, factor=float(factor), interleaved=bool(interleaved),
                             q_gain=put(q_gain), k_gain=put(k_gain),
                             eps=None if head_gains is None else self.eps)
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
                 key_ranges=None, positions=None):
        """(Y, h) of X (batch x tokens x K, fp16 or bf16), on the current stream. Masks
        as in attention(): ``causal``, ``prefix`` tokens per sequence that all see,
        ``key_ranges``. ``positions`` (int32, batch x tokens): of the rotation, by default
        those behind the tokens held; a page table has its own."""
        torch = api._torch()
        if not isinstance(X, torch.Tensor):
            raise TypeError(f"X: expected a torch tensor, got {type(X).__name__}")
        if X.dtype not in (torch.float16, torch.bfloat16):
            raise ValueError(f"X: dtype {X.dtype}, expected float16 or bfloat16")
        if X.dim() != 3 or X.shape[2] != self.K:
            raise ValueError(f"X: shape {tuple(X.shape)}, expected (batch, tokens, {self.K})")
        if positions is not None and (self.turn is None or self.turn["freqs"] is None):
            raise ValueError("positions: the block has no rotation")
        if positions is not None and not isinstance(positions, torch.Tensor):
            raise TypeError(f"positions: expected a torch tensor, got {type(positions).__name__}")
        if residual is not None and residual.shape != X.shape:
            raise ValueError(f"residual: shape {tuple(residual.shape)}, X has {tuple(X.shape)}")
        if isinstance(cache, PagedKeyValueCache):
            rows, table = X.shape[0] * X.shape[1], cache.table
            if prefix is not None or key_ranges is not None or positions is not None:
                raise ValueError("prefix, key_ranges, positions: a paged cache's table has its own masks and "
                                 "positions")
            if not table.tokens <= rows <= table.step_tokens:
                raise ValueError(f"X: {rows} rows, the step has {table.tokens} tokens (of up to "
                                 f"{table.step_tokens})")
            held = cache.k
            if held.dtype not in (X.dtype, torch.float8_e4m3fn) or held.device != X.device:
                raise ValueError(f"cache: {held.dtype} on {held.device}, X has {X.dtype} on {X.device}")
            if (held.shape[1], held.shape[3]) != (self.kv_heads, self.head_dim):
                raise ValueError(f"cache: {held.shape[1]} heads of {held.shape[3]}, the block has "
                                 f"{self.kv_heads} of {self.head_dim}")
            return self._run(X, residual, cache, causal, None, None, None)
        if positions is not None and positions.shape != X.shape[:2]:
            raise ValueError(f"positions: shape {tuple(positions.shape)}, expected {tuple(X.shape[:2])}")
        if positions is not None and (positions.dtype is not torch.int32 or positions.device != X.device):
            raise ValueError(f"positions: {positions.dtype} on {positions.device}, expected int32 on {X.device}")
        held = None if cache is None else cache.length
        try:
            return self._run(X, residual, cache, causal, prefix, key_ranges, positions)
        except BaseException:
            if cache is not None:
                cache.length = held      # tokens behind it are not seen and written again
            raise

    def _positions(self, B, L, first):
        torch = api._torch()
        return torch.arange(first, first + L, dtype=torch.int32, device=self.device).repeat(B)

    def _run(self, X, residual, cache, causal, prefix, key_ranges, positions):
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
        o = self._buffer("o", (B, L, Hq, D), X.dtype)
        if isinstance(cache, PagedKeyValueCache):
            self._paged(t.view(M, Hq + 2 * Hkv, D), cache, causal, o.view(M, Hq, D))
        else:
            if self.turn is not None:
                if self.turn["freqs"] is None:
                    positions = None
                elif positions is None:
                    positions = self._positions(B, L, 0 if cache is None else cache.length)
                x = t.view(M, Hq + 2 * Hkv, D)
                q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
                paged.norm_rotary(q, k, q, k, positions=None if positions is None else positions.reshape(M),
                                  **self.turn)
            t = t.view(B, L, Hq + 2 * Hkv, D)
            q, k, v = t[:, :, :Hq], t[:, :, Hq:Hq + Hkv], t[:, :, Hq + Hkv:]
            if cache is not None:
                k, v = cache.append(k, v)
            need = api.attention_workspace_bytes(B, L, k.shape[1], Hq, Hkv, D)
            api.attention(q, k, v, o, softcap=self.softcap, slopes=self.slopes, causal=causal,
                          prefix=prefix, key_ranges=key_ranges,
                          ws=self._buffer("attention", (need,), torch.uint8) if need else None)
        codes = self._codes("c", M, Hq * D)
        api.quantize_act_fp8(o.view(M, Hq * D), *codes)
        self._product(*codes, self.out, Y.view(M, K))
        return Y, h

    def _paged(self, t, cache, causal, o):
        """o from the rows t of the QKV product, keys and values through the cache's pages."""
        M, heads, D = t.shape
        Hq, Hkv, table = self.heads, self.kv_heads, cache.table
        q, k, v = t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:]
        pool = (cache.k, cache.v, cache.k_scales, cache.v_scales)
        if self.turn is None:
            paged.paged_write(k, v, table.slots[:M], *pool)
        else:
            paged.norm_rotary_write(q, k, v, q, table.slots[:M], *pool,
                                    positions=None if self.turn["freqs"] is None else table.positions[:M],
                                    **self.turn)
        need = paged.paged_attention_workspace_bytes(M, table.batch, table.width * table.page_size, Hq, Hkv, D)
        paged.paged_attention(q, cache.k, cache.v, table.tables, table.lengths, table.starts, o, cache.k_scales,
                              cache.v_scales, softcap=self.softcap, slopes=self.slopes, causal=causal,
                              ws=self._buffer("attention", (need,), api._torch().uint8) if need else None)
