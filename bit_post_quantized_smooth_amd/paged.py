"""A paged key-value cache: the entry points of include/svdq.h that write, read and
attend to it, and the norm and rotation of heads in front of it.

Pages are tensors of (pages, key heads, page size, D), 16 bits or e4m3 codes
(float8_e4m3fn, or its bits as uint8), each page contiguous. Slots, page tables, lengths
and starts are int32 tensors on the device: a graph captured once serves sequences that
grow and change, since only these tensors' values say which tokens there are.
"""
from __future__ import annotations

import math
import struct

import numpy as np

from . import _lib, api
from ._lib import E4M3, check, lib
from .api import _buf, _dt_block, _dtypes, _on_gpu, _stream, _torch

_HALVES = ("float16", "bfloat16")
_CODES = ("uint8", "float8_e4m3fn")


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str | None = None,
                       scale: float = 1.0, trained: int = 4096, slow: float = 1.0,
                       fast: float = 32.0):
    """(freqs, factor) of a rotation of ``rotary_dim`` channels: radians per position of each
    pair (fp64, base ** (-2i / rotary_dim)) and the factor that its cosines and sines take.

    ``scaling`` stretches a model trained on ``trained`` positions to ``scale`` times as many:
    "linear": every pair turns `scale` times slower; "base": a larger base, which slows the
    slowest pair by `scale` and leaves the fastest; "parts": pairs that turn more than ``fast``
    times over the trained length are left, those that turn less than ``slow`` times are slowed
    by `scale`, those between in proportion, and the factor is 1 + 0.1 ln(scale)."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim: {rotary_dim}, expected a positive even number")
    if not (base > 0 and math.isfinite(base)) or not (scale >= 1 and math.isfinite(scale)):
        raise ValueError(f"base {base} must be positive and scale {scale} at least 1")
    two_i = np.arange(0, rotary_dim, 2, dtype=np.float64)
    if scaling == "base":
        if rotary_dim > 2:
            base = base * scale ** (rotary_dim / (rotary_dim - 2))
        return base ** (-two_i / rotary_dim), 1.0
    freqs = base ** (-two_i / rotary_dim)
    if scaling is None:
        if scale != 1.0:
            raise ValueError("scale: needs a scaling")
        return freqs, 1.0
    if scaling == "linear":
        return freqs / scale, 1.0
    if scaling == "parts":
        if trained < 1 or not slow < fast:
            raise ValueError("parts: needs a trained length and slow < fast")
        turns = trained * freqs / (2 * math.pi)
        kept = np.clip((turns - slow) / (fast - slow), 0.0, 1.0)
        return freqs * kept + freqs / scale * (1.0 - kept), 1.0 + 0.1 * math.log(scale)
    raise ValueError(f"scaling: {scaling!r}, expected None, 'linear', 'base' or 'parts'")


def _here(stream, *ts):
    """All tensors on one GPU, the one that the work is queued on."""
    _on_gpu(*ts)
    for t in ts:
        if t is not None:
            at = _torch().cuda.current_device() if stream is None else stream.device.index
            if t.get_device() != at:
                raise ValueError(f"tensors on device {t.get_device()}, the stream is on {at}")
            return


def _rows(name, t, T, H, D, dtype):
    """Token and head strides of a T x H x D tensor (None: any size)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype is not torch.float16 and t.dtype is not torch.bfloat16:
        raise ValueError(f"{name}: dtype {t.dtype}, expected float16 or bfloat16")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    shape = t.shape
    if len(shape) != 3 or (T is not None and shape[0] != T) or (H is not None and shape[1] != H) \
            or (D is not None and shape[2] != D):
        raise ValueError(f"{name}: shape {tuple(shape)}, expected {(T, H, D)}")
    st, sh, sd = t.stride()
    n, h, d = shape
    if d > 1 and sd != 1:
        raise ValueError(f"{name}: the inner stride must be 1, got {sd}")
    # a dimension of one (or of none) is never stepped over: its stride is free
    return st if n > 1 else 0, sh if h > 1 else 0


def _i32(name, t, *shape):
    """A contiguous int32 tensor of this shape (None: any size)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype is not torch.int32:
        raise ValueError(f"{name}: dtype {t.dtype}, expected int32")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t


def _pool(k_pages, v_pages, k_scales, v_scales, dtype, Hkv, D):
    """(cache dtype, pages, page size, bytes between K's pages, between V's)."""
    torch = _torch()
    strides = []
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
        if t.dtype is not dtype and t.dtype not in _dtypes(_CODES):
            raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype} or one of {_CODES}")
        if t.dim() != 4 or (Hkv is not None and t.shape[1] != Hkv) or (D is not None and t.shape[3] != D):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected (pages, {Hkv}, page size, {D})")
        pages, heads, size, d = t.shape
        sp, sh, ss, sd = t.stride()
        if sd != 1 or ss != d or (heads > 1 and sh != size * d):
            raise ValueError(f"{name}: strides {t.stride()}, each page must be contiguous")
        strides.append((sp if pages > 1 else heads * size * d) * t.element_size())
    if v_pages.dtype is not k_pages.dtype or v_pages.shape != k_pages.shape:
        raise ValueError(f"v_pages: {v_pages.dtype} {tuple(v_pages.shape)}, k_pages has {k_pages.dtype} "
                         f"{tuple(k_pages.shape)}")
    coded = k_pages.dtype is not dtype
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        if t is not None:
            if not coded:
                raise ValueError(f"{name}: 16-bit pages have none")
            _buf(name, t, api._F32, nbytes=4 * k_pages.shape[1])
    return (E4M3 if coded else _dt_block(k_pages), k_pages.shape[0], k_pages.shape[2], *strides)


def _p(t):
    return None if t is None else t.data_ptr()


def _rotation(T, D, positions, freqs, q_gain, k_gain, eps):
    """(pairs, eps of the library) after the checks."""
    if (positions is None) != (freqs is None):
        raise ValueError("positions and freqs: a rotation needs both")
    pairs = 0
    if freqs is not None:
        _i32("positions", positions, T)
        _buf("freqs", freqs, ("float64",))
        pairs = freqs.numel()
        if freqs.dim() != 1 or 2 * pairs > D:
            raise ValueError(f"freqs: shape {tuple(freqs.shape)}, expected up to {D // 2} pairs")
    for name, t in (("q_gain", q_gain), ("k_gain", k_gain)):
        if t is not None:
            if eps is None:
                raise ValueError(f"{name}: needs eps, without which there is no norm")
            _buf(name, t, api._F32, nbytes=4 * D)
    if eps is not None and not (eps >= 0 and math.isfinite(eps)):
        raise ValueError(f"eps: {eps}, expected a finite value >= 0")
    return pairs, -1.0 if eps is None else eps


def norm_rotary(Q, K, Q_out, K_out, positions=None, freqs=None, factor: float = 1.0,
                interleaved: bool = False, q_gain=None, k_gain=None, eps: float | None = None,
                stream=None):
    """svdq_norm_rotary: query heads Q (T x Hq x D) and key heads K (T x Hkv x D, or None
    with K_out), fp16 or bf16, strided views with contiguous channels, into Q_out and K_out
    (which may be Q and K).

    eps: the RMS norm of each head, times q_gain and k_gain (fp32, D); None: no norm.
    positions (int32, T) and freqs (fp64, radians per position of each pair:
    rotary_frequencies): the rotation of the first 2 * len(freqs) channels, pairs of channels
    (i, i + len(freqs)) or, ``interleaved``, (2i, 2i + 1), times ``factor``."""
    q, qo = _rows("Q", Q, None, None, None, None), None
    T, Hq, D = Q.shape
    qo = _rows("Q_out", Q_out, T, Hq, D, Q.dtype)
    k = ko = (0, 0)
    Hkv = 0
    if K is not None or K_out is not None:
        k = _rows("K", K, T, None, D, Q.dtype)
        Hkv = K.shape[1]
        ko = _rows("K_out", K_out, T, Hkv, D, Q.dtype)
    pairs, e = _rotation(T, D, positions, freqs, q_gain, k_gain, eps)
    _here(stream, Q, K, Q_out, K_out, positions, freqs, q_gain, k_gain)
    status = lib.svdq_norm_rotary(
        Q.data_ptr(), _p(K), Q_out.data_ptr(), _p(K_out), _dt_block(Q), T, Hq, Hkv, D,
        struct.pack("8q", *q, *k, *qo, *ko), _p(positions), _p(freqs), pairs, factor,
        1 if interleaved else 0, _p(q_gain), _p(k_gain), e, _stream(stream))
    if status:
        check(status, "svdq_norm_rotary")


def norm_rotary_write(Q, K, V, Q_out, slots, k_pages, v_pages, k_scales=None, v_scales=None,
                      positions=None, freqs=None, factor: float = 1.0, interleaved: bool = False,
                      q_gain=None, k_gain=None, eps: float | None = None, stream=None):
    """svdq_paged_write: norm_rotary with the keys, and the values V (T x Hkv x D) as they are,
    stored into the pages at ``slots`` (int32, T: page * page size + place in the page; a token
    whose slot is outside the pool, such as -1, is stored nowhere). Slots in the pool must
    differ. k_scales, v_scales (fp32, Hkv): the scales of e4m3 pages; values beyond 448 scales
    are clamped."""
    k = _rows("K", K, None, None, None, None)
    T, Hkv, D = K.shape
    v = _rows("V", V, T, Hkv, D, K.dtype)
    q = qo = (0, 0)
    Hq = 0
    if Q is not None or Q_out is not None:
        q = _rows("Q", Q, T, None, D, K.dtype)
        Hq = Q.shape[1]
        qo = _rows("Q_out", Q_out, T, Hq, D, K.dtype)
    pool = _pool(k_pages, v_pages, k_scales, v_scales, K.dtype, Hkv, D)
    _i32("slots", slots, T)
    pairs, e = _rotation(T, D, positions, freqs, q_gain, k_gain, eps)
    _here(stream, K, V, Q, Q_out, slots, k_pages, v_pages, k_scales, v_scales, positions, freqs,
          q_gain, k_gain)
    status = lib.svdq_paged_write(
        _p(Q), K.data_ptr(), V.data_ptr(), _p(Q_out), _dt_block(K), T, Hq, Hkv, D,
        struct.pack("8q", *q, *k, *v, *qo), _p(positions), _p(freqs), pairs, factor,
        1 if interleaved else 0, _p(q_gain), _p(k_gain), e, slots.data_ptr(), k_pages.data_ptr(),
        v_pages.data_ptr(), *pool, _p(k_scales), _p(v_scales), _stream(stream))
    if status:
        check(status, "svdq_paged_write")


def paged_write(K, V, slots, k_pages, v_pages, k_scales=None, v_scales=None, stream=None):
    """svdq_paged_write without queries, norm and rotation: K and V (T x Hkv x D) into the
    pages at ``slots``, as in norm_rotary_write."""
    norm_rotary_write(None, K, V, None, slots, k_pages, v_pages, k_scales, v_scales, stream=stream)


def paged_read(k_pages, v_pages, tables, lengths, K_out, V_out, k_scales=None, v_scales=None,
               stream=None):
    """svdq_paged_read: the first lengths[b] (int32, B) tokens of each sequence out of the pages
    tables[b] (int32, B x width) into K_out and V_out (B x L x Hkv x D, fp16 or bf16; of 16-bit
    pages the same type), codes times their scales. Rows behind a sequence's length are left as
    they were."""
    so = api._heads("K_out", K_out, None, None, None, None, None)
    B, L, Hkv, D = K_out.shape
    sv = api._heads("V_out", V_out, B, L, Hkv, D, K_out.dtype)
    pool = _pool(k_pages, v_pages, k_scales, v_scales, K_out.dtype, Hkv, D)
    _i32("tables", tables, B, None)
    _i32("lengths", lengths, B)
    _here(stream, K_out, V_out, k_pages, v_pages, tables, lengths, k_scales, v_scales)
    status = lib.svdq_paged_read(
        k_pages.data_ptr(), v_pages.data_ptr(), *pool, _p(k_scales), _p(v_scales), tables.data_ptr(),
        tables.shape[1], lengths.data_ptr(), B, L, Hkv, D, K_out.data_ptr(), V_out.data_ptr(),
        _dt_block(K_out), struct.pack("6q", *so, *sv), _stream(stream))
    if status:
        check(status, "svdq_paged_read")


def paged_attention_workspace_bytes(T: int, B: int, capacity: int, Hq: int, Hkv: int, D: int) -> int:
    """Of T tokens of B sequences over up to ``capacity`` keys each (table width * page size)."""
    return int(lib.svdq_paged_attention_workspace_bytes(T, B, capacity, Hq, Hkv, D))


def paged_attention(Q, k_pages, v_pages, tables, lengths, starts, Out, k_scales=None, v_scales=None,
                    scale: float | None = None, softcap: float = 0.0, slopes=None,
                    causal: bool = True, ws=None, stream=None):
    """svdq_paged_attention: Out (T x Hq x D) from Q (T x Hq x D), the new tokens of B sequences
    one after the other: sequence b has rows starts[b] .. starts[b + 1] - 1 (int32, B + 1), which
    are the last of its lengths[b] (int32, B) tokens in the pages tables[b] (int32, B x width),
    their own keys and values written before.

    scale: of the scores, D**-0.5 by default; softcap, slopes: as in attention(); causal: a
    token sees the keys up to its own position, else all of its sequence. A row that sees no
    key is 0, rows of no sequence are left as they were. With a workspace of
    paged_attention_workspace_bytes(T, B, width * page size, Hq, Hkv, D) work is split along
    the keys; calls that may run at once need one each."""
    q = _rows("Q", Q, None, None, None, None)
    T, Hq, D = Q.shape
    o = _rows("Out", Out, T, Hq, D, Q.dtype)
    pool = _pool(k_pages, v_pages, k_scales, v_scales, Q.dtype, None, D)
    Hkv = k_pages.shape[1]
    if Hkv < 1 or Hq < 1 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads over {Hkv} key heads")
    _i32("tables", tables, None, None)
    B, width = tables.shape
    _i32("lengths", lengths, B)
    _i32("starts", starts, B + 1)
    if slopes is not None:
        _buf("slopes", slopes, api._F32, nbytes=4 * Hq)
    if ws is not None:
        _buf("ws", ws, api._BYTES + api._HALF + api._F32)
    _here(stream, Q, Out, k_pages, v_pages, tables, lengths, starts, k_scales, v_scales, slopes, ws)
    status = lib.svdq_paged_attention(
        Q.data_ptr(), Out.data_ptr(), _dt_block(Q), T, Hq, Hkv, D, struct.pack("4q", *q, *o),
        k_pages.data_ptr(), v_pages.data_ptr(), *pool, _p(k_scales), _p(v_scales), tables.data_ptr(),
        width, lengths.data_ptr(), starts.data_ptr(), B, D ** -0.5 if scale is None else scale,
        softcap, _p(slopes), 1 if causal else 0, _p(ws), 0 if ws is None else ws.nbytes,
        _stream(stream))
    if status:
        check(status, "svdq_paged_attention")
