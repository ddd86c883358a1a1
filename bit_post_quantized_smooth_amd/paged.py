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
from ._lib import BF16, E4M3, F16, check, lib
from .api import _buf, _on_gpu, _torch

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


# The checks run on every call and a token's kernels take no longer than they do: each
# first tests the whole of what it requires with the cheapest accessors, and only a
# tensor that fails is looked at piece by piece for the message.

# (without torch there are no tensors to look at, and _torch() says so)
_I32, _F32, _F64, _F16, _BF16, _CODED = (
    getattr(_lib.torch, n, None)
    for n in ("int32", "float32", "float64", "float16", "bfloat16", "float8_e4m3fn"))
_U8 = getattr(_lib.torch, "uint8", None)
_eight, _six, _four = (struct.Struct(f"{n}q").pack for n in (8, 6, 4))


_device = getattr(getattr(_lib.torch, "_C", None), "_cuda_getDevice", None)
_raw_stream = getattr(getattr(_lib.torch, "_C", None), "_cuda_getCurrentRawStream", None)
if _device is None or _raw_stream is None:        # a torch without these names
    def _device():
        return _torch().cuda.current_device()

    def _raw_stream(device):
        return _torch().cuda.current_stream(device).cuda_stream


def _queue(stream, first, *others):
    """The handle of the stream that the work goes to, all tensors being on its GPU."""
    at = first.get_device()
    for t in others:
        if t is not None and t.get_device() != at:
            break
    else:
        if at >= 0:
            if stream is None:
                if at == _device():
                    return _raw_stream(at)
            elif at == stream.device.index:
                return stream.cuda_stream
    _on_gpu(first, *others)
    raise ValueError(f"tensors on device {at}, the stream is on "
                     f"{_device() if stream is None else stream.device.index}")


def _refuse_heads(first, second, positions, freqs, slots=None):
    """Raises for the first thing wrong with tensors of heads, (name, tensor) each: `first` of
    one shape T x H x D and type, `second` of another H; with a rotation and slots of T."""
    torch = _torch()
    T = D = dtype = None
    for some in (first, second):
        H = None
        for name, t in some:
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
            if t.dtype is not _F16 and t.dtype is not _BF16:
                raise ValueError(f"{name}: dtype {t.dtype}, expected float16 or bfloat16")
            if dtype is not None and t.dtype is not dtype:
                raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
            shape = tuple(t.shape)
            if len(shape) != 3 or any(n is not None and n != m for n, m in zip((T, H, D), shape)):
                raise ValueError(f"{name}: shape {shape}, expected {(T, H, D)}")
            (T, H, D), dtype = shape, t.dtype
            if t.stride(2) != 1:
                raise ValueError(f"{name}: the inner stride must be 1, got {t.stride(2)}")
    if slots is not None:
        _flat("slots", slots, _I32, (T,))
    if (positions is None) != (freqs is None):
        raise ValueError("positions and freqs: a rotation needs both")
    if freqs is not None:
        _flat("positions", positions, _I32, (T,))
        shape = tuple(getattr(freqs, "shape", ()))
        if len(shape) != 1 or 2 * shape[0] > D:
            raise ValueError(f"freqs: shape {shape}, expected up to {D // 2} pairs")
        _flat("freqs", freqs, _F64, shape)


def _flat(name, t, dtype, shape):
    """A contiguous tensor of this type and shape."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return
    except AttributeError:
        pass
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name}: must be contiguous")


def _tables(t, B):
    """(sequences, width) of the page tables; B: of that many sequences (None: any)."""
    try:
        shape = t.shape
        if len(shape) == 2 and (B is None or shape[0] == B) and t.dtype is _I32 and t.is_contiguous():
            return shape
    except AttributeError:
        pass
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"tables: expected a torch tensor, got {type(t).__name__}")
    if len(t.shape) != 2 or (B is not None and t.shape[0] != B):
        raise ValueError(f"tables: shape {tuple(t.shape)}, expected ({B}, pages)")
    _flat("tables", t, _I32, t.shape)


def _pool(k_pages, v_pages, k_scales, v_scales, dtype, Hkv, D):
    """(cache dtype, pages, page size, bytes between K's pages, between V's); Hkv None: any."""
    kind = None
    try:
        shape, kind = k_pages.shape, k_pages.dtype
        pages, heads, size, d = shape
        kp, kh, kr, kd = k_pages.stride()
        vp, vh, vr, vd = v_pages.stride()
        good = ((kind is dtype or kind is _CODED or kind is _U8) and v_pages.dtype is kind and v_pages.shape == shape
                and d == D and (Hkv is None or heads == Hkv) and kd == vd == 1 and kr == vr == d
                and (heads < 2 or kh == vh == size * d))
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        _refuse_pages(k_pages, v_pages, dtype, Hkv, D)
    if k_scales is not None or v_scales is not None:
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            if t is not None:
                if kind is dtype:
                    raise ValueError(f"{name}: 16-bit pages have none")
                _flat(name, t, _F32, (heads,))
    if pages < 2:
        kp = vp = heads * size * d
    if kind is dtype:
        return BF16 if kind is _BF16 else F16, pages, size, 2 * kp, 2 * vp
    return E4M3, pages, size, kp, vp


def _refuse_pages(k_pages, v_pages, dtype, Hkv, D):
    """Raises for the first of the two that is not pages of this type, heads and channels."""
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if not isinstance(t, _torch().Tensor):
            raise TypeError(f"{name}: expected a torch tensor, got {type(t).__name__}")
        if t.dtype is not dtype and t.dtype is not _CODED and t.dtype is not _U8:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype} or one of {_CODES}")
        if t.dim() != 4 or (Hkv is not None and t.shape[1] != Hkv) or t.shape[3] != D:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected (pages, {Hkv}, page size, {D})")
        _, heads, size, d = t.shape
        _, sh, sr, sd = t.stride()
        if sd != 1 or sr != d or (heads > 1 and sh != size * d):
            raise ValueError(f"{name}: strides {t.stride()}, each page must be contiguous")
    raise ValueError(f"v_pages: {v_pages.dtype} {tuple(v_pages.shape)}, k_pages has {k_pages.dtype} "
                     f"{tuple(k_pages.shape)}")


def _norm(eps, q_gain, k_gain, D):
    """eps after the checks of the norm."""
    if q_gain is not None:
        _flat("q_gain", q_gain, _F32, (D,))
    if k_gain is not None:
        _flat("k_gain", k_gain, _F32, (D,))
    if not (eps >= 0 and math.isfinite(eps)):
        raise ValueError(f"eps: {eps}, expected a finite value >= 0")
    return eps


def norm_rotary(Q, K, Q_out, K_out, positions=None, freqs=None, factor: float = 1.0,
                interleaved: bool = False, q_gain=None, k_gain=None, eps: float | None = None,
                stream=None):
    """svdq_norm_rotary: query heads Q (T x Hq x D) and key heads K (T x Hkv x D, or None
    with K_out), fp16 or bf16, strided views with contiguous channels, into Q_out and K_out
    (which may be Q and K, but not one memory).

    eps: the RMS norm of each head, times q_gain and k_gain (fp32, D); None: no norm.
    positions (int32, T) and freqs (fp64, radians per position of each pair:
    rotary_frequencies): the rotation of the first 2 * len(freqs) channels, pairs of channels
    (i, i + len(freqs)) or, ``interleaved``, (2i, 2i + 1), times ``factor``."""
    try:
        T, Hq, D = shape = Q.shape
        dtype = Q.dtype
        qt, qh, qd = Q.stride()
        ot, oh, od = Q_out.stride()
        good = (Q_out.shape == shape and Q_out.dtype is dtype and (dtype is _F16 or dtype is _BF16)
                and qd == od == 1)
        Hkv = kt = kh = nt = nh = pairs = 0
        if K is not None or K_out is not None:
            Tk, Hkv, Dk = shape = K.shape
            kt, kh, kd = K.stride()
            nt, nh, nd = K_out.stride()
            good = (good and Tk == T and Dk == D and K.dtype is dtype and K_out.dtype is dtype
                    and K_out.shape == shape and kd == nd == 1)
        if freqs is not None:
            pairs, = freqs.shape
            good = (good and 2 * pairs <= D and freqs.dtype is _F64 and freqs.is_contiguous()
                    and positions.dtype is _I32 and positions.shape == (T,) and positions.is_contiguous())
        elif positions is not None:
            good = False
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        _refuse_heads((("Q", Q), ("Q_out", Q_out)),
                      () if K is None and K_out is None else (("K", K), ("K_out", K_out)),
                      positions, freqs)
    # a dimension of one (or of none) is never stepped over: its stride is free
    if T < 2:
        qt = ot = kt = nt = 0
    if Hq < 2:
        qh = oh = 0
    if Hkv < 2:
        kh = nh = 0
    if eps is None:
        e = -1.0
        if q_gain is not None or k_gain is not None:
            raise ValueError("q_gain and k_gain: need eps, without which there is no norm")
    else:
        e = _norm(eps, q_gain, k_gain, D)
    queue = _queue(stream, Q, K, Q_out, K_out, positions, freqs, q_gain, k_gain)
    status = lib.svdq_norm_rotary(
        Q.data_ptr(), None if K is None else K.data_ptr(), Q_out.data_ptr(),
        None if K_out is None else K_out.data_ptr(), BF16 if dtype is _BF16 else F16, T, Hq, Hkv, D,
        _eight(qt, qh, kt, kh, ot, oh, nt, nh), None if freqs is None else positions.data_ptr(),
        None if freqs is None else freqs.data_ptr(), pairs, factor, 1 if interleaved else 0,
        None if q_gain is None else q_gain.data_ptr(), None if k_gain is None else k_gain.data_ptr(),
        e, queue)
    if status:
        check(status, "svdq_norm_rotary")


def norm_rotary_write(Q, K, V, Q_out, slots, k_pages, v_pages, k_scales=None, v_scales=None,
                      positions=None, freqs=None, factor: float = 1.0, interleaved: bool = False,
                      q_gain=None, k_gain=None, eps: float | None = None, stream=None):
    """svdq_paged_write: norm_rotary with the keys, and the values V (T x Hkv x D) as they are,
    stored into the pages at ``slots`` (int32, T: page * page size + place in the page; a token
    whose slot is outside the pool, such as -1, is stored nowhere). Slots in the pool must
    differ. k_scales, v_scales (fp32, Hkv, 2^-64 .. 2^64): the scales of e4m3 pages; values beyond
    448 scales are clamped."""
    try:
        T, Hkv, D = shape = K.shape
        dtype = K.dtype
        kt, kh, kd = K.stride()
        vt, vh, vd = V.stride()
        good = (V.shape == shape and V.dtype is dtype and (dtype is _F16 or dtype is _BF16) and kd == vd == 1
                and slots.dtype is _I32 and slots.shape == (T,) and slots.is_contiguous())
        Hq = qt = qh = ot = oh = pairs = 0
        if Q is not None or Q_out is not None:
            Tq, Hq, Dq = shape = Q.shape
            qt, qh, qd = Q.stride()
            ot, oh, od = Q_out.stride()
            good = (good and Tq == T and Dq == D and Q.dtype is dtype and Q_out.dtype is dtype
                    and Q_out.shape == shape and qd == od == 1)
        if freqs is not None:
            pairs, = freqs.shape
            good = (good and 2 * pairs <= D and freqs.dtype is _F64 and freqs.is_contiguous()
                    and positions.dtype is _I32 and positions.shape == (T,) and positions.is_contiguous())
        elif positions is not None:
            good = False
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        _refuse_heads((("K", K), ("V", V)),
                      () if Q is None and Q_out is None else (("Q", Q), ("Q_out", Q_out)),
                      positions, freqs, slots)
    if T < 2:
        kt = vt = qt = ot = 0
    if Hkv < 2:
        kh = vh = 0
    if Hq < 2:
        qh = oh = 0
    pool = _pool(k_pages, v_pages, k_scales, v_scales, dtype, Hkv, D)
    if eps is None:
        e = -1.0
        if q_gain is not None or k_gain is not None:
            raise ValueError("q_gain and k_gain: need eps, without which there is no norm")
    else:
        e = _norm(eps, q_gain, k_gain, D)
    queue = _queue(stream, K, V, Q, Q_out, slots, k_pages, v_pages, k_scales, v_scales, positions,
                   freqs, q_gain, k_gain)
    status = lib.svdq_paged_write(
        None if Q is None else Q.data_ptr(), K.data_ptr(), V.data_ptr(),
        None if Q_out is None else Q_out.data_ptr(), BF16 if dtype is _BF16 else F16, T, Hq, Hkv, D,
        _eight(qt, qh, kt, kh, vt, vh, ot, oh), None if freqs is None else positions.data_ptr(),
        None if freqs is None else freqs.data_ptr(), pairs, factor, 1 if interleaved else 0,
        None if q_gain is None else q_gain.data_ptr(), None if k_gain is None else k_gain.data_ptr(),
        e, slots.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), *pool,
        None if k_scales is None else k_scales.data_ptr(),
        None if v_scales is None else v_scales.data_ptr(), queue)
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
    pages the same type; not one memory), codes times their scales. Rows behind a sequence's
    length are left as they were."""
    try:
        B, L, Hkv, D = shape = K_out.shape
        dtype = K_out.dtype
        kb, kt, kh, kd = K_out.stride()
        vb, vt, vh, vd = V_out.stride()
        rows, width = tables.shape
        good = (V_out.shape == shape and V_out.dtype is dtype and (dtype is _F16 or dtype is _BF16)
                and kd == vd == 1 and rows == B and tables.dtype is _I32 and tables.is_contiguous()
                and lengths.dtype is _I32 and lengths.shape == (B,) and lengths.is_contiguous())
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        api._heads("K_out", K_out, None, None, None, None, None)
        api._heads("V_out", V_out, *K_out.shape, K_out.dtype)
        _tables(tables, K_out.shape[0])
        _flat("lengths", lengths, _I32, (K_out.shape[0],))
    # a dimension of one (or of none) is never stepped over: its stride is free
    if B < 2:
        kb = vb = 0
    if L < 2:
        kt = vt = 0
    if Hkv < 2:
        kh = vh = 0
    pool = _pool(k_pages, v_pages, k_scales, v_scales, dtype, Hkv, D)
    queue = _queue(stream, K_out, V_out, k_pages, v_pages, tables, lengths, k_scales, v_scales)
    status = lib.svdq_paged_read(
        k_pages.data_ptr(), v_pages.data_ptr(), *pool,
        None if k_scales is None else k_scales.data_ptr(),
        None if v_scales is None else v_scales.data_ptr(), tables.data_ptr(), width,
        lengths.data_ptr(), B, L, Hkv, D, K_out.data_ptr(), V_out.data_ptr(),
        BF16 if dtype is _BF16 else F16, _six(kb, kt, kh, vb, vt, vh), queue)
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

    scale: of the scores, D**-0.5 by default, its size with k_scales 0 or 2^-40 .. 2^60 (with
    slopes 0 or from 2^-40 on); softcap, slopes: as in attention(); causal: a
    token sees the keys up to its own position, else all of its sequence. A row that sees no
    key is 0, rows of no sequence are left as they were. With a workspace of
    paged_attention_workspace_bytes(T, B, width * page size, Hq, Hkv, D) work is split along
    the keys; calls that may run at once need one each."""
    try:
        T, Hq, D = shape = Q.shape
        dtype = Q.dtype
        qt, qh, qd = Q.stride()
        ot, oh, od = Out.stride()
        B, width = tables.shape
        good = (Out.shape == shape and Out.dtype is dtype and (dtype is _F16 or dtype is _BF16)
                and qd == od == 1 and tables.dtype is _I32 and tables.is_contiguous()
                and lengths.dtype is _I32 and lengths.shape == (B,) and lengths.is_contiguous()
                and starts.dtype is _I32 and starts.shape == (B + 1,) and starts.is_contiguous())
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        _refuse_heads((("Q", Q), ("Out", Out)), (), None, None)
        B, width = _tables(tables, None)
        _flat("lengths", lengths, _I32, (B,))
        _flat("starts", starts, _I32, (B + 1,))
    if T < 2:
        qt = ot = 0
    if Hq < 2:
        qh = oh = 0
    pool = _pool(k_pages, v_pages, k_scales, v_scales, dtype, None, D)
    Hkv = k_pages.shape[1]
    if Hkv < 1 or Hq < 1 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads over {Hkv} key heads")
    if slopes is not None:
        _flat("slopes", slopes, _F32, (Hq,))
    if ws is not None:
        _buf("ws", ws, api._BYTES + api._HALF + api._F32)
    queue = _queue(stream, Q, Out, k_pages, v_pages, tables, lengths, starts, k_scales, v_scales, slopes,
                   ws)
    status = lib.svdq_paged_attention(
        Q.data_ptr(), Out.data_ptr(), BF16 if dtype is _BF16 else F16, T, Hq, Hkv, D,
        _four(qt, qh, ot, oh), k_pages.data_ptr(), v_pages.data_ptr(), *pool,
        None if k_scales is None else k_scales.data_ptr(),
        None if v_scales is None else v_scales.data_ptr(), tables.data_ptr(), width,
        lengths.data_ptr(), starts.data_ptr(), B, D ** -0.5 if scale is None else scale, softcap,
        None if slopes is None else slopes.data_ptr(), 1 if causal else 0,
        None if ws is None else ws.data_ptr(), 0 if ws is None else ws.nbytes, queue)
    if status:
        check(status, "svdq_paged_attention")
