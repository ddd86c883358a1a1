"""The paged cache's C entry points on the CPU: each refusal is its own check's, by its message,
every argument but the one being good (all tensors at addresses of their own)."""
import ctypes as C
import math

import pytest

torch = pytest.importorskip("torch")
pytest.importorskip("bit_post_quantized_smooth_amd")
from bit_post_quantized_smooth_amd import _lib  # noqa: E402

SHAPE, ALIGN, NULL, DTYPE = _lib.ERR_SHAPE, _lib.ERR_ALIGN, _lib.ERR_NULL, _lib.ERR_DTYPE


def at(i, odd=0):
    """An address of its own, never read: every call here is refused before the device is asked for."""
    return C.c_void_p((i + 1 << 30) + odd)


def strides(*s):
    return (C.c_int64 * len(s))(*s)


def refused(status, want, match):
    assert status == want, (status, _lib.last_error())
    assert match in _lib.last_error(), _lib.last_error()


def write(over=None, st=None, dt=1, t=4, Hq=2, Hkv=1, d=64, cd=4, pages=5, size=16, ks_=16 * 64, vs_=16 * 64, n=8,
          factor=1.0, eps=-1.0):
    p = dict(Q=at(0), K=at(1), V=at(2), Qo=at(3), pos=at(4), fr=at(5), qg=None, kg=None, slots=at(6), kp=at(7), vp=at(8),
             ks=None, vs=None)
    p.update(over or {})
    s = [Hq * d, d, Hkv * d, d, Hkv * d, d, Hq * d, d]
    for i, x in (st or {}).items():
        s[i] = x
    return _lib.lib.svdq_paged_write(p["Q"], p["K"], p["V"], p["Qo"], dt, t, Hq, Hkv, d, strides(*s), p["pos"], p["fr"], n,
                                     factor, 0, p["qg"], p["kg"], eps, p["slots"], p["kp"], p["vp"], cd, pages, size, ks_, vs_,
                                     p["ks"], p["vs"], None)


@pytest.mark.parametrize("a,status,match", [
    *((dict(size=x), SHAPE, "page size") for x in (8, 24, 2048, 0, -16)),
    (dict(pages=-1), SHAPE, "2^31 tokens"), (dict(pages=(1 << 27) + 1), SHAPE, "2^31 tokens"),
    (dict(Hkv=0), SHAPE, "no key heads"),
    *((dict(ks_=x), SHAPE, "page stride") for x in (16 * 64 - 16, 16 * 64 + 8, -1024, 1 << 41)),
    *((dict(vs_=x), SHAPE, "page stride") for x in (16 * 64 - 16, 16 * 64 + 8, -1024, 1 << 41)),
    (dict(cd=1, ks_=32 * 64), SHAPE, "page stride"),       # 16-bit pages are twice as long
    (dict(cd=1, ks_=32 * 64, vs_=32 * 64, over=dict(ks=at(9))), SHAPE, "no scales"),
    (dict(cd=1, ks_=32 * 64, vs_=32 * 64, over=dict(vs=at(9))), SHAPE, "no scales"),
    (dict(cd=2), DTYPE, "neither e4m3"), (dict(cd=3), DTYPE, "neither e4m3"), (dict(dt=2), DTYPE, "f16 or bf16"),
    (dict(t=-1), SHAPE, "out of range"), (dict(d=12), SHAPE, "multiple of 8"), (dict(d=136), SHAPE, "multiple of 8"),
    (dict(t=1 << 30, Hq=1 << 10), SHAPE, "one launch"),
    (dict(n=33), SHAPE, "rotated channels"), (dict(factor=math.inf), SHAPE, "factor"), (dict(eps=math.nan), SHAPE, "eps"),
    (dict(eps=1e-40), SHAPE, "normal numbers"), (dict(over=dict(qg=at(9))), SHAPE, "gain needs"),
    *((dict(over={x: None}), NULL, "null pointer") for x in ("Q", "K", "V", "Qo", "pos", "fr", "slots")),
    *((dict(over={x: None}), NULL, "null pages") for x in ("kp", "vp")),
    *((dict(over={x: at(9, 2)}), ALIGN, "16-byte") for x in ("Q", "K", "V", "Qo", "kp", "vp")),
    (dict(over=dict(slots=at(9, 2))), ALIGN, "4-byte"), (dict(over=dict(ks=at(9, 2))), ALIGN, "4-byte"),
    (dict(st={2: 68}), ALIGN, "stride"), (dict(st={6: 64}), SHAPE, "overlap itself"),
    (dict(over=dict(Q=at(3)), st={0: 256}), SHAPE, "in place"),
    (dict(over=dict(vp=at(7))), SHAPE, "same pages"),
])
def test_write(a, status, match):
    refused(write(**a), status, match)


def rotate(over=None, st=None, dt=1, t=4, Hq=2, Hkv=1, d=64, n=8, factor=1.0, eps=-1.0):
    p = dict(Q=at(0), K=at(1), Qo=at(2), Ko=at(3), pos=at(4), fr=at(5), qg=None, kg=None)
    p.update(over or {})
    s = [Hq * d, d, Hkv * d, d, Hq * d, d, Hkv * d, d]
    for i, x in (st or {}).items():
        s[i] = x
    return _lib.lib.svdq_norm_rotary(p["Q"], p["K"], p["Qo"], p["Ko"], dt, t, Hq, Hkv, d, strides(*s), p["pos"], p["fr"], n,
                                     factor, 0, p["qg"], p["kg"], eps, None)


@pytest.mark.parametrize("a,status,match", [
    (dict(dt=2), DTYPE, "f16 or bf16"), (dict(t=-1), SHAPE, "out of range"), (dict(Hq=1 << 20), SHAPE, "out of range"),
    (dict(d=12), SHAPE, "multiple of 8"), (dict(t=1 << 30, Hq=1 << 10), SHAPE, "one launch"),
    (dict(n=33), SHAPE, "rotated channels"), (dict(n=-1), SHAPE, "rotated channels"), (dict(factor=math.inf), SHAPE, "factor"),
    (dict(eps=math.nan), SHAPE, "eps"), (dict(eps=1.1e-38), SHAPE, "normal numbers"),
    (dict(over=dict(kg=at(9))), SHAPE, "gain needs"),
    *((dict(over={x: None}), NULL, "null pointer") for x in ("Q", "K", "Qo", "Ko", "pos", "fr")),
    *((dict(over={x: at(9, 2)}), ALIGN, "16-byte") for x in ("Q", "K", "Qo", "Ko")),
    (dict(over=dict(fr=at(9, 4))), ALIGN, "alignment"), (dict(over=dict(pos=at(9, 2))), ALIGN, "alignment"),
    (dict(st={1: 4}), ALIGN, "stride"), (dict(st={0: -8}), ALIGN, "stride"),
    (dict(st={4: 64}), SHAPE, "overlap itself"), (dict(st={5: 0}), SHAPE, "overlap itself"),
    (dict(st={6: 8}), SHAPE, "overlap itself"), (dict(over=dict(Q=at(2)), st={0: 256}), SHAPE, "in place"),
    (dict(over=dict(K=at(3)), st={2: 256}), SHAPE, "in place"),
])
def test_rotation(a, status, match):
    refused(rotate(**a), status, match)


def read(over=None, st=None, dt=1, cd=4, B=2, L=9, width=3, Hkv=2, d=64, size=16, pages=5):
    p = dict(kp=at(0), vp=at(1), ks=None, vs=None, tb=at(2), ln=at(3), Ko=at(4), Vo=at(5))
    p.update(over or {})
    s = [L * Hkv * d, Hkv * d, d] * 2
    for i, x in (st or {}).items():
        s[i] = x
    page = 2 * abs(size) * Hkv * d
    return _lib.lib.svdq_paged_read(p["kp"], p["vp"], cd, pages, size, page, page, p["ks"], p["vs"], p["tb"], width, p["ln"], B,
                                    L, Hkv, d, p["Ko"], p["Vo"], dt, strides(*s), None)


@pytest.mark.parametrize("a,status,match", [
    (dict(dt=2), DTYPE, "f16 or bf16"), (dict(cd=3), DTYPE, "neither e4m3"), (dict(d=4), SHAPE, "multiple of 8"),
    (dict(L=-1), SHAPE, "out of range"), (dict(size=24), SHAPE, "page size"), (dict(pages=-1), SHAPE, "2^31 tokens"),
    *((dict([kv]), SHAPE, "pages out of range") for kv in (("B", -1), ("width", -1), ("width", 1 << 30))),
    (dict(B=1 << 20, L=1 << 20), SHAPE, "pages out of range"),
    *((dict(over={x: None}), NULL, "null pointer") for x in ("tb", "ln", "Ko", "Vo")),
    *((dict(over={x: None}), NULL, "null pages") for x in ("kp", "vp")),
    *((dict(over={x: at(9, 2)}), ALIGN, "16-byte") for x in ("kp", "vp", "Ko", "Vo")),
    *((dict(over={x: at(9, 2)}), ALIGN, "4-byte") for x in ("tb", "ln")),
    (dict(st={0: 9 * 128 + 4}), ALIGN, "stride"), (dict(st={1: 0}), SHAPE, "overlap itself"),
    (dict(st={5: 32}), SHAPE, "overlap itself"), (dict(st={3: 128}), SHAPE, "overlap itself"),
])
def test_read(a, status, match):
    refused(read(**a), status, match)


def attend(over=None, st=None, dt=1, t=4, Hq=2, Hkv=1, d=64, cd=4, size=16, pages=5, width=3, B=2, scale=1.0, cap=0.0):
    p = dict(Q=at(0), Out=at(1), kp=at(2), vp=at(3), ks=None, vs=None, tb=at(4), ln=at(5), sr=at(6), sl=None, ws=None)
    p.update(over or {})
    s = [Hq * d, d, Hq * d, d]
    for i, x in (st or {}).items():
        s[i] = x
    page = 2 * abs(size) * Hkv * d
    return _lib.lib.svdq_paged_attention(p["Q"], p["Out"], dt, t, Hq, Hkv, d, strides(*s), p["kp"], p["vp"], cd, pages, size,
                                         page, page, p["ks"], p["vs"], p["tb"], width, p["ln"], p["sr"], B, scale, cap,
                                         p["sl"], 1, p["ws"], 0, None)


@pytest.mark.parametrize("a,status,match", [
    (dict(dt=2), DTYPE, "f16 or bf16"), (dict(cd=3), DTYPE, "neither e4m3"), (dict(d=132), SHAPE, "multiple of 8"),
    (dict(size=12), SHAPE, "page size"), (dict(Hkv=0), SHAPE, "no key heads"),
    (dict(cd=1, over=dict(ks=at(9))), SHAPE, "no scales"),
    *((a, SHAPE, "heads out of range") for a in (dict(Hq=3, Hkv=2), dict(Hq=0), dict(B=-1), dict(t=1 << 29, Hq=4),
                                                 dict(t=1, Hq=257), dict(width=(1 << 22) + 1))),
    (dict(width=-1), SHAPE, "width"), (dict(width=1 << 28), SHAPE, "width"),
    *((a, SHAPE, "finite") for a in (dict(cap=-1.0), dict(cap=math.inf), dict(scale=math.nan))),
    (dict(scale=1e-15, over=dict(sl=at(9))), SHAPE, "2^-40"),
    *((dict(over={x: None}), NULL, "null pointer") for x in ("Q", "Out", "tb", "ln", "sr")),
    *((dict(over={x: None}), NULL, "null pages") for x in ("kp", "vp")),
    *((dict(over={x: at(9, 2)}), ALIGN, "16-byte") for x in ("Q", "Out", "ws", "kp", "vp")),
    *((dict(over={x: at(9, 2)}), ALIGN, "4-byte") for x in ("tb", "ln", "sr", "sl", "vs")),
    (dict(st={3: 68}), ALIGN, "stride"), (dict(st={2: 64}), SHAPE, "overlap itself"),
])
def test_attention(a, status, match):
    refused(attend(**a), status, match)
