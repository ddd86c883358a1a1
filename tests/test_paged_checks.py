"""The paged cache on the CPU: frequencies, argument checks of the binding and of the C
entry points."""
import ctypes as C
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
sq = pytest.importorskip("bit_post_quantized_smooth_amd")
from bit_post_quantized_smooth_amd import _lib  # noqa: E402

u8, i32, f16, bf16, f32, f64 = torch.uint8, torch.int32, torch.float16, torch.bfloat16, torch.float32, torch.float64
e4m3 = torch.float8_e4m3fn


def z(*shape, dtype=f16):
    return torch.zeros(*shape, dtype=dtype)


def test_frequencies():
    f, a = sq.rotary_frequencies(8, 100.0)
    assert a == 1.0 and f.dtype == np.float64 and np.allclose(f, [1, 100 ** -0.25, 0.1, 100 ** -0.75], rtol=1e-15)
    lin, a = sq.rotary_frequencies(8, 100.0, scaling="linear", scale=4.0)
    assert a == 1.0 and np.array_equal(lin, f / 4)
    b, a = sq.rotary_frequencies(8, 100.0, scaling="base", scale=4.0)
    assert a == 1.0 and b[0] == 1.0 and math.isclose(b[-1], f[-1] / 4, rel_tol=1e-14) and np.all(b[1:-1] < f[1:-1])
    f, _ = sq.rotary_frequencies(64)
    p, a = sq.rotary_frequencies(64, scaling="parts", scale=8.0, trained=4096)
    turns = 4096 * f / (2 * math.pi)
    assert np.array_equal(p[turns >= 32], f[turns >= 32]) and np.allclose(p[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all(p[mid] < f[mid]) and np.all(p[mid] > f[mid] / 8) and np.all(np.diff(p) < 0)
    assert math.isclose(a, 1 + 0.1 * math.log(8))
    for kw in (dict(scaling="parts"), dict(scaling="linear"), dict(scaling="base")):
        assert np.allclose(sq.rotary_frequencies(64, **kw)[0], f, rtol=1e-15)    # times 1: as it is
    assert sq.rotary_frequencies(2, scaling="base", scale=2.0)[0].tolist() == [1.0]


@pytest.mark.parametrize("a", [dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=8, base=0.0),
                               dict(rotary_dim=8, scale=2.0), dict(rotary_dim=8, scaling="linear", scale=0.5),
                               dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, scaling="parts", fast=1.0),
                               dict(rotary_dim=8, scaling="base", scale=math.inf), dict(rotary_dim=8, base=math.nan)])
def test_frequencies_refused(a):
    with pytest.raises(ValueError):
        sq.rotary_frequencies(**a)


T, HQ, HKV, D = 7, 6, 2, 64


def rotary_args(**over):
    a = dict(Q=z(T, HQ, D), K=z(T, HKV, D), Q_out=z(T, HQ, D), K_out=z(T, HKV, D), positions=z(T, dtype=i32),
             freqs=z(16, dtype=f64), q_gain=z(D, dtype=f32), k_gain=z(D, dtype=f32), eps=1e-6)
    a.update(over)
    return a


def write_args(**over):
    a = dict(Q=z(T, HQ, D), K=z(T, HKV, D), V=z(T, HKV, D), Q_out=z(T, HQ, D), slots=z(T, dtype=i32),
             k_pages=z(4, HKV, 16, D).to(e4m3), v_pages=z(4, HKV, 16, D).to(e4m3), k_scales=z(HKV, dtype=f32),
             v_scales=z(HKV, dtype=f32), positions=z(T, dtype=i32), freqs=z(16, dtype=f64))
    a.update(over)
    return a


def read_args(**over):
    a = dict(k_pages=z(4, HKV, 16, D), v_pages=z(4, HKV, 16, D), tables=z(3, 2, dtype=i32), lengths=z(3, dtype=i32),
             K_out=z(3, 20, HKV, D), V_out=z(3, 20, HKV, D))
    a.update(over)
    return a


def attn_args(**over):
    a = dict(Q=z(T, HQ, D), k_pages=z(4, HKV, 16, D), v_pages=z(4, HKV, 16, D), tables=z(3, 2, dtype=i32),
             lengths=z(3, dtype=i32), starts=z(4, dtype=i32), Out=z(T, HQ, D))
    a.update(over)
    return a


def test_correct_cpu_arguments_stop_at_the_device_check():
    for f, a in ((sq.norm_rotary, rotary_args()), (sq.norm_rotary, rotary_args(K=None, K_out=None)),
                 (sq.norm_rotary_write, write_args()), (sq.paged_read, read_args()), (sq.paged_attention, attn_args()),
                 (sq.paged_attention, attn_args(k_pages=z(4, HKV, 16, D, dtype=u8), v_pages=z(4, HKV, 16, D, dtype=u8)))):
        with pytest.raises(ValueError, match="GPU"):
            f(**a)
    w = write_args()
    with pytest.raises(ValueError, match="GPU"):
        sq.paged_write(w["K"], w["V"], w["slots"], w["k_pages"], w["v_pages"], w["k_scales"], w["v_scales"])


@pytest.mark.parametrize("over,match", [
    (dict(Q=z(T, HQ, D, dtype=f32)), "Q"), (dict(K=z(T, HKV, D, dtype=bf16)), "K"), (dict(K=z(T + 1, HKV, D)), "K"),
    (dict(K=None), "K"), (dict(Q_out=z(T, HQ, D + 8)), "Q_out"), (dict(K_out=z(T, HKV + 1, D)), "K_out"),
    (dict(Q=z(T, HQ, 2 * D)[..., ::2]), "inner stride"), (dict(Q=z(T, HQ * D)), "Q"), (dict(Q=np.zeros((T, HQ, D))), "Q"),
    (dict(positions=None), "both"), (dict(freqs=None), "both"), (dict(positions=z(T, dtype=torch.int64)), "positions"),
    (dict(positions=z(T - 1, dtype=i32)), "positions"), (dict(positions=z(2 * T, dtype=i32)[::2]), "contiguous"),
    (dict(freqs=z(16, dtype=f32)), "freqs"), (dict(freqs=z(D // 2 + 1, dtype=f64)), "freqs"),
    (dict(q_gain=z(D - 1, dtype=f32)), "q_gain"), (dict(k_gain=z(D)), "k_gain"), (dict(eps=None), "eps"),
    (dict(eps=-1.0), "eps"), (dict(eps=math.nan), "eps"),
])
def test_rotary_refusals(over, match):
    with pytest.raises((ValueError, TypeError), match=match):
        sq.norm_rotary(**rotary_args(**over))


@pytest.mark.parametrize("over,match", [
    (dict(V=z(T, HKV + 1, D)), "V"), (dict(V=z(T, HKV, D, dtype=bf16)), "V"), (dict(Q=None), "Q"), (dict(Q_out=None), "Q_out"),
    (dict(slots=z(T, dtype=torch.int64)), "slots"), (dict(slots=z(T + 1, dtype=i32)), "slots"),
    (dict(k_pages=z(4, HKV + 1, 16, D).to(e4m3)), "k_pages"), (dict(k_pages=z(4, HKV, 16, D)), "v_pages"),
    (dict(v_pages=z(5, HKV, 16, D).to(e4m3)), "v_pages"), (dict(k_pages=z(4, HKV, 16, D, dtype=bf16)), "k_pages"),
    (dict(k_pages=z(4, HKV, 16, D, dtype=f32)), "k_pages"), (dict(k_pages=z(4, HKV, 16, 2 * D).to(e4m3)[..., :D]), "contiguous"),
    (dict(k_pages=z(4, HKV, 16, D), v_pages=z(4, HKV, 16, D)), "k_scales"), (dict(k_scales=z(HKV + 1, dtype=f32)), "k_scales"),
    (dict(v_scales=z(HKV)), "v_scales"), (dict(k_pages=z(HKV, 16, D).to(e4m3)), "k_pages"), (dict(eps=-1.0), "eps"),
])
def test_write_refusals(over, match):
    with pytest.raises((ValueError, TypeError), match=match):
        sq.norm_rotary_write(**write_args(**over))


@pytest.mark.parametrize("over,match", [
    (dict(K_out=z(3, 20, HKV, D, dtype=bf16)), "V_out"), (dict(V_out=z(3, 20, HKV, D + 8)), "V_out"),
    (dict(K_out=z(3, 20, HKV, D, dtype=bf16), V_out=z(3, 20, HKV, D, dtype=bf16)), "k_pages"),
    (dict(tables=z(2, 2, dtype=i32)), "tables"), (dict(lengths=z(2, dtype=i32)), "lengths"),
    (dict(tables=z(3, 4, dtype=i32)[:, ::2]), "contiguous"), (dict(k_scales=z(HKV, dtype=f32)), "k_scales"),
])
def test_read_refusals(over, match):
    with pytest.raises((ValueError, TypeError), match=match):
        sq.paged_read(**read_args(**over))


@pytest.mark.parametrize("over,match", [
    (dict(Q=z(T, 5, D), Out=z(T, 5, D)), "heads"), (dict(Out=z(T, HQ, D, dtype=bf16)), "Out"), (dict(Out=z(T, D)), "Out"),
    (dict(starts=z(3, dtype=i32)), "starts"), (dict(lengths=z(4, dtype=i32)), "lengths"), (dict(tables=z(6, dtype=i32)), "tables"),
    (dict(lengths=z(3, dtype=torch.int64)), "lengths"), (dict(slopes=z(HKV, dtype=f32)), "slopes"), (dict(ws=[1]), "ws"),
    (dict(Q=z(T, HQ, 72), Out=z(T, HQ, 72)), "k_pages"), (dict(k_scales=z(HKV, dtype=f32)), "k_scales"),
    (dict(Q=z(T, 0, D), Out=z(T, 0, D)), "heads"),
])
def test_attention_refusals(over, match):
    with pytest.raises((ValueError, TypeError), match=match):
        sq.paged_attention(**attn_args(**over))


P, ODD = C.c_void_p(1 << 20), C.c_void_p((1 << 20) + 2)        # never read


def strides(*s):
    return (C.c_int64 * len(s))(*s)


def rot(Q=P, K=P, Qo=P, Ko=P, dt=1, t=4, Hq=2, Hkv=1, d=64, st=None, pos=P, fr=P, n=8, factor=1.0, qg=None, eps=-1.0):
    s = [Hq * d, d, Hkv * d, d, Hq * d, d, Hkv * d, d]
    for i, x in (st or {}).items():
        s[i] = x
    return _lib.lib.svdq_norm_rotary(Q, K, Qo, Ko, dt, t, Hq, Hkv, d, strides(*s), pos, fr, n, factor, 0, qg, None, eps, None)


def test_c_rotary_refuses_on_the_host():
    assert rot(dt=2) == rot(dt=4) == _lib.ERR_DTYPE
    assert rot(t=-1) == rot(d=12) == rot(d=136) == rot(n=33) == rot(n=-1) == rot(Hq=1 << 20) == _lib.ERR_SHAPE
    assert rot(factor=math.inf) == rot(eps=math.nan) == rot(qg=P) == rot(t=1 << 30, Hq=1 << 10) == _lib.ERR_SHAPE
    assert rot(Q=None) == rot(Ko=None) == rot(pos=None) == rot(fr=None) == _lib.ERR_NULL
    assert rot(Q=ODD) == rot(Ko=ODD) == rot(fr=C.c_void_p(4)) == rot(st={1: 4}) == rot(st={0: -8}) == _lib.ERR_ALIGN
    # outputs over themselves, and in place with other strides
    assert rot(st={4: 64}) == rot(st={5: 0}) == rot(st={6: 8}) == _lib.ERR_SHAPE
    assert rot(Q=P, Qo=P, st={0: 256}) == _lib.ERR_SHAPE
    assert rot(t=0, Q=None) == rot(Hq=0, Hkv=0) == _lib.OK
    assert rot(Q=C.c_void_p(1 << 21), K=C.c_void_p(1 << 22), n=0, pos=None, fr=None, Qo=None) == _lib.ERR_NULL


def write(K=P, V=P, slots=P, kp=P, cd=4, dt=1, pages=5, size=16, ks=None, st=16 * 64, t=4, Hq=0, Hkv=1, d=64, kst=None):
    s = [Hq * d, d, Hkv * d, d, Hkv * d, d, Hq * d, d]
    return _lib.lib.svdq_paged_write(None, K, V, None, dt, t, Hq, Hkv, d, strides(*s), None, None, 0, 1.0, 0, None, None,
                                     -1.0, slots, kp, P, cd, pages, size, st if kst is None else kst, st, ks, None, None)


def test_c_write_refuses_on_the_host():
    assert write(dt=2) == write(cd=3) == write(cd=2) == _lib.ERR_DTYPE
    assert write(size=8) == write(size=24) == write(size=2048) == write(size=0) == write(size=-16) == _lib.ERR_SHAPE
    assert write(pages=-1) == write(pages=1 << 28) == write(Hkv=0) == write(kst=16 * 64 - 16) == _lib.ERR_SHAPE
    assert write(kst=16 * 64 + 8) == write(cd=1, st=16 * 64) == write(cd=1, st=32 * 64, ks=P) == _lib.ERR_SHAPE
    assert write(K=None) == write(slots=None) == write(kp=None) == write(Hq=2) == _lib.ERR_NULL
    assert write(kp=C.c_void_p((1 << 20) + 8)) == write(V=ODD) == _lib.ERR_ALIGN
    assert write(t=0, K=None, slots=None, kp=None) == _lib.OK


def read(kp=P, tb=P, ln=P, Ko=P, B=2, L=9, width=3, dt=1, cd=4, st=None, Hkv=1, d=64):
    s = [L * Hkv * d, Hkv * d, d] * 2
    for i, x in (st or {}).items():
        s[i] = x
    return _lib.lib.svdq_paged_read(kp, P, cd, 5, 16, 16 * Hkv * d * 2, 16 * Hkv * d * 2, None, None, tb, width, ln, B, L, Hkv, d,
                                    Ko, P, dt, strides(*s), None)


def test_c_read_refuses_on_the_host():
    assert read(dt=2) == read(cd=3) == _lib.ERR_DTYPE
    assert read(B=-1) == read(L=-1) == read(width=-1) == read(width=1 << 30) == read(d=4) == _lib.ERR_SHAPE
    assert read(st={1: 0}) == read(st={3: 64}) == read(B=1 << 20, L=1 << 20) == _lib.ERR_SHAPE
    assert read(kp=None) == read(tb=None) == read(ln=None) == read(Ko=None) == _lib.ERR_NULL
    assert read(Ko=ODD) == read(tb=ODD) == read(st={0: 9 * 64 + 4}) == _lib.ERR_ALIGN
    assert read(B=0, Ko=None) == read(L=0, Ko=None) == _lib.OK


def attn(Q=P, Out=P, dt=1, t=4, Hq=2, Hkv=1, d=64, st=None, cd=4, size=16, pages=5, tb=P, width=3, ln=P, sr=P, B=2, scale=1.0,
         cap=0.0, ws=None, slopes=None):
    s = [Hq * d, d, Hq * d, d]
    for i, x in (st or {}).items():
        s[i] = x
    page = size * Hkv * d * 2
    return _lib.lib.svdq_paged_attention(Q, Out, dt, t, Hq, Hkv, d, strides(*s), P, P, cd, pages, size, page, page, None, None, tb,
                                         width, ln, sr, B, scale, cap, slopes, 1, ws, 0, None)


def test_c_attention_refuses_on_the_host():
    assert attn(dt=2) == attn(cd=3) == _lib.ERR_DTYPE
    assert attn(Hq=3, Hkv=2) == attn(Hq=0) == attn(Hkv=0) == attn(t=-1) == attn(B=-1) == attn(d=132) == _lib.ERR_SHAPE
    assert attn(cap=-1.0) == attn(cap=math.inf) == attn(scale=math.nan) == attn(width=-1) == attn(size=12) == _lib.ERR_SHAPE
    assert attn(t=1 << 29, Hq=4) == attn(st={2: 64}) == attn(width=1 << 28) == _lib.ERR_SHAPE
    assert attn(t=1, Hq=257) == attn(width=(1 << 22) + 1) == attn(scale=1e-15, slopes=P) == _lib.ERR_SHAPE
    assert attn(t=1, Hq=256, Q=None) == attn(width=1 << 22, Q=None) == attn(scale=0.0, slopes=P, Q=None) == _lib.ERR_NULL
    assert attn(Q=None) == attn(Out=None) == attn(tb=None) == attn(ln=None) == attn(sr=None) == _lib.ERR_NULL
    assert attn(Q=ODD) == attn(ws=ODD) == attn(sr=ODD) == attn(st={3: 68}) == _lib.ERR_ALIGN
    assert attn(t=0, Q=None) == attn(B=0, Q=None) == _lib.OK


def test_workspace_of_what_is_refused():
    assert sq.paged_attention_workspace_bytes(4, 1, 4000, 3, 2, 64) == 0
    assert sq.paged_attention_workspace_bytes(-1, 1, 4000, 2, 2, 64) == 0


def test_c_write_refuses_one_memory_for_keys_and_values():
    assert write(kp=P) == _lib.ERR_SHAPE                     # keys and values into the same bytes, in any order
    assert write(kp=P, pages=0, t=0) == _lib.OK


@pytest.mark.parametrize("eps", [1e-40, 1.1e-38])
def test_c_eps_below_normal_numbers_refused(eps):
    k = C.c_void_p(1 << 22)
    out = C.c_void_p(1 << 24)
    assert rot(K=k, Qo=out, Ko=C.c_void_p(1 << 26), eps=eps) == _lib.ERR_SHAPE


def test_block_positions_must_be_a_tensor():
    w = np.zeros((64, 3 * 64), np.float32)
    block = sq.AttentionBlock(np.ones(64, np.float32), sq.prepare_weights_fp8(w), sq.prepare_weights_fp8(w[:, :64]), 1, 1, 64,
                              device="cpu", rotary=sq.rotary_frequencies(64))
    with pytest.raises(TypeError, match="positions"):
        block(z(1, 2, 64), positions=[0, 1])
    with pytest.raises(ValueError, match="positions"):
        block(z(1, 2, 64), positions=z(1, 3, dtype=i32))
