"""The 8-bit attention block on the CPU: host weight preparation against the
format, argument checks of the binding and of the C entry points."""
import ctypes as C

import numpy as np
import pytest

torch = pytest.importorskip("torch")
sq = pytest.importorskip("bit_post_quantized_smooth_amd")
import block_ref as R  # noqa: E402
from bit_post_quantized_smooth_amd import _lib  # noqa: E402

u8, i32, f16, bf16, f32 = torch.uint8, torch.int32, torch.float16, torch.bfloat16, torch.float32


def z(*shape, dtype=f16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("K,N", [(1, 1), (128, 128), (130, 257), (300, 40), (1000, 129)])
def test_weight_preparation(K, N):
    rng = np.random.default_rng(K + N)
    W = (rng.standard_normal((K, N)) * 0.02).astype(np.float32)
    W[K // 2] *= 30
    p = sq.prepare_weights_fp8(W)
    Kp, G, NB = R.padded(K), R.padded(K) // 128, -(-N // 128)
    assert p.fmt == "fp8" and p.w_codes.shape == (N, Kp) and p.w_scales.shape == (NB, G)
    q = R.decode(torch.from_numpy(p.w_codes)).numpy()
    assert np.all(q[:, K:] == 0)
    for nb in range(NB):
        for g in range(G):
            blk = W[g * 128:(g + 1) * 128, nb * 128:(nb + 1) * 128].T
            s = np.float32(max(np.float32(np.abs(blk).max()) / np.float32(448), np.float32(2.0 ** -126)))
            assert p.w_scales[nb, g] == s
            v = torch.from_numpy((blk * (np.float32(1) / s)).astype(np.float64))
            got = torch.from_numpy(q[nb * 128:(nb + 1) * 128, g * 128:(g + 1) * 128][:, :blk.shape[1]])
            assert torch.equal((got - v).abs(), R.nearest_distance(v))


def test_weight_codes_round_ties_to_even():
    """Every midpoint of neighbouring e4m3 values goes to the even code; 448 fixes the scale at 1."""
    t = R.e4m3_values()
    pos = t[:127]
    mid = (pos[1:] + pos[:-1]) / 2
    W = np.zeros((128, 1), np.float32)
    W[:126, 0] = mid
    W[127, 0] = 448
    c = sq.prepare_weights_fp8(W).w_codes[0]
    lower = np.arange(126)
    assert np.array_equal(c[:126], np.where(lower % 2 == 0, lower, lower + 1))
    assert np.array_equal(sq.prepare_weights_fp8(-W).w_codes[0][:126], c[:126] | 0x80)


def test_weights_of_zero_infinity_and_nan():
    W = np.zeros((128, 3), np.float32)
    p = sq.prepare_weights_fp8(W)
    assert not p.w_codes.any() and p.w_scales[0, 0] == np.float32(2.0 ** -126)
    W[5, 1] = np.nan
    W[6, 1] = 1
    assert sq.prepare_weights_fp8(W).w_codes[1, 5] & 0x7F == 0x7F
    W[7, 2] = np.inf
    p = sq.prepare_weights_fp8(W)
    assert p.w_codes[2, 7] & 0x7F == 0x7F and np.isinf(p.w_scales[0, 0])


def test_document_ranges():
    r = sq.document_key_ranges([2, 0, 3], 7)
    assert r.shape == (1, 7, 2) and r.dtype == np.int32
    assert r[0].tolist() == [[0, 2], [0, 2], [2, 5], [2, 5], [2, 5], [0, 0], [0, 0]]
    assert sq.document_key_ranges([4]).tolist() == [[[0, 4]] * 4]
    with pytest.raises(ValueError):
        sq.document_key_ranges([5], 4)
    with pytest.raises(ValueError):
        sq.document_key_ranges([5, -1], 9)


M, K, N = 5, 200, 300


def norm_args(**over):
    a = dict(X=z(M, K), residual=z(M, K), gain=z(K, dtype=f32), eps=1e-6, a_codes=z(M, 256, dtype=u8),
             a_scales=z(M, 2, dtype=f32), residual_out=z(M, K))
    a.update(over)
    return a


def gemm_args(**over):
    a = dict(a_codes=z(M, 256, dtype=u8), a_scales=z(M, 2, dtype=f32), w_codes=z(N, 256, dtype=u8),
             w_scales=z(3, 2, dtype=f32), bias=z(N, dtype=f32), Y=z(M, N))
    a.update(over)
    return a


def attn_args(**over):
    a = dict(Q=z(2, 7, 4, 64), K=z(2, 9, 2, 64), V=z(2, 9, 2, 64), Out=z(2, 7, 4, 64))
    a.update(over)
    return a


def test_correct_cpu_arguments_stop_at_the_device_check():
    lin = dict(X=z(M, K), w_codes=z(N, 256, dtype=u8), w_scales=z(3, 2, dtype=f32), bias=None, Y=z(M, N),
               ws=z(max(1, sq.linear_fp8_workspace_bytes(M, K, N)), dtype=u8))
    for f, a in ((sq.rmsnorm_quantize_fp8, norm_args()), (sq.gemm_fp8, gemm_args()), (sq.attention, attn_args()),
                 (sq.linear_fp8, lin)):
        with pytest.raises(ValueError, match="GPU"):
            f(**a)


@pytest.mark.parametrize("over,match", [
    (dict(residual=z(M, K + 1)), "residual"), (dict(residual=z(M, K, dtype=bf16)), "residual"),
    (dict(gain=z(K - 1, dtype=f32)), "gain"), (dict(gain=z(K)), "gain"),
    (dict(a_codes=z(M, K, dtype=u8)), "a_codes"), (dict(a_scales=z(M, 1, dtype=f32)), "a_scales"),
    (dict(X=z(M, 2 * K)[:, ::2]), "inner stride"), (dict(X=z(M, K, dtype=torch.float64)), "X"),
    (dict(residual_out=z(M - 1, K)), "residual_out"), (dict(a_codes=None), "a_codes"),
])
def test_norm_refusals(over, match):
    with pytest.raises((ValueError, TypeError), match=match):
        sq.rmsnorm_quantize_fp8(**norm_args(**over))


@pytest.mark.parametrize("over,match", [
    (dict(a_codes=z(M, 192, dtype=u8)), "multiple of 128"), (dict(a_codes=z(M + 1, 256, dtype=u8)), "a_codes"),
    (dict(w_codes=z(N, 128, dtype=u8)), "w_codes"), (dict(w_scales=z(2, 2, dtype=f32)), "w_scales"),
    (dict(w_scales=z(3, 2)), "w_scales"), (dict(bias=z(N)), "bias"), (dict(Y=z(M, N, dtype=torch.float64)), "Y"),
    (dict(a_codes=z(M, 512, dtype=u8)[:, ::2]), "stride"), (dict(activation="relu"), "activation"),
])
def test_gemm_refusals(over, match):
    with pytest.raises((ValueError, TypeError), match=match if "activation" not in over else "activation|GPU"):
        sq.gemm_fp8(**gemm_args(**over))


@pytest.mark.parametrize("over,match", [
    (dict(Q=z(2, 7, 4, 64, dtype=f32)), "Q"), (dict(K=z(2, 9, 2, 64, dtype=bf16)), "K"),
    (dict(K=z(2, 9, 3, 64), V=z(2, 9, 3, 64)), "heads"), (dict(V=z(2, 8, 2, 64)), "V"),
    (dict(V=z(2, 9, 2, 72)), "V"), (dict(Out=z(2, 7, 2, 64)), "Out"), (dict(Q=z(7, 4, 64)), "Q"),
    (dict(Q=z(2, 7, 4, 128)[..., ::2]), "inner stride"), (dict(prefix=z(2, dtype=i32)), "prefix"),
    (dict(prefix=z(3, dtype=i32), causal=True), "prefix"), (dict(slopes=z(2, dtype=f32)), "slopes"),
    (dict(key_ranges=z(2, 7, dtype=i32)), "key_ranges"), (dict(key_ranges=z(3, 7, 2, dtype=i32)), "key_ranges"),
    (dict(key_ranges=z(2, 7, 2, dtype=torch.int64)), "key_ranges"),
])
def test_attention_refusals(over, match):
    with pytest.raises((ValueError, TypeError), match=match):
        sq.attention(**attn_args(**over))


def test_c_entry_points_refuse_on_the_host():
    """Each check comes before any HIP call: pointers that are never read."""
    p, lib = C.c_void_p(1 << 20), _lib.lib
    odd = C.c_void_p((1 << 20) + 1)
    norm = lambda X=p, dt=1, M=4, K=64, ldx=64, eps=1e-6, c=p, o=None, ldo=64, r=None, ldr=64: (  # noqa: E731
        lib.svdq_rmsnorm_quantize_fp8(X, r, dt, M, K, ldx, ldr, None, eps, c, p, o, ldo, None))
    assert norm(dt=7) == _lib.ERR_DTYPE
    assert norm(M=-1) == norm(K=0) == norm(ldx=63) == norm(eps=-1.0) == norm(eps=float("nan")) == _lib.ERR_SHAPE
    assert norm(X=None) == _lib.ERR_NULL and norm(c=None) == _lib.ERR_NULL
    assert norm(X=odd) == _lib.ERR_ALIGN and norm(c=C.c_void_p((1 << 20) + 8)) == _lib.ERR_ALIGN
    assert norm(o=p, ldo=65) == _lib.ERR_SHAPE and norm(r=p, ldr=10) == _lib.ERR_SHAPE
    assert norm(M=0, X=None, c=None) == _lib.OK

    gemm = lambda a=p, dt=1, M=4, N=8, Kp=128, ldy=8, act=0, ws=None, Y=p: (  # noqa: E731
        lib.svdq_gemm_fp8(a, p, p, p, None, Y, dt, M, N, Kp, ldy, act, ws, 0, None))
    assert gemm(dt=0) == _lib.ERR_DTYPE and gemm(act=5) == _lib.ERR_ACT and gemm(Kp=100) == _lib.ERR_GROUP
    assert gemm(N=0) == gemm(ldy=7) == gemm(M=-2) == gemm(Kp=1 << 23) == _lib.ERR_SHAPE
    assert gemm(a=None) == _lib.ERR_NULL and gemm(a=odd) == gemm(Y=odd) == gemm(ws=odd) == _lib.ERR_ALIGN
    assert gemm(M=0, a=None) == _lib.OK

    lin = lambda ws=p, n=1 << 20, K=64: lib.svdq_linear_fp8(  # noqa: E731
        p, 1, 64, p, p, None, p, 1, 8, 4, K, 8, ws, n, 0, None)
    assert lin(ws=None) == _lib.ERR_NULL and lin(n=4) == _lib.ERR_WORKSPACE and lin(K=0) == _lib.ERR_SHAPE
    assert lin(ws=C.c_void_p((1 << 20) + 16)) == _lib.ERR_ALIGN

    def attn(dt=1, B=1, Lq=2, Lk=3, Hq=2, Hkv=1, D=64, st=None, cap=0.0, causal=0, prefix=None, Q=p, ws=None, scale=1.0):
        s = [128 * Lq, 128, 64, 64 * Lk, 64, 64, 64 * Lk, 64, 64, 128 * Lq, 128, 64]
        for i, x in (st or {}).items():
            s[i] = x
        return lib.svdq_attention(Q, p, p, p, dt, B, Lq, Lk, Hq, Hkv, D, (C.c_int64 * 12)(*s), scale, cap, None, causal,
                                  prefix, None, 0, ws, 0, None)
    assert attn(dt=2) == _lib.ERR_DTYPE
    assert attn(B=-1) == attn(Hq=3, Hkv=2) == attn(D=12) == attn(D=136) == attn(Hkv=0) == attn(Lq=1 << 40) == _lib.ERR_SHAPE
    assert attn(cap=-1.0) == attn(cap=float("inf")) == attn(scale=float("nan")) == attn(prefix=p) == _lib.ERR_SHAPE
    assert attn(st={4: 4}) == attn(st={0: -8}) == attn(st={2: 12}) == _lib.ERR_ALIGN
    assert attn(st={4: 32}) == attn(st={7: 1 << 23}) == _lib.ERR_SHAPE
    assert attn(Q=None) == _lib.ERR_NULL and attn(Q=odd) == attn(ws=odd) == _lib.ERR_ALIGN
    assert attn(B=0, Q=None) == attn(Lq=0, Q=None) == _lib.OK
    assert "svdq_attention" in _lib.last_error() or _lib.last_error() == ""


def test_workspace_sizes():
    assert sq.gemm_fp8_workspace_bytes(0, 5, 128) == sq.gemm_fp8_workspace_bytes(5, 5, 100) == 0
    assert sq.linear_fp8_workspace_bytes(3, 200, 10) >= 3 * 256 + 3 * 2 * 4
    assert sq.attention_workspace_bytes(1, 1, 4000, 3, 2, 64) == 0
    assert sq.attention_workspace_bytes(0, 1, 4000, 2, 2, 64) == 0
