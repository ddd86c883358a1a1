"""Products and attentions of more rows than a launch's 2^32 threads cover are refused
on the host, where a launch of more would run a part of them and report nothing, and
so are outputs that overlap themselves."""
import ctypes as C

import pytest

sq = pytest.importorskip("bit_post_quantized_smooth_amd")
from bit_post_quantized_smooth_amd import _lib  # noqa: E402

P = C.c_void_p(1 << 20)                                # never read


def gemm(M, N, dt=1):
    # sizes are checked before pointers: a null pointer says that the sizes passed
    return _lib.lib.svdq_gemm_fp8(None, P, P, P, None, P, dt, M, N, 128, N, 0, None, 0, None)


def attention(B, Hkv, Lq=1, G=1):
    s = [8 * G * Hkv * Lq, 8 * G * Hkv, 8, 8 * Hkv, 8 * Hkv, 8, 8 * Hkv, 8 * Hkv, 8, 8 * G * Hkv * Lq, 8 * G * Hkv, 8]
    return _lib.lib.svdq_attention(None, P, P, P, 1, B, Lq, 1, G * Hkv, Hkv, 8, (C.c_int64 * 12)(*s), 1.0, 0.0, None, 0,
                                   None, None, 0, None, 0, None)


@pytest.mark.parametrize("dt", [1, 2, 3])
def test_product(dt):
    # 16 columns a workgroup of 512 threads, up to 16 rows
    assert gemm(1, (1 << 27) - 16, dt) == _lib.ERR_NULL
    assert gemm(16, 1 << 27, dt) == gemm(1, (1 << 31) - 1, dt) == _lib.ERR_SHAPE
    assert gemm(1 << 16, 1 << 16, dt) == _lib.ERR_NULL


def test_attention():
    # a workgroup of 256 threads for each key head of a sequence, at least
    assert attention(1 << 20, 15) == _lib.ERR_NULL
    assert attention(1 << 20, 16) == attention(1 << 24, 4, 1, 8) == _lib.ERR_SHAPE
    assert "rows" in _lib.last_error()
    assert attention(1 << 16, 8, 32) == _lib.ERR_NULL


def test_workspace_of_what_is_refused():
    assert sq.attention_workspace_bytes(1 << 20, 1, 1, 16, 16, 8) == 0


def test_attention_output_over_itself():
    """Rows written to one place by several workgroups would hold any one of them."""
    def out(B, L, H, D, *strides):
        s = [H * L * D, H * D, D] * 3 + list(strides)
        return _lib.lib.svdq_attention(None, P, P, P, 1, B, L, L, H, H, D, (C.c_int64 * 12)(*s), 1.0, 0.0, None, 0, None,
                                       None, 0, None, 0, None)
    good = [(2, 5, 3, 16, 240, 48, 16), (2, 5, 3, 16, 240, 16, 80), (2, 5, 3, 16, 48, 96, 16), (1, 5, 3, 16, 0, 48, 16),
            (2, 1, 3, 16, 48, 0, 16), (2, 5, 1, 16, 80, 16, 0), (3, 5, 2, 8, 1000, 64, 24)]
    bad = [(2, 5, 3, 16, 0, 48, 16), (2, 5, 3, 16, 240, 0, 16), (2, 5, 3, 16, 240, 48, 0), (2, 5, 3, 16, 240, 48, 8),
           (2, 5, 3, 16, 232, 48, 16), (2, 5, 3, 16, 240, 40, 16)]
    assert [out(*g) for g in good] == [_lib.ERR_NULL] * len(good)
    assert [out(*b) for b in bad] == [_lib.ERR_SHAPE] * len(bad)
