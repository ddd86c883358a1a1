"""The e4m3 product split along K: its second kernel adds the slices' sums and applies
what the tiles apply otherwise, the bias, the GELU, the rounding and the rows' stride
and alignment."""
import pytest
import torch

import block_ref as R
from test_gpu_fp8_gemm import DTYPES, check, operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


SPLIT = [(40, 640, 12288), (17, 67, 8448), (128, 256, 12288)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,Kp", SPLIT)
@pytest.mark.parametrize("act", [None, "gelu_tanh"])
def test_activation_and_row_stride(sq, M, N, Kp, dtype, act):
    assert sq.gemm_fp8_workspace_bytes(M, N, Kp) >= 2 * M * N * 4          # two slices or more
    for ldy, bias in ((N, True), (N + 1, True), (N + 8, False), (N + 5, True)):
        check(sq, M, N, Kp, dtype, bias=bias, act=act, ldy=ldy)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,Kp", SPLIT)
def test_output_at_any_address(sq, M, N, Kp, dtype):
    a, sa, w, sw, b = operands(M, N, Kp)
    y, env, peak = R.gemm(a, sa, w, sw, b, True)
    ws = torch.full((sq.gemm_fp8_workspace_bytes(M, N, Kp) // 4,), float("nan"), device="cuda")
    for off in (1, 2, 3):
        flat = torch.full((M * N + off + 8,), 7.0, device="cuda", dtype=dtype)
        Y = flat[off:off + M * N].view(M, N)
        sq.gemm_fp8(a, sa, w, sw, b, Y, ws=ws, activation="gelu_tanh")
        R.assert_within(Y, y, R.gemm_bound(y, env, peak, Kp, dtype))
        assert bool((flat[:off] == 7.0).all()) and bool((flat[off + M * N:] == 7.0).all())
