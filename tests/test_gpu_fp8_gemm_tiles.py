"""The e4m3 product at sizes that take each of its tile shapes, split and unsplit,
and more groups than one load of the weight scales brings (64). A sample of rows
against fp64: the first, the last, every tile edge's neighbours and some between."""
import pytest
import torch

import block_ref as R
from test_gpu_fp8_gemm import operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


def check(sq, M, N, Kp, dtype, ws=True):
    a, sa, w, sw, b = operands(M, N, Kp)
    Y = torch.full((M, N), float("nan"), device="cuda", dtype=dtype)
    need = sq.gemm_fp8_workspace_bytes(M, N, Kp)
    work = torch.full((need // 4,), float("nan"), device="cuda") if ws and need else None
    sq.gemm_fp8(a, sa, w, sw, b, Y, ws=work)
    assert not bool(torch.isnan(Y).any())
    edges = {r for e in range(0, M + 64, 64) for r in (e - 1, e) if 0 <= r < M}
    rows = torch.tensor(sorted((edges if M < 400 else {r for r in edges if r < 320 or r > M - 70})
                               | {M - 1} | set(range(7, M, M // 7 + 1))))
    y, env, peak = R.gemm(a[rows.cuda()], sa[rows.cuda()], w, sw, b, False)
    R.assert_within(Y[rows.cuda()], y, R.gemm_bound(y, env, peak, Kp, dtype))


# 256 x 256, 256 x 192, 128 x 128, 64 x 128 and 64 x 64 tiles
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,N,Kp", [
    (2500, 5120, 128), (2304, 6000, 384), (2500, 5127, 640), (4100, 2048, 128), (2304, 3840, 256),
    (2305, 3840, 640), (1000, 6000, 128), (1023, 6001, 1280), (1000, 6000, 8448), (2048, 1030, 256),
    (600, 3840, 640), (2048, 2304, 8448), (17, 64, 8448), (40, 130, 12288), (65, 640, 8320)])
def test_16_bits(sq, M, N, Kp, dtype):
    check(sq, M, N, Kp, dtype, ws=False)


# 256 x 128, 64 x 128 and 64 x 64 tiles
@pytest.mark.parametrize("M,N,Kp", [
    (2500, 2500, 128), (2048, 3840, 640), (2500, 2501, 8448), (2048, 1030, 384), (600, 3840, 8448),
    (17, 64, 8448), (200, 130, 12288)])
def test_32_bits(sq, M, N, Kp):
    check(sq, M, N, Kp, torch.float32, ws=False)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("M,N,Kp", [
    (2048, 1030, 12288), (600, 3840, 12288), (17, 64, 3072), (17, 67, 8448), (65, 5120, 12288),
    (40, 640, 12288), (200, 1283, 12288)])
def test_split(sq, M, N, Kp, dtype):
    assert sq.gemm_fp8_workspace_bytes(M, N, Kp) > 0
    check(sq, M, N, Kp, dtype)


def test_a_short_workspace_runs_unsplit(sq):
    M, N, Kp = 40, 640, 12288
    a, sa, w, sw, b = operands(M, N, Kp)
    ys = []
    for size in (0, 64, sq.gemm_fp8_workspace_bytes(M, N, Kp)):
        Y = torch.empty(M, N, device="cuda", dtype=torch.float16)
        ws = torch.full((size + 64,), 0x5A, device="cuda", dtype=torch.uint8)
        sq.gemm_fp8(a, sa, w, sw, b, Y, ws=ws[:size])
        assert bool((ws[size:] == 0x5A).all())
        ys.append(Y)
    y, env, peak = R.gemm(a, sa, w, sw, b, False)
    assert torch.equal(ys[0], ys[1])
    for Y in ys:
        R.assert_within(Y, y, R.gemm_bound(y, env, peak, Kp, torch.float16))
