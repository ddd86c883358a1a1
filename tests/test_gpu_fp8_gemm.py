"""The e4m3 product with block scales, and the 8-bit linear, against fp64."""
import numpy as np
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


def operands(M, N, Kp, seed=0):
    """Random finite codes, scales over three orders of magnitude, a bias."""
    g = torch.Generator().manual_seed(seed)
    def codes(r):
        c = torch.randint(0, 127, (r, Kp), generator=g, dtype=torch.uint8)
        return c | (torch.randint(0, 2, (r, Kp), generator=g, dtype=torch.uint8) << 7)
    G = Kp // 128
    sa = torch.exp(torch.randn(M, G, generator=g)) * 1e-2
    sw = torch.exp(torch.randn(-(-N // 128), G, generator=g)) * 1e-3
    return codes(M).cuda(), sa.cuda(), codes(N).cuda(), sw.cuda(), torch.randn(N, generator=g).cuda()


def check(sq, M, N, Kp, dtype, bias=True, act=None, ws=True, seed=0, ldy=None):
    a, sa, w, sw, b = operands(M, N, Kp, seed)
    b = b if bias else None
    full = torch.full((M, ldy or N), 7.0, device="cuda", dtype=dtype)
    Y = full[:, :N]
    need = sq.gemm_fp8_workspace_bytes(M, N, Kp)
    work = torch.full((need // 4,), float("nan"), device="cuda") if ws and need else None
    sq.gemm_fp8(a, sa, w, sw, b, Y, ws=work, activation=act)
    y, env, peak = R.gemm(a, sa, w, sw, b, act is not None)
    R.assert_within(Y, y, R.gemm_bound(y, env, peak, Kp, dtype))
    assert bool((full[:, N:] == 7.0).all())
    return Y


DTYPES = [torch.float16, torch.bfloat16, torch.float32]
SIZES = [  # few rows, each count of row blocks; tiles with ragged edges; one and many groups
    (1, 16, 128), (1, 1, 128), (3, 130, 384), (16, 48, 1280), (17, 129, 640), (33, 257, 256),
    (64, 100, 2176), (65, 64, 128), (100, 300, 1152), (129, 193, 640), (200, 65, 3200),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,Kp", SIZES)
def test_sizes(sq, M, N, Kp, dtype):
    check(sq, M, N, Kp, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,Kp", [(2048, 2304, 256), (2049, 2303, 640), (4100, 1030, 128)])
def test_large_tiles(sq, M, N, Kp, dtype):
    check(sq, M, N, Kp, dtype, bias=False)


@pytest.mark.parametrize("dtype", DTYPES)
def test_activation_and_row_stride(sq, dtype):
    for M, N, ldy in ((5, 70, 77), (150, 130, 131), (150, 128, 136), (2050, 2050, 2053)):
        check(sq, M, N, 256, dtype, act="gelu_tanh", ldy=ldy)


def test_with_and_without_a_workspace(sq):
    """The product split along K and the unsplit one, each within the bound."""
    M, N, Kp = 128, 256, 12288
    assert sq.gemm_fp8_workspace_bytes(M, N, Kp) > 0
    for dtype in DTYPES:
        check(sq, M, N, Kp, dtype, ws=True)
        check(sq, M, N, Kp, dtype, ws=False)


def test_repeats_bit_for_bit(sq):
    for M, N, Kp in ((7, 300, 2048), (128, 256, 12288), (2048, 2304, 384)):
        y = check(sq, M, N, Kp, torch.float16)
        assert torch.equal(y, check(sq, M, N, Kp, torch.float16))


def test_unaligned_scales_and_output(sq):
    """Scales, bias and Y at addresses aligned to their elements only."""
    M, N, Kp = 70, 90, 384
    a, sa, w, sw, b = operands(M, N, Kp)
    def shift(t):
        u = torch.empty(t.numel() + 1, device="cuda", dtype=t.dtype)[1:]
        u.copy_(t.flatten())
        return u.view(t.shape)
    for rows in (70, 9):
        for dtype in DTYPES:
            Y = torch.empty(rows * N + 1, device="cuda", dtype=dtype)[1:].view(rows, N)
            sq.gemm_fp8(a[:rows], shift(sa[:rows].contiguous()), w, shift(sw), shift(b), Y)
            y, env, peak = R.gemm(a[:rows], sa[:rows], w, sw, b, False)
            R.assert_within(Y, y, R.gemm_bound(y, env, peak, Kp, dtype))


def test_nan_codes_stay_in_their_row_and_column(sq):
    for M, N in ((5, 40), (130, 140)):
        a, sa, w, sw, b = operands(M, N, 256)
        a[2, 17] = 0x7F
        w[30, 200] = 0xFF
        Y = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
        sq.gemm_fp8(a, sa, w, sw, b, Y)
        bad = torch.isnan(Y.cpu())
        want = torch.zeros(M, N, dtype=torch.bool)
        want[2] = True
        want[:, 30] = True
        assert torch.equal(bad, want)


def test_no_rows(sq):
    a, sa, w, sw, b = operands(0, 40, 256)
    sq.gemm_fp8(a, sa, w, sw, b, torch.empty(0, 40, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", [(1, 640, 320), (77, 1001, 515), (300, 320, 1280)])
def test_linear(sq, M, K, N, dtype):
    """prepare_weights_fp8 -> Linear: the product of the codes its own quantizer gives."""
    rng = np.random.default_rng(M)
    W = (rng.standard_normal((K, N)) * 0.02).astype(np.float32)
    W[K // 2] *= 10
    bias = rng.standard_normal(N).astype(np.float32)
    p = sq.prepare_weights_fp8(W)
    X = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(dtype).cuda()
    lin = sq.Linear(p, bias, out_dtype=dtype)
    Y = lin(X)
    c = torch.empty(M, R.padded(K), dtype=torch.uint8, device="cuda")
    s = torch.empty(M, R.padded(K) // 128, device="cuda")
    sq.quantize_act_fp8(X, c, s)
    wc, ws = torch.from_numpy(p.w_codes), torch.from_numpy(p.w_scales)
    y, env, peak = R.gemm(c, s, wc, ws, torch.from_numpy(bias), False)
    R.assert_within(Y, y, R.gemm_bound(y, env, peak, R.padded(K), dtype))
    # and near the unquantized product: 8-bit operands keep 2^-4 per term, at random
    ref = X.cpu().double() @ torch.from_numpy(W).double() + torch.from_numpy(bias).double()
    assert float((Y.cpu().double() - ref).norm() / ref.norm()) < 0.05
