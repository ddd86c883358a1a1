"""Residual + RMS norm + e4m3 quantization, and the quantizer alone, against the
fp64 formulas."""
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


def inputs(M, K, dtype, seed=0, ld=None):
    """M x K values with outlier channels, as a view of rows of `ld` elements."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, ld or K, generator=g)
    x[:, :max(1, K // 100)] *= 20
    return x.to(dtype).cuda()[:, :K]


def buffers(M, K):
    Kp = R.padded(K)
    return (torch.full((M, Kp), 0x55, dtype=torch.uint8, device="cuda"),
            torch.full((M, Kp // 128), float("nan"), device="cuda"))


def sum_error(K):
    """Relative error of u: the row sum of squares (each thread adds its run of the
    row, then log2 steps), the mean, square root, division and two products."""
    return (K / 64 + 24) * 2.0 ** -24


DTYPES = [torch.float16, torch.bfloat16, torch.float32]
# each register path of the kernel, its edges, odd widths and a row longer than registers hold
WIDTHS = [1, 7, 128, 129, 320, 512, 513, 1001, 1024, 1280, 2048, 2049, 4096, 5000, 8192, 16384, 16385]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", WIDTHS)
def test_norm(sq, K, dtype):
    for M, res, gain in ((1, False, True), (3, True, True), (130, True, False)):
        x = inputs(M, K, dtype)
        r = inputs(M, K, dtype, 1) if res else None
        gn = (1 + 0.2 * torch.randn(K, generator=torch.Generator().manual_seed(2))).cuda() if gain else None
        c, s = buffers(M, K)
        out = torch.empty_like(x) if res else None
        sq.rmsnorm_quantize_fp8(x, r, gn, 1e-6, c, s, out)
        h, u = R.norm(x.cpu(), r.cpu() if res else None, gn.cpu() if gain else None, 1e-6)
        R.check_quantized(c, s, u, sum_error(K))
        if res:
            assert torch.equal(out.cpu(), (x.cpu().float() + r.cpu().float()).to(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [1, 130, 640, 3000, 20000])
def test_quantizer_alone(sq, K, dtype):
    x = inputs(37, K, dtype)
    c, s = buffers(37, K)
    sq.quantize_act_fp8(x, c, s)
    R.check_quantized(c, s, x.cpu().to(torch.float64), 2.0 ** -23)


@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_and_in_place(sq, dtype):
    """Rows at odd strides, and residual_out on X and on residual themselves."""
    M, K = 19, 777
    x, r = inputs(M, K, dtype, 3, 1001), inputs(M, K, dtype, 4, 779)
    h, u = R.norm(x.cpu(), r.cpu(), None, 1e-5)
    want = (x.cpu().float() + r.cpu().float()).to(dtype)
    for target in (x, r):
        xi, ri = x.clone(), r.clone()
        xi, ri = (t if t.stride(0) > K else t for t in (xi, ri))
        out = xi if target is x else ri
        c, s = buffers(M, K)
        sq.rmsnorm_quantize_fp8(xi, ri, None, 1e-5, c, s, out)
        R.check_quantized(c, s, u, sum_error(K))
        assert torch.equal(out.cpu(), want)
    c, s = buffers(M, K)
    out = inputs(M, K, dtype, 5, 783)
    beyond = out.as_strided((M, 783), (783, 1))[:, K:].clone()
    sq.rmsnorm_quantize_fp8(x, r, None, 1e-5, c, s, out)
    R.check_quantized(c, s, u, sum_error(K))
    assert torch.equal(out.cpu(), want)
    assert torch.equal(out.as_strided((M, 783), (783, 1))[:, K:], beyond)   # nothing past K


def test_zeros_infinities_and_nan(sq):
    M, K = 5, 300
    x = torch.zeros(M, K)
    x[1] = 1.0
    x[2] = 1.0
    x[2, 200] = float("inf")
    x[3] = 1.0
    x[3, 10] = float("nan")
    x[4, 7] = 1e-38                     # a group whose scale would be subnormal
    c, s = buffers(M, K)
    sq.quantize_act_fp8(x.cuda(), c, s)
    v, s = R.decode(c), s.cpu()
    assert bool((v[0] == 0).all()) and bool((s[0] == 2.0 ** -126).all())
    assert bool((v[1, :K] == 448).all()) and bool((v[1, K:] == 0).all())
    assert torch.isnan(v[2, 200]) and bool((v[2, 128:200] == 0).all()) and s[2, 1] == float("inf")
    assert bool((v[2, :128] == 448).all())
    assert torch.isnan(v[3, 10]) and bool((v[3, :10] == 448).all()) and s[3, 0] == 1 / 448
    assert s[4, 0] == 2.0 ** -126 and v[4, 7] != 0
    # through the norm a NaN or an infinity spoils its row, and only its row
    c, s = buffers(M, K)
    sq.rmsnorm_quantize_fp8(x.cuda(), None, None, 1e-6, c, s)
    v = R.decode(c)
    assert bool(torch.isnan(v[3, :K]).all()) and torch.isnan(v[2, 200])
    assert bool((v[1, :K] == 448).all()) and bool((v[0] == 0).all())


def test_no_rows(sq):
    x = torch.empty(0, 64, device="cuda")
    c, s = buffers(0, 64)
    sq.rmsnorm_quantize_fp8(x, x, None, 1e-6, c, s, x)
    sq.quantize_act_fp8(x, c, s)


def test_other_stream_and_repeat(sq):
    """Enqueued on the given stream, and the same bits every time."""
    x = inputs(300, 1280, torch.bfloat16)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):
        with torch.cuda.stream(st):
            c, s = buffers(300, 1280)
            sq.rmsnorm_quantize_fp8(x, None, None, 1e-6, c, s, stream=st)
        st.synchronize()
        got.append((c, s))
    for c, s in got[1:]:
        assert torch.equal(c, got[0][0]) and torch.equal(s, got[0][1])
