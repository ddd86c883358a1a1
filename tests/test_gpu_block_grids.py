"""More rows than one launch's 2^32 threads cover: the quantizer takes them in several
launches; the product and the attention, whose inputs would have to be that long too,
refuse them (tests/test_block_grids.py)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


# a workgroup of 256 threads takes one row of fewer than 8 channels, four of 8
@pytest.mark.parametrize("M,K", [((1 << 24) + 5, 1), ((1 << 26) + 5, 8)])
def test_rows_beyond_one_launch(sq, M, K):
    x = torch.ones(M, K, device="cuda", dtype=torch.float16)
    r = torch.ones(M, K, device="cuda", dtype=torch.float16)
    x[-1], r[-2] = 3.0, 2.0
    out = torch.zeros_like(x)
    c = torch.full((M, 128), 0x55, device="cuda", dtype=torch.uint8)
    s = torch.zeros(M, 1, device="cuda")
    sq.quantize_act_fp8(x, c, s)
    assert bool((c[:, :K] == 126).all()) and bool((c[:, K:] == 0).all())     # 448, the largest
    assert float(s[-1]) == float(torch.tensor(3.0) / 448) and bool((s[:-1] == s[0]).all())
    sq.rmsnorm_quantize_fp8(x, r, None, 0.0, c.fill_(0x55), s.zero_(), out)
    assert bool((c[:, :K] == 126).all()) and bool((c[:, K:] == 0).all())
    assert bool(((s * 448 - 1).abs() < 1e-6).all())                          # the norm of equal values is 1
    assert out[-1].tolist() == [4.0] * K and out[-2].tolist() == [3.0] * K
    assert bool((out[:-2] == 2.0).all())
