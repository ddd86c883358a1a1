"""The bounds of an 8-bit cache's scales and of the scores' scale beside them, without a GPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import bit_post_quantized_smooth_amd as sq
from test_paged_messages import SHAPE, at, attend, refused


@pytest.mark.parametrize("name", ["k_scales", "v_scales"])
@pytest.mark.parametrize("bad", [2.0 ** -65, 1e-36, 1e-45, 2.0 ** 65, 3e38])
def test_cache_refuses_scales_out_of_range(name, bad):
    """Below: slope / (scale * k_scale) and the reciprocals that codes are made with leave fp32."""
    t = sq.PageTable(2, 64, device="cpu")
    with pytest.raises(ValueError, match=name):
        sq.PagedKeyValueCache(t, 2, 32, torch.float8_e4m3fn, **{name: [1.0, bad]})


def test_cache_takes_the_bounds():
    t = sq.PageTable(2, 64, device="cpu")
    c = sq.PagedKeyValueCache(t, 2, 32, torch.float8_e4m3fn, [2.0 ** -64, 2.0 ** 64], [2.0 ** 64, 2.0 ** -64])
    assert c.k_scales.tolist() == [2.0 ** -64, 2.0 ** 64] and c.v_scales.tolist() == [2.0 ** 64, 2.0 ** -64]


@pytest.mark.parametrize("scale,over", [(2.0 ** -41, dict(ks=at(9))), (-1e-30, dict(ks=at(9))), (1e-45, dict(ks=at(9))),
                                        (2.0 ** -41, dict(sl=at(9))), (2.0 ** -41, dict(sl=at(9), ks=at(10)))])
def test_attention_refuses_a_scale_that_leaves_fp32(scale, over):
    """Times a key scale of 2^-64 it would underflow, and a masked score become -inf * 0."""
    refused(attend(scale=scale, over=over), SHAPE, "2^-40")


@pytest.mark.parametrize("scale", [2.0 ** 61, -3e38])
def test_attention_refuses_a_scale_above(scale):
    refused(attend(scale=scale, over=dict(ks=at(9))), SHAPE, "2^60")


def test_the_bounds_hold_in_fp32():
    """The smallest and the largest products that are let through, and the slopes and codes made
    with them."""
    f = np.float32
    log2e = f(1.4426950408889634)
    small, large = f(2.0 ** -40) * log2e * f(2.0 ** -64), f(2.0 ** 60) * log2e * f(2.0 ** 64)
    assert small >= f(2.0 ** -126) and np.isfinite(large)
    assert np.isfinite(f(2.0 ** 20) * log2e / small)
    assert np.isfinite(f(1) / f(2.0 ** -64)) and f(1) / f(2.0 ** 64) >= f(2.0 ** -126)
