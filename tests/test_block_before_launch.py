"""What AttentionBlock refuses, it refuses before anything is launched."""
import numpy as np
import pytest
import torch

import bit_post_quantized_smooth_amd as sq
from bit_post_quantized_smooth_amd import block as module
from test_block_class import weights

F16, BF16, I32, E4M3 = torch.float16, torch.bfloat16, torch.int32, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    def launched(*a, **k):
        raise AssertionError("launched")
    for f in ("rmsnorm_quantize_fp8", "gemm_fp8", "quantize_act_fp8", "attention"):
        monkeypatch.setattr(module.api, f, launched)
    for f in ("norm_rotary", "norm_rotary_write", "paged_write", "paged_attention"):
        monkeypatch.setattr(module.paged, f, launched)


def make(**kw):
    return sq.AttentionBlock(np.ones(256, np.float32), *weights(), 4, 2, 32, device="cpu", **kw)


X = torch.zeros(2, 3, 256, dtype=F16)


def test_a_good_call_launches():
    block = make(rotary=sq.rotary_frequencies(32))
    table = sq.PageTable(2, 64, device="cpu")
    table.begin([3, 3])
    for kw in (dict(), dict(positions=torch.zeros(2, 3, dtype=I32)), dict(positions=torch.zeros(2, 6, dtype=I32)[:, ::2]),
               dict(cache=sq.PagedKeyValueCache(table, 2, 32, F16)), dict(cache=sq.PagedKeyValueCache(table, 2, 32, E4M3))):
        with pytest.raises(AssertionError, match="launched"):
            block(X, **kw)


@pytest.mark.parametrize("positions", [torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3), torch.zeros(2, 2, dtype=I32),
                                       torch.zeros(6, dtype=I32), torch.zeros(2, 3, dtype=I32, device="meta")],
                         ids=["int64", "float", "shape", "flat", "device"])
def test_positions(positions):
    with pytest.raises(ValueError, match="positions"):
        make(rotary=sq.rotary_frequencies(32))(X, positions=positions)


@pytest.mark.parametrize("eps", [1e-40, 1.1e-38, -1e-6, float("nan"), float("inf")])
def test_eps_of_the_heads_norm(eps):
    """Fixed when the block is made, and refused there."""
    gains = (np.ones(32, np.float32), np.ones(32, np.float32))
    with pytest.raises(ValueError, match="eps"):
        make(head_gains=gains, eps=eps)


def test_eps_that_the_heads_norm_takes():
    gains = (np.ones(32, np.float32), None)
    for eps in (0.0, 2.0 ** -126, 1e-6):
        assert make(head_gains=gains, eps=eps).turn["eps"] == eps
    assert make(eps=1e-40).turn is None                    # no norm of heads


@pytest.mark.parametrize("cache,match", [
    (lambda t: sq.PagedKeyValueCache(t, 2, 32, BF16), "bfloat16"), (lambda t: sq.PagedKeyValueCache(t, 4, 32, F16), "heads"),
    (lambda t: sq.PagedKeyValueCache(t, 2, 64, F16), "heads"), (lambda t: sq.PagedKeyValueCache(t, 1, 32, E4M3), "heads")])
def test_a_paged_cache_of_another_layer(cache, match):
    table = sq.PageTable(2, 64, device="cpu")
    table.begin([3, 3])
    with pytest.raises(ValueError, match=match):
        make()(X, cache=cache(table))


def test_a_paged_cache_on_another_device():
    table = sq.PageTable(2, 64, device="cpu")
    table.begin([3, 3])
    cache = sq.PagedKeyValueCache(table, 2, 32, F16)
    cache.k = cache.k.to("meta")
    with pytest.raises(ValueError, match="meta"):
        make()(X, cache=cache)
