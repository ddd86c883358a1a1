"""The attention block's refusals, and its cache, without a GPU."""
import dataclasses

import numpy as np
import pytest
import torch

import bit_post_quantized_smooth_amd as sq
from bit_post_quantized_smooth_amd import block as block_module


def weights(K=256, Hq=4, Hkv=2, D=32):
    rng = np.random.default_rng(0)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)
    return sq.prepare_weights_fp8(f(K, (Hq + 2 * Hkv) * D)), sq.prepare_weights_fp8(f(Hq * D, K))


def test_weights_that_do_not_fit():
    qkv, out = weights()
    gain = np.ones(256, np.float32)
    with pytest.raises(ValueError, match="do not fit"):
        sq.AttentionBlock(gain, qkv, out, 4, 4, 32, device="cpu")
    with pytest.raises(ValueError, match="do not fit"):
        sq.AttentionBlock(gain, out, qkv, 4, 2, 32, device="cpu")
    with pytest.raises(ValueError, match="prepare_weights_fp8"):
        sq.AttentionBlock(gain, sq.prepare_weights(np.ones((256, 256), np.float32), np.ones(256, np.float32), 0),
                          out, 4, 2, 32, device="cpu")


def test_inputs_that_do_not_fit():
    block = sq.AttentionBlock(np.ones(256, np.float32), *weights(), 4, 2, 32, device="cpu")
    X = torch.zeros(2, 3, 256, dtype=torch.float16)
    for bad, match in ((X[0], "shape"), (X[..., :128], "shape"), (X.float(), "dtype")):
        with pytest.raises(ValueError, match=match):
            block(bad)
    with pytest.raises(TypeError):
        block(X.numpy())
    with pytest.raises(ValueError, match="residual"):
        block(X, X[:1])
    with pytest.raises(ValueError, match="dtype"):
        block(X, X.bfloat16())
    with pytest.raises(ValueError, match="on a GPU"):
        block(X)


def test_cache():
    c = sq.KeyValueCache(2, 10, 3, 8, torch.float16, device="cpu")
    a = torch.arange(2 * 4 * 3 * 8, dtype=torch.float16).view(2, 4, 3, 8)
    k, v = c.append(a, -a)
    assert torch.equal(k, a) and torch.equal(v, -a) and c.length == 4
    k, v = c.append(a + 1, a)
    assert k.shape[1] == 8 and torch.equal(k[:, 4:], a + 1) and torch.equal(v[:, :4], -a)
    with pytest.raises(ValueError, match="cache of 10"):
        c.append(a, a)
    assert c.length == 8


def test_cache_refuses_what_does_not_fit():
    """A batch of one is not spread over the sequences, another type is not converted:
    what is held stays as it was."""
    c = sq.KeyValueCache(2, 10, 3, 8, torch.float16, device="cpu")
    a = torch.ones(2, 4, 3, 8, dtype=torch.float16)
    c.append(a, a)
    held = c.k.clone(), c.v.clone()
    for k, v in ((a[:1], a[:1]), (a, a[:, :1]), (a[:, :, :1], a), (a, a[..., :1]), (a[0], a[0]),
                 (a.float(), a.float()), (a, a.bfloat16()), (a.to("meta"), a)):
        with pytest.raises(ValueError, match="k: |v: "):
            c.append(k, v)
    with pytest.raises(TypeError):
        c.append(a.numpy(), a)
    assert c.length == 4 and torch.equal(c.k[:, :4], held[0][:, :4]) and torch.equal(c.v[:, :4], held[1][:, :4])


def test_a_refused_call_leaves_the_cache_as_it_was(monkeypatch):
    """Attention's refusals come behind the append: the length goes back."""
    block = sq.AttentionBlock(np.ones(256, np.float32), *weights(), 4, 2, 32, device="cpu")
    for f in ("rmsnorm_quantize_fp8", "gemm_fp8", "quantize_act_fp8"):
        monkeypatch.setattr(block_module.api, f, lambda *a, **k: None)
    X = torch.zeros(2, 3, 256, dtype=torch.float16)
    cache = sq.KeyValueCache(2, 10, 2, 32, torch.float16, device="cpu")
    for kw, match in ((dict(causal=False, prefix=torch.zeros(2, dtype=torch.int32)), "prefix"),
                      (dict(key_ranges=torch.zeros(3, 3, 2, dtype=torch.int32)), "key_ranges"),
                      (dict(), "on a GPU")):
        with pytest.raises(ValueError, match=match):
            block(X, cache=cache, **kw)
        assert cache.length == 0


def test_a_low_rank_branch_is_not_dropped():
    """concat_lora on an 8-bit prep gives a branch that no 8-bit layer applies."""
    qkv, out = weights()
    rng = np.random.default_rng(1)
    A, B = rng.standard_normal((256, 16)), rng.standard_normal((16, 256))
    lora = sq.concat_lora(sq.prepare_weights_fp8(np.ones((256, 256), np.float32)), np.ones(256), A, B)
    assert lora.rank == 16
    with pytest.raises(ValueError, match="low-rank"):
        sq.Linear(lora, device="cpu")
    both = dict(rank=16, L1t=np.zeros((16, 256), np.uint16), L2t=np.zeros((256, 16), np.uint16))
    for a, b in ((dataclasses.replace(qkv, **both), out), (qkv, dataclasses.replace(out, **both))):
        with pytest.raises(ValueError, match="low-rank"):
            sq.AttentionBlock(np.ones(256, np.float32), a, b, 4, 2, 32, device="cpu")


@pytest.mark.parametrize("heads,kv_heads,D", [(3, 2, 32), (4, 2, 20), (4, 2, 136), (0, 2, 32), (4, 0, 32), (4, -2, 32)])
def test_heads_that_attention_does_not_take(heads, kv_heads, D):
    """Refused when the block is made, not when its first call has done half its work."""
    n = max(heads + 2 * kv_heads, 1) * D
    f = lambda *s: np.ones(s, np.float32)  # noqa: E731
    with pytest.raises(ValueError):
        sq.AttentionBlock(f(256), sq.prepare_weights_fp8(f(256, n)), sq.prepare_weights_fp8(f(max(heads, 1) * D, 256)),
                          heads, kv_heads, D, device="cpu")


@pytest.mark.parametrize("over", [dict(gain=255), dict(qkv_bias=255), dict(out_bias=1), dict(slopes=2)])
def test_vectors_of_another_length(over):
    a = dict(gain=np.ones(256, np.float32))
    a.update({k: np.ones(n, np.float32) for k, n in over.items()})
    qkv, out = weights()
    with pytest.raises(ValueError, match=next(iter(over))):
        sq.AttentionBlock(qkv=qkv, out=out, heads=4, kv_heads=2, head_dim=32, device="cpu", **a)


def test_buffers_of_smaller_calls_outlive_larger_ones(monkeypatch):
    """A graph's replays write to the buffers of its capture: a later, larger call may
    not give them back. All that are outgrown take no more than those in use."""
    for f in ("rmsnorm_quantize_fp8", "gemm_fp8", "quantize_act_fp8", "attention", "linear_fp8"):
        monkeypatch.setattr(block_module.api, f, lambda *a, **k: None)
    block = sq.AttentionBlock(np.ones(256, np.float32), *weights(), 4, 2, 32, device="cpu")
    lin = sq.Linear(sq.prepare_weights_fp8(np.ones((256, 256), np.float32)), device="cpu")
    for thing, rank in ((block, 3), (lin, 2)):
        b, addresses = thing._buffers, set()
        for n in (8, 9, 10, 64, 100, 101, 1000):
            thing(torch.zeros((1, n, 256)[3 - rank:], dtype=torch.float16))
            addresses |= {t.data_ptr() for t in b.kept.values()}
        assert addresses == {t.data_ptr() for t in (*b.kept.values(), *b.outgrown)}
        assert sum(t.nbytes for t in b.outgrown) <= sum(t.nbytes for t in b.kept.values())
        kept = dict(b.kept)
        thing(torch.zeros((1, 500, 256)[3 - rank:], dtype=torch.float16))
        assert all(b.kept[k] is t for k, t in kept.items())
