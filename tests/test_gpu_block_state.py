"""What an attention block keeps between calls: its cache after a refused call, its
buffers beside graphs and on other streams."""
import numpy as np
import pytest
import torch

from test_gpu_block import make, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


def test_a_retry_after_a_refused_call_is_the_call(sq):
    B, K, Hq, Hkv, D = 2, 256, 4, 2, 64
    block, _ = make(sq, K, Hq, Hkv, D)
    X = tokens(B, 12, K, torch.float16)
    caches = [sq.KeyValueCache(B, 16, Hkv, D, torch.float16) for _ in range(2)]
    for c in caches:
        block(X[:, :9], cache=c)
    for kw in (dict(causal=False, prefix=torch.zeros(B, dtype=torch.int32, device="cuda")),
               dict(key_ranges=torch.zeros(B + 1, 3, 2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            block(X[:, 9:], cache=caches[1], **kw)
    want, got = (block(X[:, 9:], cache=c)[0] for c in caches)
    assert torch.equal(want, got) and caches[0].length == caches[1].length == 12
    assert torch.equal(caches[0].k[:, :12], caches[1].k[:, :12])


def replayed_beside_larger_calls(step, larger, fill):
    """step() captured, then larger() eagerly and its memory's neighbours taken by other
    tensors: every replay gives the eager bits and changes none of those."""
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(2):
        larger()
        others = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in fill for _ in range(8)]
        torch.cuda.synchronize()
        for t in got:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for t, u in zip(got, want):
            assert torch.equal(t, u)
        for t in others:
            assert bool((t == 0x5A).all())
    del g


def test_a_graph_beside_larger_calls_of_its_block(sq):
    K, Hq, Hkv, D = 2560, 8, 2, 64
    block, _ = make(sq, K, Hq, Hkv, D)
    X, Z = tokens(1, 5, K, torch.bfloat16), tokens(2, 300, K, torch.bfloat16, 2)
    sizes = {t.nbytes for t in (X, Z)}
    block(X)
    sizes |= {t.nbytes for t in block._kept.values()}
    replayed_beside_larger_calls(lambda: block(X), lambda: block(Z), sorted(sizes))


@pytest.mark.parametrize("fmt", ["fp8", "int4"])
def test_a_graph_beside_larger_calls_of_its_layer(sq, fmt):
    g = torch.Generator().manual_seed(3)
    W = (torch.randn(2560, 640, generator=g) / 50).numpy()
    prep = sq.prepare_weights_fp8(W) if fmt == "fp8" else sq.prepare_weights(W, np.ones(2560, np.float32), 16)
    lin = sq.Linear(prep)
    X, Z = (torch.randn(m, 2560, generator=g).half().cuda() for m in (20, 900))
    n = lin.workspace(20).nbytes
    replayed_beside_larger_calls(lambda: (lin(X),), lambda: lin(Z), [n])


def test_a_buffer_outgrown_on_another_stream(sq):
    """The outgrown buffers come from the default stream's memory and are still read by
    work queued on another: what that stream allocates next does not overwrite them."""
    K, Hq, Hkv, D = 2560, 8, 2, 64
    block, _ = make(sq, K, Hq, Hkv, D)
    X, Z = tokens(1, 200, K, torch.bfloat16), tokens(2, 300, K, torch.bfloat16, 2)
    want, _ = block(X)
    sizes = [t.nbytes for t in block._kept.values()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got, _ = block(X)
        block(Z)
    for n in sizes:
        torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(got, want)
