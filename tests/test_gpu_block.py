"""The 8-bit attention block as a whole: against fp64 on the unquantized weights,
one token at a time against the whole prompt, and captured in a graph."""
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


def make(sq, K, Hq, Hkv, D, seed=0, softcap=0.0, slopes=False):
    """(block, its fp32 weights)."""
    rng = np.random.default_rng(seed)
    w = {"gain": 1 + 0.2 * rng.standard_normal(K), "qkv": rng.standard_normal((K, (Hq + 2 * Hkv) * D)) / K ** 0.5,
         "out": rng.standard_normal((Hq * D, K)) / (Hq * D) ** 0.5,
         "qkv_bias": 0.1 * rng.standard_normal((Hq + 2 * Hkv) * D), "out_bias": 0.1 * rng.standard_normal(K),
         "slopes": 2.0 ** -np.arange(1, Hq + 1) if slopes else None}
    w = {k: None if v is None else v.astype(np.float32) for k, v in w.items()}
    block = sq.AttentionBlock(w["gain"], sq.prepare_weights_fp8(w["qkv"]), sq.prepare_weights_fp8(w["out"]),
                              Hq, Hkv, D, w["qkv_bias"], w["out_bias"], softcap=softcap, slopes=w["slopes"])
    return block, w


def reference(w, X, residual, Hq, Hkv, D, softcap, **mask):
    t = {k: None if v is None else torch.from_numpy(v).double() for k, v in w.items()}
    B, L, K = X.shape
    r = None if residual is None else residual.cpu().reshape(-1, K)
    h, u = R.norm(X.cpu().reshape(-1, K), r, t["gain"], 1e-6)
    q = (u @ t["qkv"] + t["qkv_bias"]).view(B, L, Hq + 2 * Hkv, D)
    o, _ = R.attention(q[:, :, :Hq], q[:, :, Hq:Hq + Hkv], q[:, :, Hq + Hkv:], D ** -0.5, softcap, t["slopes"], **mask)
    return (o.reshape(B * L, -1) @ t["out"] + t["out_bias"]).view(B, L, K), h.view(B, L, K)


def tokens(B, L, K, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, L, K, generator=g).to(dtype).cuda()


# An e4m3 rounding is off by 2.6% (rms) of a value: a product of two such operands
# by 3.7%; the logits of unit deviation by 5%, and the averages by as much besides;
# with the second product 7.3% of the whole. Twice that is allowed.
NEAR = 0.15


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B,L,K,Hq,Hkv,D,softcap,slopes,causal", [
    (1, 1, 256, 4, 2, 64, 0.0, False, True), (2, 77, 320, 5, 1, 64, 20.0, False, True),
    (2, 65, 640, 8, 8, 80, 0.0, False, False), (1, 200, 136, 6, 3, 24, 0.0, True, True)])
def test_near_the_unquantized_block(sq, B, L, K, Hq, Hkv, D, softcap, slopes, causal, dtype):
    block, w = make(sq, K, Hq, Hkv, D, softcap=softcap, slopes=slopes)
    X, r = tokens(B, L, K, dtype), tokens(B, L, K, dtype, 2)
    Y, h = block(X, r, causal=causal)
    y, hr = reference(w, X, r, Hq, Hkv, D, softcap, causal=causal)
    eps = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    assert float(((h.cpu().double() - hr).abs() - eps * hr.abs()).max()) <= 2.0 ** -20
    # the whole, and no row much further off than the others
    d, n = (Y.cpu().double() - y).norm(dim=2), y.norm(dim=2)
    assert float(d.norm() / n.norm()) < NEAR
    assert float((d / n.mean()).max()) < 3 * NEAR


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_token_by_token_is_the_whole_prompt(sq, dtype):
    """The same codes but where a 16-bit rounding of another order flips one: at
    most 3% of them by 9%, which is 1.5% of the output's norm."""
    B, L, K, Hq, Hkv, D = 3, 40, 256, 4, 2, 64
    block, _ = make(sq, K, Hq, Hkv, D)
    X = tokens(B, L, K, dtype)
    whole, _ = block(X)
    cache = sq.KeyValueCache(B, 64, Hkv, D, dtype)
    parts = [block(X[:, :33], cache=cache)[0]]
    parts += [block(X[:, i:i + 1], cache=cache)[0] for i in range(33, L)]
    got = torch.cat(parts, 1)
    assert cache.length == L
    assert float((got.double() - whole.double()).norm() / whole.double().norm()) < 0.04
    with pytest.raises(ValueError, match="cache of 64"):
        block(X, cache=cache)


def test_documents_do_not_see_each_other(sq):
    K, Hq, Hkv, D = 256, 4, 4, 64
    block, _ = make(sq, K, Hq, Hkv, D)
    lengths = [5, 70, 31]
    X = tokens(1, 110, K, torch.bfloat16)
    rg = torch.from_numpy(sq.document_key_ranges(lengths, 110)).cuda()
    packed, _ = block(X, key_ranges=rg)
    at = 0
    for n in lengths:
        alone, _ = block(X[:, at:at + n].contiguous())
        d = (packed[:, at:at + n].double() - alone.double()).norm() / alone.double().norm()
        assert float(d) < 0.04
        at += n


def test_no_tokens(sq):
    block, _ = make(sq, 256, 4, 2, 64)
    Y, h = block(tokens(2, 0, 256, torch.float16))
    assert Y.shape == h.shape == (2, 0, 256)


def test_another_stream(sq):
    block, _ = make(sq, 256, 4, 2, 64)
    X = tokens(2, 50, 256, torch.float16)
    want, _ = block(X)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got, _ = block(X)
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("B,L,cached", [(2, 77, 0), (4, 1, 600), (1, 300, 0)])
def test_replays_in_a_graph(sq, B, L, cached):
    """Every replay bit for bit the eager result, with eager work and
    synchronizations between the replays. The cached form splits its attention
    along the keys and, with K = 2560, its products along K."""
    K, Hq, Hkv, D = 2560, 8, 2, 64
    block, _ = make(sq, K, Hq, Hkv, D)
    X, r = tokens(B, L, K, torch.bfloat16), tokens(B, L, K, torch.bfloat16, 2)
    cache = None
    if cached:
        cache = sq.KeyValueCache(B, cached + L, Hkv, D, torch.bfloat16)
        cache.append(*(tokens(B, cached * Hkv, D, torch.bfloat16, i).view(B, cached, Hkv, D) for i in (3, 4)))

    def step():
        if cache is not None:
            cache.length = cached
        return block(X, r, cache=cache)

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    a = torch.randn(256, 256, device="cuda")
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        for t in block._kept.values():
            t.view(torch.uint8).fill_(0xA5)
        b = a @ a
        torch.cuda.synchronize()
        g.replay()
        c = b.sum()
        torch.cuda.synchronize()
        assert bool(torch.isfinite(c))
        for t, u in zip(got, want):
            assert torch.equal(t, u)
