"""The attention block over a paged cache: against fp64 on the unquantized weights, against
the block without a cache, step by step with sequences of different lengths, in a graph."""
import numpy as np
import pytest
import torch

import block_ref as R
import paged_ref as P
from test_gpu_block import NEAR, make as plain_block, tokens

pytestmark = pytest.mark.gpu
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


def make(sq, K, Hq, Hkv, D, turned=True, interleaved=False, **kw):
    """(block, its fp32 weights): plain_block's with norms and rotation of the heads."""
    _, w = plain_block(sq, K, Hq, Hkv, D)
    rng = np.random.default_rng(9)
    if turned:
        w["head_gains"] = [(1 + 0.3 * rng.standard_normal(D)).astype(np.float32) for _ in range(2)]
        w["rotary"] = sq.rotary_frequencies(D // 2 if interleaved else D, 100.0)
        kw.update(head_gains=w["head_gains"], rotary=w["rotary"], interleaved=interleaved)
    w["interleaved"] = interleaved
    return sq.AttentionBlock(w["gain"], sq.prepare_weights_fp8(w["qkv"]), sq.prepare_weights_fp8(w["out"]), Hq, Hkv, D,
                             w["qkv_bias"], w["out_bias"], **kw), w


def reference(w, X, Hq, Hkv, D):
    """One whole sequence X (L x K) in fp64: Y."""
    t = {k: torch.from_numpy(w[k]).double() for k in ("gain", "qkv", "out", "qkv_bias", "out_bias")}
    L, K = X.shape
    _, u = R.norm(X.cpu(), None, t["gain"], 1e-6)
    x = (u @ t["qkv"] + t["qkv_bias"]).view(L, Hq + 2 * Hkv, D)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if "rotary" in w:
        f, a = torch.from_numpy(w["rotary"][0]), w["rotary"][1]
        gq, gk = (torch.from_numpy(g) for g in w["head_gains"])
        q, k = (P.heads(x, torch.arange(L), f, a, w["interleaved"], g, 1e-6)[0] for x, g in ((q, gq), (k, gk)))
    o, _ = R.attention(q[None], k[None], v[None], D ** -0.5, causal=True)
    return o.reshape(L, -1) @ t["out"] + t["out_bias"]


def near(got, want, limit=NEAR):
    d, n = (got.double().cpu() - want.double().cpu()).norm(dim=-1), want.double().cpu().norm(dim=-1)
    assert float(d.norm() / n.norm()) < limit, float(d.norm() / n.norm())


STEPS = ([30, 1, 0, 17], [1, 40, 90, 1], [1, 1, 1, 0], [3, 1, 1, 60], [1, 1, 1, 1])


@pytest.mark.parametrize("cached", ["own", E4M3])
@pytest.mark.parametrize("dtype,turned,interleaved", [(F16, True, False), (BF16, True, True), (BF16, False, False)])
def test_steps_of_unequal_sequences(sq, dtype, turned, interleaved, cached):
    """Five steps of four sequences are, together, each sequence's whole prompt: near the
    unquantized block, and near the same block without a cache (the bounds of the block's own
    tests; e4m3 keys and values are off by 2.6% rms each besides, as much as one more
    quantized operand)."""
    K, Hq, Hkv, D = 256, 8, 2, 64
    block, w = make(sq, K, Hq, Hkv, D, turned, interleaved)
    table = sq.PageTable(4, 130, page_size=16, step_tokens=160)
    scales = [0.05] * Hkv if cached is E4M3 else None
    cache = sq.PagedKeyValueCache(table, Hkv, D, dtype if cached == "own" else E4M3, scales, scales)
    whole = tokens(4, 130, K, dtype)
    at, parts = [0] * 4, [[] for _ in range(4)]
    for counts in STEPS:
        table.begin(counts)
        X = torch.cat([whole[b, at[b]:at[b] + n] for b, n in enumerate(counts)])[None]
        Y, h = block(X, cache=cache)
        assert torch.equal(h, X)
        row = 0
        for b, n in enumerate(counts):
            parts[b].append(Y[0, row:row + n])
            at[b] += n
            row += n
    for b in range(4):
        got = torch.cat(parts[b])
        assert table.length(b) == at[b] == len(got)
        near(got, reference(w, whole[b, :at[b]], Hq, Hkv, D), NEAR if cached == "own" else 1.5 * NEAR)
        alone, _ = block(whole[b:b + 1, :at[b]])
        near(got, alone[0], 0.04 if cached == "own" else NEAR)


def test_rotated_heads_without_a_cache(sq):
    """The block's norms and rotation in the dense path: a prompt, and token by token."""
    K, Hq, Hkv, D = 256, 4, 2, 64
    for interleaved in (False, True):
        block, w = make(sq, K, Hq, Hkv, D, True, interleaved)
        X = tokens(2, 40, K, BF16)
        whole, _ = block(X)
        for b in range(2):
            near(whole[b], reference(w, X[b], Hq, Hkv, D))
        cache = sq.KeyValueCache(2, 64, Hkv, D, BF16)
        parts = [block(X[:, :33], cache=cache)[0]] + [block(X[:, i:i + 1], cache=cache)[0] for i in range(33, 40)]
        near(torch.cat(parts, 1), whole, 0.04)
        given, _ = block(X, positions=torch.arange(40, dtype=torch.int32, device="cuda").repeat(2, 1))
        assert torch.equal(given, whole)


def test_two_layers_one_table_and_a_released_sequence(sq):
    K, Hq, Hkv, D = 256, 4, 2, 64
    blocks = [make(sq, K, Hq, Hkv, D)[0] for _ in range(2)]
    table = sq.PageTable(2, 64, page_size=16, pages=6)
    caches = [sq.PagedKeyValueCache(table, Hkv, D, BF16) for _ in range(2)]

    def step(X, counts):
        table.begin(counts)
        h = None
        for b, c in zip(blocks, caches):
            X, h = b(X, h, cache=c)
        return X

    X = tokens(1, 50, K, BF16)
    first = step(X, [50, 0])                            # 4 of 6 pages
    table.release(0)
    assert torch.equal(step(X, [0, 50]), first)         # the same sequence in its place, over old pages
    with pytest.raises(ValueError, match="pages"):
        table.begin([40, 0])
    table.release(1)
    assert torch.equal(step(X, [50, 0]), first)


def test_rows_behind_the_step(sq):
    """A call of more rows than the step has tokens: the tokens' rows are those of a call without
    the others, and nothing of the others' is stored."""
    K, Hq, Hkv, D = 256, 4, 2, 64
    block, _ = make(sq, K, Hq, Hkv, D)
    out, pages = [], []
    for extra in (0, 9):
        table = sq.PageTable(2, 64, step_tokens=64)
        cache = sq.PagedKeyValueCache(table, Hkv, D, BF16)
        cache.k.zero_(), cache.v.zero_()
        X = tokens(1, 30, K, BF16)
        junk = torch.full((1, extra, K), float("nan"), dtype=BF16, device="cuda")
        for counts in ([20, 10], [1, 0]):
            table.begin(counts)
            Y, _ = block(torch.cat([X[:, :sum(counts)], junk], 1), cache=cache)
            out.append(Y[:, :sum(counts)])
        pages.append((cache.k.clone(), cache.v.clone()))
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])
    assert torch.equal(pages[0][0], pages[1][0]) and torch.equal(pages[0][1], pages[1][1])


@pytest.mark.parametrize("cached", [BF16, E4M3])
def test_one_graph_generates(sq, cached):
    """A graph of the layer captured once, replayed while the sequences grow, one ends and another
    takes its place: every replay the eager result's bits."""
    K, Hq, Hkv, D = 1280, 8, 2, 64
    block, _ = make(sq, K, Hq, Hkv, D)
    prompts, steps = tokens(1, 1300, K, BF16), [tokens(1, 4, K, BF16, 20 + i) for i in range(6)]

    def run(graphed):
        table = sq.PageTable(4, 1400, page_size=64, step_tokens=1300)
        cache = sq.PagedKeyValueCache(table, Hkv, D, cached, *([[0.05] * Hkv] * 2 if cached is E4M3 else ()))
        table.begin([1200, 60, 40, 0])
        block(prompts, cache=cache)
        X = torch.empty(1, 4, K, dtype=BF16, device="cuda")
        out, g = [], None
        for i, x in enumerate(steps):
            if i == 3:
                table.release(1)
            table.begin([1, 1, 1, 0] if i < 3 else [1, 2, 1, 0] if i == 4 else [1, 1, 1, 1])
            X.copy_(x)
            if not graphed:
                Y, _ = block(X, cache=cache)
            else:
                if g is None:
                    block(X, cache=cache)               # buffers, and the same slots written once before
                    torch.cuda.synchronize()
                    g = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(g):
                        Y, _ = block(X, cache=cache)
                torch.cuda.synchronize()
                Y.fill_(float("nan"))
                for t in block._kept.values():
                    t.view(torch.uint8).fill_(0xA5)
                g.replay()
                torch.cuda.synchronize()
            out.append(Y[:, :table.tokens].clone())
        return out

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)
