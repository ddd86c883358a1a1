"""Masked attention against the fp64 formula: lengths from one token on, every
head layout, mask and score change, strides, hidden infinities and NaN."""
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


def qkv(B, Lq, Lk, Hq, Hkv, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda L, H: torch.randn(B, L, H, D, generator=g).to(dtype).cuda()  # noqa: E731
    return mk(Lq, Hq), mk(Lk, Hkv), mk(Lk, Hkv)


def run(sq, q, k, v, ws=True, scale=None, out=None, **kw):
    B, Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[1:3]
    out = torch.full_like(q, 9.0, memory_format=torch.contiguous_format) if out is None else out
    need = sq.attention_workspace_bytes(B, Lq, Lk, Hq, Hkv, D)
    work = torch.full((need // 4,), float("nan"), device="cuda") if ws and need else None
    sq.attention(q, k, v, out, scale=scale, ws=work, **kw)
    return out


def check(sq, q, k, v, ws=True, scale=None, out=None, **kw):
    got = run(sq, q, k, v, ws, scale, out, **kw)
    ref, bound = R.attention(q, k, v, q.shape[3] ** -0.5 if scale is None else scale,
                             kw.get("softcap", 0.0), kw.get("slopes"), kw.get("causal", False),
                             kw.get("prefix"), kw.get("key_ranges"))
    R.assert_within(got, ref, bound)
    return got


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [8, 40, 64, 72, 80, 96, 120, 128])
def test_head_sizes(sq, D, dtype):
    check(sq, *qkv(1, 70, 90, 2, 2, D, dtype))
    check(sq, *qkv(2, 3, 200, 4, 2, D, dtype))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Lq,Lk", [(1, 1), (1, 2), (1, 31), (1, 33), (2, 64), (31, 31), (32, 65), (33, 128),
                                   (64, 64), (65, 129), (127, 191), (128, 128), (129, 257), (300, 300)])
def test_lengths(sq, Lq, Lk, causal):
    check(sq, *qkv(1, Lq, Lk, 2, 2, 64, F16), causal=causal)
    check(sq, *qkv(1, Lq, Lk, 2, 1, 128, BF16), causal=causal)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (6, 2), (8, 1), (5, 1), (16, 4)])
def test_grouped_heads(sq, Hq, Hkv):
    check(sq, *qkv(2, 50, 77, Hq, Hkv, 64, F16), causal=True)
    check(sq, *qkv(2, 1, 300, Hq, Hkv, 128, BF16))


def test_more_queries_than_keys(sq):
    """Causal rows before the first key see nothing and come out 0."""
    out = check(sq, *qkv(1, 150, 40, 2, 2, 64, F16), causal=True)
    assert bool((out[:, :110] == 0).all()) and bool((out[:, 110:] != 0).any())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("Lq", [1, 4, 200])
def test_cap_and_slopes(sq, Lq, dtype):
    q, k, v = qkv(2, Lq, 333, 4, 2, 128, dtype)
    sl = torch.tensor([0.5, 0.1, 0.01, 1.0], device="cuda")
    check(sq, 4 * q, k, v, softcap=3.0)
    check(sq, q, k, v, slopes=sl)
    check(sq, q, k, v, softcap=20.0, slopes=sl, causal=True)
    check(sq, 60 * q, 60 * k, v, softcap=30.0)          # scores deep in the saturated part


@pytest.mark.parametrize("Lq,Lk", [(100, 100), (257, 257), (5, 400), (1, 700)])
def test_prefix(sq, Lq, Lk):
    q, k, v = qkv(3, Lq, Lk, 2, 2, 64, F16)
    p = torch.tensor([0, Lk // 2, Lk + 5], device="cuda", dtype=torch.int32)
    check(sq, q, k, v, causal=True, prefix=p)


def test_documents(sq):
    q, k, v = qkv(2, 300, 300, 2, 1, 64, BF16)
    r = torch.from_numpy(sq.document_key_ranges([1, 63, 0, 64, 100, 2], 300)).cuda()
    out = check(sq, q, k, v, key_ranges=r)
    assert bool((out[:, 230:] == 0).all())               # padding sees nothing
    check(sq, q, k, v, key_ranges=r, causal=True)
    # each document alone gives the same rows
    alone = run(sq, q[:, 128:228], k[:, 128:228], v[:, 128:228])
    assert bool(((alone - out[:, 128:228]).abs() <= 2.0 ** -7 * alone.abs() + 2.0 ** -7).all())


@pytest.mark.parametrize("Lq", [1, 7, 140])
def test_arbitrary_ranges(sq, Lq):
    """Unordered, empty, reversed and out-of-range intervals, per batch entry."""
    B, Lk = 3, 500
    q, k, v = qkv(B, Lq, Lk, 4, 2, 128, F16)
    g = torch.Generator().manual_seed(5)
    r = torch.randint(-50, Lk + 50, (B, Lq, 2), generator=g, dtype=torch.int32)
    r[0] = r[0].sort(dim=1).values
    r[1, : Lq // 2] = 0
    check(sq, q, k, v, key_ranges=r.cuda())
    check(sq, q, k, v, key_ranges=r.cuda(), causal=True,
          prefix=torch.tensor([100, 0, 499], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("Lq", [1, 40, 200])
def test_everything_hidden(sq, Lq):
    q, k, v = qkv(2, Lq, 400, 4, 4, 64, F16)
    k.fill_(float("nan"))
    v.fill_(float("nan"))
    r = torch.zeros(1, Lq, 2, dtype=torch.int32, device="cuda")
    assert bool((run(sq, q, k, v, key_ranges=r) == 0).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("Lq,kw", [(1, {}), (130, dict(causal=True)), (200, {}), (12, {})])
def test_hidden_infinities_and_nan(sq, Lq, kw, dtype):
    """K and V of hidden keys hold NaN and infinities: no row that does not see them
    changes; a visible NaN or infinity in V arrives in its channel and rows."""
    Lk = 230
    q, k, v = qkv(1, Lq, Lk, 2, 2, 64, dtype)
    r = torch.zeros(1, Lq, 2, dtype=torch.int32)
    r[..., 0], r[..., 1] = 20, 190
    r[0, Lq // 2:, 1] = 150
    for key, val in ((3, float("nan")), (210, float("inf"))):          # hidden from all rows
        k[:, key], v[:, key] = val, val
    v[0, 160, 0, 5], v[0, 170, 0, 6] = float("inf"), float("nan")      # hidden from half of them
    v[0, 165, 1, 7], v[0, 166, 1, 9] = float("-inf"), float("inf")
    v[0, 167, 1, 9] = float("-inf")
    check(sq, q, k, v, key_ranges=r.cuda(), **kw)


def test_hidden_nan_in_keys_of_a_shared_tile(sq):
    q, k, v = qkv(1, 64, 64, 1, 1, 128, F16)
    k[0, 40] = float("nan")
    out = run(sq, q, k, v, causal=True).cpu()
    assert not bool(torch.isnan(out[0, :40]).any()) and bool(torch.isnan(out[0, 40:]).all())


def test_scores_of_the_lowest_value(sq):
    """Scores near fp32's and fp16's lowest finite values are scores, not masks."""
    q = torch.full((1, 40, 1, 64), 60000.0, dtype=F16, device="cuda")
    k = torch.full((1, 50, 1, 64), -60000.0, dtype=F16, device="cuda")
    v = torch.randn(1, 50, 1, 64, generator=torch.Generator().manual_seed(1)).to(F16).cuda()
    out = run(sq, q, k, v, scale=1e20).cpu().double()
    ref = v.cpu().double().mean(1, keepdim=True).expand_as(out)
    assert float((out - ref).abs().max()) < 2.0 ** -10
    check(sq, q, k, v, softcap=5.0, scale=1.0)


@pytest.mark.parametrize("kw", [{}, dict(softcap=4.0)])
def test_negative_and_zero_scale(sq, kw):
    q, k, v = qkv(1, 70, 200, 2, 2, 64, BF16)
    check(sq, q, k, v, scale=-0.3, **kw)
    check(sq, q, k, v, scale=0.0, causal=True, **kw)


def test_logits_that_grow_along_the_keys(sq):
    """Each block of keys outgrows the reference maximum of the one before, slowly,
    suddenly, and beyond what one rounding of scale times score would survive."""
    q, k, v = qkv(1, 130, 512, 1, 1, 128, BF16)
    ramp = torch.arange(512, device="cuda")[None, :, None, None]
    check(sq, q, (k * (1 + ramp / 32)).to(BF16), v)
    check(sq, q, (k * torch.where(ramp % 96 < 32, 1.0, 40.0)).to(BF16), v)
    check(sq, q, (k * torch.where(ramp < 300, 1.0, 3e4)).to(BF16), v, scale=10.0)
    check(sq, q, (k * torch.where(ramp < 300, 1.0, 1e30)).to(BF16), v)
    check(sq, (q * 1e30).to(BF16), k, v)


@pytest.mark.parametrize("Lq,Lk,Hq,Hkv", [(1, 5000, 8, 2), (3, 3000, 4, 4), (128, 4096, 2, 1), (260, 2100, 1, 1)])
def test_split_along_the_keys(sq, Lq, Lk, Hq, Hkv):
    """With the workspace the keys are split over workgroups, without it they are not."""
    q, k, v = qkv(1, Lq, Lk, Hq, Hkv, 128, BF16)
    assert sq.attention_workspace_bytes(1, Lq, Lk, Hq, Hkv, 128) > 0
    r = torch.zeros(1, Lq, 2, dtype=torch.int32)
    r[..., 1] = torch.arange(Lq) * 7 + Lk // 3           # some splits see nothing
    for ws in (True, False):
        check(sq, q, k, v, ws=ws)
        check(sq, q, k, v, ws=ws, causal=True, softcap=10.0)
        check(sq, q, k, v, ws=ws, key_ranges=r.cuda())


def test_strides(sq):
    """Fused QKV slices, head-major caches, batch and head broadcast, a strided output."""
    B, L, H, D = 2, 90, 4, 72
    g = torch.Generator().manual_seed(3)
    x = torch.randn(B, L, 3 * H * D + 16, generator=g).to(F16).cuda()
    q, k, v = (x[..., i * H * D:(i + 1) * H * D].unflatten(2, (H, D)) for i in range(3))
    out = torch.full((B, H, L, D + 8), 5.0, dtype=F16, device="cuda")
    check(sq, q, k, v, out=out[..., :D].transpose(1, 2), causal=True)
    assert bool((out[..., D:] == 5.0).all())
    hm = torch.randn(2, 2, 400, D, generator=g).to(F16).cuda()
    check(sq, q, hm.transpose(1, 2), hm.transpose(1, 2))
    one = torch.randn(1, 1, 77, D, generator=g).to(F16).cuda().transpose(1, 2)
    check(sq, q, one.expand(B, 77, 2, D), one.expand(B, 77, 2, D))
    check(sq, q[:, :1], one.expand(B, 77, 1, D), one.expand(B, 77, 1, D))


def test_key_offsets_past_32_bits(sq):
    """A cache whose last keys lie more than 2^32 elements behind its first."""
    L, ld = 1100, 1 << 22
    buf = torch.empty(L * ld, dtype=F16, device="cuda")
    g = torch.Generator().manual_seed(4)
    kv = buf.as_strided((1, L, 2, 64), (0, ld, 64, 1))
    kv.copy_(torch.randn(1, L, 2, 64, generator=g))
    k, v = kv[:, :, :1], kv[:, :, 1:]
    for Lq in (1, 64):
        q = torch.randn(1, Lq, 1, 64, generator=g).to(F16).cuda()
        check(sq, q, k, v)
    del buf, kv


def test_nothing_to_do(sq):
    q, k, v = qkv(0, 5, 5, 2, 2, 64, F16)
    run(sq, q, k, v)
    q, k, v = qkv(2, 0, 5, 2, 2, 64, F16)
    run(sq, q, k, v)
    q, k, v = qkv(2, 5, 0, 2, 2, 64, F16)
    assert bool((run(sq, q, k, v, causal=True) == 0).all())
    assert bool((run(sq, q, k, v) == 0).all())


def test_repeats_bit_for_bit_and_on_another_stream(sq):
    for Lq, Lk in ((1, 4000), (300, 300)):
        q, k, v = qkv(2, Lq, Lk, 8, 2, 128, BF16)
        ref = run(sq, q, k, v, causal=True)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got = run(sq, q, k, v, causal=True)
        st.synchronize()
        assert torch.equal(ref, got)
