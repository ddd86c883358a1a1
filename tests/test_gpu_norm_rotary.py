"""Norm and rotation of heads against the fp64 formula, and the same pass into the pages."""
import pytest
import torch

import paged_ref as P
from paged_ref import BF16, F16, F64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


def heads(T, H, D, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(T, H, D, generator=g)).to(dtype).cuda()


def gains(D, seed=3):
    g = torch.Generator().manual_seed(seed)
    return [(1 + 0.3 * torch.randn(D, generator=g)).cuda() for _ in range(2)]


def angles(sq, T, R, far=5000, seed=1, **kw):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, far, (T,), generator=g, dtype=torch.int32).cuda()
    f, a = sq.rotary_frequencies(R, **kw)
    return pos, torch.from_numpy(f).cuda(), a


def check(sq, q, k, q_out=None, k_out=None, positions=None, freqs=None, factor=1.0, interleaved=False, q_gain=None,
          k_gain=None, eps=None):
    qs, ks = q.clone(), None if k is None else k.clone()
    q_out = torch.full_like(q, 9.0, memory_format=torch.contiguous_format) if q_out is None else q_out
    if k is not None and k_out is None:
        k_out = torch.full_like(k, 9.0, memory_format=torch.contiguous_format)
    sq.norm_rotary(q, k, q_out, k_out, positions, freqs, factor, interleaved, q_gain, k_gain, eps)
    for x, out, gain in ((qs, q_out, q_gain), (ks, k_out, k_gain)):
        if x is not None:
            ref, err = P.heads(x, positions, freqs, factor, interleaved, gain, eps)
            P.assert_rounded(out, ref, err, x.dtype)
    return q_out, k_out


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(8, 8), (8, 2), (40, 40), (40, 20), (64, 64), (64, 16), (72, 72), (72, 6), (80, 32),
                                 (96, 24), (120, 120), (128, 128), (128, 64), (128, 32), (128, 16), (128, 2)])
def test_head_sizes(sq, D, R, interleaved, dtype):
    q, k = heads(13, 5, D, dtype), heads(13, 2, D, dtype, 1)
    pos, f, a = angles(sq, 13, R)
    gq, gk = gains(D)
    check(sq, q, k, positions=pos, freqs=f, interleaved=interleaved)
    check(sq, q, k, positions=pos, freqs=f, interleaved=interleaved, q_gain=gq, k_gain=gk, eps=1e-6)


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 32, 8), (2, 3, 0), (77, 12, 12), (300, 20, 4), (1031, 24, 24),
                                      (4099, 9, 3)])
def test_tokens_and_heads(sq, T, Hq, Hkv):
    for D, dtype in ((128, BF16), (64, F16)):
        q, k = heads(T, Hq, D, dtype), heads(T, Hkv, D, dtype, 1) if Hkv else None
        pos, f, a = angles(sq, T, D)
        gq, gk = gains(D)
        check(sq, q, k, positions=pos, freqs=f, q_gain=gq, k_gain=gk if Hkv else None, eps=1e-6)


@pytest.mark.parametrize("kw", [dict(), dict(eps=1e-6), dict(eps=1e-2, q_gain=True), dict(eps=1e-6, k_gain=True)])
def test_norm_alone_and_neither(sq, kw):
    q, k = heads(50, 4, 96, F16, scale=3.0), heads(50, 4, 96, F16, 1)
    gq, gk = gains(96)
    kw = dict(kw, **{n: t for n, t in (("q_gain", gq), ("k_gain", gk)) if n in kw})
    qo, ko = check(sq, q, k, **kw)
    if not kw:
        assert torch.equal(q, qo) and torch.equal(k, ko)


def test_far_positions(sq):
    """Angles of a million turns and of negative positions are those of the formula."""
    q = heads(64, 2, 128, F16)
    pos = torch.tensor([0, 1, -1, 2 ** 20, 2 ** 24 + 1, -(2 ** 30), 2 ** 31 - 1, 1000003] * 8, dtype=torch.int32).cuda()
    for kw in (dict(), dict(scaling="parts", scale=8.0), dict(base=500000.0)):
        f, a = sq.rotary_frequencies(128, **kw)
        for inter in (False, True):
            check(sq, q, None, positions=pos, freqs=torch.from_numpy(f).cuda(), factor=a, interleaved=inter)


def test_rotation_keeps_products_by_distance(sq):
    """q at i times k at j depends on i - j alone."""
    D, n = 64, 40
    q, k = heads(1, 1, D, F16).expand(n, 1, D).contiguous(), heads(1, 1, D, F16, 1).expand(n, 1, D).contiguous()
    f = torch.from_numpy(sq.rotary_frequencies(D)[0]).cuda()
    out = []
    for first in (0, 100000):
        pos = torch.arange(first, first + n, dtype=torch.int32).cuda()
        qo, ko = check(sq, q, k, positions=pos, freqs=f)
        out.append(qo[:, 0].double() @ ko[:, 0].double().t())
    # each of D terms: two fp16 roundings, twice; |q| |k| bounds the sum of the terms
    most = 2 * 2 * 2.0 ** -11 * float(q[0].double().norm() * k[0].double().norm()) * 1.01
    assert float((out[0] - out[1]).abs().max()) <= most
    d = out[0]
    assert float((d[1:, 1:] - d[:-1, :-1]).abs().max()) <= most


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_strides_and_in_place(sq, dtype):
    """Heads of one QKV product, rotated where they lie; V and the gaps stay."""
    T, Hq, Hkv, D = 37, 6, 2, 80
    x = heads(T, Hq + 2 * Hkv + 1, D, dtype)
    before = x.clone()
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    pos, f, a = angles(sq, T, 36)                      # 18 pairs: partners in the middle of other lanes
    for R in (36, 80):
        x.copy_(before)
        pos, f, a = angles(sq, T, R)
        check(sq, q, k, q, k, positions=pos, freqs=f, eps=1e-6)
        assert torch.equal(x[:, Hq + Hkv:], before[:, Hq + Hkv:])
    # heads before tokens, into rows with gaps
    y = before[:, :Hq].transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.full((T, Hq, D + 8), 7.0, dtype=dtype, device="cuda")
    check(sq, y, None, out[..., :D], positions=pos, freqs=f)
    assert bool((out[..., D:] == 7.0).all())


def test_infinities_and_nan_stay_in_their_head(sq):
    q = heads(6, 4, 128, BF16)
    q[1, 2, 5] = float("nan")
    q[2, 0, 127] = float("inf")
    q[3, 1, 40] = float("-inf")
    pos, f, a = angles(sq, 6, 32)
    out = torch.empty_like(q)
    sq.norm_rotary(q, None, out, None, pos, f)
    ref, err = P.heads(q, pos, f)
    bad = ~torch.isfinite(out.cpu())
    want = torch.zeros_like(bad)
    want[1, 2, [5, 21]] = True                         # the pair of channels 5 and 21
    want[2, 0, 127] = True                             # behind the rotated channels
    want[3, 1, 40] = True
    assert torch.equal(bad, want) and float(out[2, 0, 127]) == float("inf")
    sq.norm_rotary(q, None, out, None, pos, f, eps=1e-6)
    rows = torch.isfinite(out.cpu()).all(2)
    assert not rows[1, 2] and int((~rows).sum()) == 3


@pytest.mark.parametrize("D", [64, 80, 128])
def test_norms_of_very_large_and_small_values(sq, D):
    """bf16 rows whose squares leave fp32: the norm is that of the formula, beside ordinary rows."""
    q = heads(8, 3, D, BF16)
    for i, x in enumerate((1e30, 3e38 / 8, 1e-25, 1.0, 1e19, 1e-37, 1e10, 1e-12)):
        q[i, 1] = (q[i, 1].float() * x).to(BF16)
    for eps in (0.0, 1e-6):
        check(sq, q, None, eps=eps)


def test_zero_rows(sq):
    q = torch.zeros(3, 2, 64, dtype=F16, device="cuda")
    out = torch.full_like(q, 5.0)
    sq.norm_rotary(q, None, out, None, eps=1e-6)
    assert bool((out == 0).all())


def test_no_tokens_and_no_heads(sq):
    q = heads(0, 4, 64, F16)
    sq.norm_rotary(q, q, q, q, eps=1e-6)
    e = torch.empty(5, 0, 64, dtype=F16, device="cuda")
    k, ko = heads(5, 2, 64, F16), torch.empty(5, 2, 64, dtype=F16, device="cuda")
    sq.norm_rotary(e, k, e, ko)
    assert torch.equal(k, ko)


def test_another_stream_and_a_graph(sq):
    q, k = heads(33, 8, 128, BF16), heads(33, 2, 128, BF16, 1)
    pos, f, a = angles(sq, 33, 128)
    want = check(sq, q, k, positions=pos, freqs=f, eps=1e-6)
    torch.cuda.synchronize()
    outs = [torch.empty_like(q), torch.empty_like(k)]
    s = torch.cuda.Stream()
    sq.norm_rotary(q, k, *outs, pos, f, eps=1e-6, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sq.norm_rotary(q, k, *outs, pos, f, eps=1e-6)
    for i in range(3):
        for t in outs:
            t.fill_(0)
        pos.add_(i)
        want = check(sq, q, k, positions=pos, freqs=f, eps=1e-6)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))
