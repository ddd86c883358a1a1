"""Attention over the whole range of its numbers. Each bound is derived from the
roundings that the header and the formula's comment state."""
import math

import pytest
import torch

import block_ref as R
from test_gpu_attention import BF16, F16, check, qkv, run

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


def capped(q, k, v, scale, cap, slopes=None, causal=False):
    """(out, bound) in fp64 with the cap's error relative to the score.

    A logit's error: D + 4 fp32 roundings of the dot product, 2^-19 of the capped
    score (tanh, whichever form; caps up to 64 may be off by 8 * 2^-24 of the cap
    instead), and 4 roundings of the largest logit in base 2. It moves an average
    of v by twice that times the average of |v|; P and the output are rounded once."""
    B, Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[1:3]
    eps, sub = (2.0 ** -11, 2.0 ** -25) if q.dtype == F16 else (2.0 ** -8, 0.0)
    q, k, v = (t.cpu().to(F64) for t in (q, k, v))
    out, bound = (torch.zeros(B, Lq, Hq, D, dtype=F64) for _ in range(2))
    far = (torch.arange(Lq)[:, None] + Lk - Lq) - torch.arange(Lk)[None]
    for b in range(B):
        for h in range(Hq):
            kk, vv = k[b, :, h // (Hq // Hkv)], v[b, :, h // (Hq // Hkv)]
            x = (q[b, :, h] @ kk.t().contiguous()) * scale
            dx = (D + 4) * 2.0 ** -24 * abs(scale) * q[b, :, h].norm(dim=1, keepdim=True) * kk.norm(dim=1).max()
            x = cap * torch.tanh(x / cap)
            dx = dx + 2.0 ** -19 * x.abs().amax(1, keepdim=True) + (8 * cap * 2.0 ** -24 if cap <= 64 else 0.0)
            if slopes is not None:
                s = float(slopes[h])
                x = x - s * far.abs()
                dx = dx + 4 * s * (Lk + Lq) * 2.0 ** -24
            if causal:
                x = torch.where(far >= 0, x, -math.inf)
            dx = dx + 4 * 2.0 ** -24 * (2 + x.amax(1, keepdim=True).abs())
            p = torch.softmax(x, 1)
            o, a = p @ vv, p @ vv.abs()
            out[b, :, h] = o
            tail = Lk * sub * vv.abs().max() / (p / p.amax(1, keepdim=True)).sum(1, keepdim=True)
            bound[b, :, h] = eps * (a + o.abs()) + (2 * dx + 2.0 ** -20) * a + tail + sub
    return out, bound


# one row, one row tile of 32 rows and more, and enough sequences for tiles of 128
SHAPES = [(1, 1, 300, 2, 1, 128), (2, 70, 130, 2, 2, 64), (16, 75, 90, 16, 16, 64)]
CAPS = [1e-44, 1e-3, 30.0, 64.0, 65.0, 1e3, 1e5, 1e6, 1e7, 1e8, 3e38]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_any_cap(sq, shape, cap, dtype):
    q, k, v = qkv(*shape, dtype)
    scale = 2 * shape[5] ** -0.5                         # logits of deviation 2
    R.assert_within(run(sq, q, k, v, scale=scale, softcap=cap), *capped(q, k, v, scale, cap))


@pytest.mark.parametrize("cap", [50.0, 300.0, 1e6])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_a_cap_with_slopes_masks_and_large_scores(sq, shape, cap):
    q, k, v = qkv(*shape, BF16)
    sl = torch.logspace(-3, 0, shape[3], device="cuda")
    R.assert_within(run(sq, q, k, v, scale=-0.1, softcap=cap, slopes=sl, causal=True),
                    *capped(q, k, v, -0.1, cap, sl, True))
    # scores from nothing to far beyond the cap in one row
    ramp = torch.logspace(-4, 3, shape[2], device="cuda")[None, :, None, None]
    k2 = (k * ramp).to(BF16)
    R.assert_within(run(sq, q, k2, v, scale=0.1, softcap=cap), *capped(q, k2, v, 0.1, cap))


@pytest.mark.parametrize("shape", [(1, 1, 4096, 1, 1, 64), (1, 40, 4096, 2, 2, 64), (16, 75, 1024, 16, 16, 64)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("nats", [8.0, 14.0, 17.0, 17.5, 20.0])
@pytest.mark.parametrize("at", [0, -1], ids=["first", "last"])
def test_many_small_weights_beside_one_large(sq, shape, nats, at):
    """A key far above all others whose V is 0, as models learn them: the output is what
    the others bring, whose weights are down to e^-21 of the row's largest. fp16 weights
    are multiples of 2^-34 of the largest at the coarsest: half of that step for every
    key, besides one rounding each of the weight and the output, and the error of a
    logit (D + 4 roundings of the product, 4 in base 2)."""
    B, Lq, Lk, Hq, Hkv, D = shape
    q, k, v = qkv(*shape, F16)
    q[..., 0], q[..., 1:] = 1.0, 0.0
    k[..., 0], k[..., 1:] = -torch.rand(k.shape[:3], generator=torch.Generator().manual_seed(1)).cuda(), 0.0
    k[:, at, :, 0] = nats
    v = (64.0 + 8 * v).clamp(0, 128).to(F16)
    v[:, at] = 0
    got = run(sq, q, k, v, scale=1.0).cpu().to(F64)
    w = torch.exp(k[..., :1].cpu().to(F64) - nats)
    total = w.sum(1, keepdim=True)
    o = ((w * v.cpu().to(F64)).sum(1, keepdim=True) / total).expand(B, Lq, Hq, D)
    dx = (D + 4) * 2.0 ** -24 * nats + 4 * 2.0 ** -24 * (2 + nats)
    bound = 2.0 ** -11 * 2 * o + 2 * dx * o + (Lk - 1) * 2.0 ** -35 * 128 / total + 2.0 ** -25
    R.assert_within(got, o, bound)


def test_weights_are_rounded_once(sq):
    """32 keys, then 32 that outgrow them while the first block's weights are waiting in
    16 bits: were those rounded again after their rescaling, the output (all of it
    theirs) would be off by 2.6 units of its type's precision, where two are allowed."""
    B, H, L, D = 16, 16, 75, 64
    q = torch.zeros(B, L, H, D, dtype=F16, device="cuda")
    k = torch.zeros(B, 64, H, D, dtype=F16, device="cuda")
    v = torch.zeros_like(k)
    q[..., 0] = 1.0
    k[:, 1:32, :, 0], k[:, 32:, :, 0] = -0.58984375, 6.296875
    v[:, 1:32] = 64.0
    check(sq, q, k, v, scale=1.0)


@pytest.mark.parametrize("shape", [(1, 1, 300, 2, 1, 64), (1, 3, 5000, 2, 2, 128), (2, 70, 130, 2, 2, 64),
                                   (16, 75, 200, 16, 16, 64)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("most", [3e38, 1e36])
def test_values_near_the_end_of_bf16(sq, shape, most):
    """Averages of values that are finite, but whose sums are not."""
    q, k, v = qkv(*shape, BF16)
    v = (v.sign() * most).to(BF16)
    for ws in (True, False):
        check(sq, q, k, v, ws=ws)
        check(sq, q, k, v.abs(), ws=ws, causal=True)


def test_the_largest_fp16_values(sq):
    """An average of 65504 is 65504 in every row."""
    q, k, v = qkv(2, 70, 300, 2, 2, 64, F16)
    v.fill_(65504.0)
    out = run(sq, q, k, v)
    assert bool((out >= 65472).all()) and bool(torch.isfinite(out).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("shape", [(2, 1, 40, 4, 2, 128), (1, 70, 70, 2, 2, 64), (16, 75, 90, 16, 16, 64)],
                         ids=lambda s: "x".join(map(str, s)))
def test_a_row_that_sees_one_key_is_its_value(sq, shape, dtype):
    """And a row of equal values is that value, up to the last ones that fp16 has: the
    weights add up to 1 after their rounding."""
    B, Lq, Lk, Hq, Hkv, D = shape
    q, k, v = qkv(*shape, dtype)
    r = torch.zeros(1, Lq, 2, dtype=torch.int32)
    r[0, :, 0] = torch.arange(Lq) % Lk
    r[0, :, 1] = r[0, :, 0] + 1
    out = run(sq, q, k, v, key_ranges=r.cuda())
    assert torch.equal(out, v[:, r[0, :, 0].long().cuda()].repeat_interleave(Hq // Hkv, 2))
    v = torch.where(v > 0, 65504.0, -65504.0)[:, :1].expand_as(v).to(dtype).contiguous()
    assert torch.equal(run(sq, q, k, v), v[:, :1].repeat_interleave(Hq // Hkv, 2).expand_as(q))
