"""Norms of bf16 heads among the type's smallest values, where the reciprocal of the root alone
leaves fp32, against the fp64 formula."""
import pytest
import torch

import paged_ref as P
from paged_ref import BF16, E4M3, F64
from test_gpu_norm_rotary import angles, check, gains, heads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


SCALES = (1e-36, 1e-38, 2e-39, 1e-40, 1.0, 3e-40, 1e38, 4e-41)


def tiny_heads(D):
    """Tokens of which one head is scaled each, beside ordinary ones, and heads of one value."""
    q = heads(len(SCALES) + 4, 3, D, BF16)
    for i, x in enumerate(SCALES):
        q[i, 1] = (q[i, 1].double() * x).to(BF16)
    for i, (ch, x) in enumerate(((0, 2.0 ** -125), (3, -2.0 ** -133), (D - 1, 2.0 ** -128), (5, 2.0 ** 127))):
        q[len(SCALES) + i, 2] = 0
        q[len(SCALES) + i, 2, ch] = x
    return q


# no rotation; halves of the head; neighbours; other lanes; partners read from memory again
@pytest.mark.parametrize("R,interleaved", [(0, False), (-1, False), (-1, True), (32, False), (36, False)])
@pytest.mark.parametrize("D", [64, 80, 128])
def test_rows_of_the_smallest_values(sq, D, R, interleaved):
    q = tiny_heads(D)
    R = D if R < 0 else R
    pos, f, a = angles(sq, q.shape[0], R) if R else (None, None, 1.0)
    gq, _ = gains(D)
    for eps in (0.0, 2.0 ** -126, 1e-30):
        check(sq, q, None, positions=pos, freqs=f, interleaved=interleaved, eps=eps)
        check(sq, q, None, positions=pos, freqs=f, interleaved=interleaved, q_gain=gq, eps=eps)


@pytest.mark.parametrize("coded", [False, True])
def test_they_are_written_so(sq, coded):
    D, page = 80, 16
    k = tiny_heads(D)
    T, H = k.shape[:2]
    pos, f, a = angles(sq, T, 36)
    pages = [torch.zeros(2, H, page, D, dtype=E4M3 if coded else BF16, device="cuda") for _ in range(2)]
    ks = torch.tensor([0.02, 0.03, 0.05], device="cuda") if coded else None
    slots = torch.arange(T, dtype=torch.int32).flip(0).contiguous()
    sq.norm_rotary_write(None, k, k, None, slots.cuda(), *pages, ks, None, pos, f, eps=0.0)
    ref, err = P.heads(k, pos, f, eps=0.0)
    i = slots.long()
    got = pages[0].cpu().view(torch.uint8 if coded else BF16)[i // page, :, i % page]
    if coded:
        P.assert_codes(got.view(E4M3), ref, err, ks.cpu().to(F64).view(-1, 1))
    else:
        P.assert_rounded(got, ref, err, BF16)
