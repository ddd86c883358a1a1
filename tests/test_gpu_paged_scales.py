"""Scales at the bounds of their range: attention with and without slopes and caps under masks,
codes written and read, against fp64."""
import pytest
import torch

import paged_ref as P
from paged_ref import BF16, E4M3, F64
from test_gpu_norm_rotary import heads
from test_gpu_paged_attention import check, queries, starts_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


@pytest.mark.parametrize("slopes,cap", [(False, 0.0), (True, 0.0), (True, 20.0), (False, 1e5)])
@pytest.mark.parametrize("ks,scale", [(2.0 ** -64, 2.0 ** -40), (2.0 ** -64, 1.0), (2.0 ** -64, 2.0 ** 58), (2.0 ** 64, 2.0 ** -40),
                                      (2.0 ** 33, -2.0 ** -38)])
def test_attention(sq, ks, scale, slopes, cap):
    held, new = [150, 40, 333], [140, 1, 3]
    p = P.Pool(held, 2, 64, BF16, True, 16).poison_free().cuda()
    p.ks = torch.tensor([ks, ks], device="cuda")
    # scores within 2^6 or so whatever the two scales are
    q = queries(sum(new), 4, 64, BF16)
    most = 448 * 64 * abs(ks * scale)
    if most > 64:
        q = (q.double() * (64 / most)).to(BF16)
    p.vs = torch.tensor([2.0 ** -64, 2.0 ** 64], device="cuda")
    sl = torch.tensor([0.5, 0.1, 0.01, 1.0], device="cuda") if slopes else None
    check(sq, q, p, starts_of(new), scale=scale, softcap=cap, slopes=sl)


def test_codes(sq):
    """Zeros stay zeros and the others are the formula's codes."""
    T, H, D, page = 20, 2, 64, 16
    s = torch.tensor([2.0 ** -64, 2.0 ** 64], device="cuda")
    k = (heads(T, H, D, BF16).double() * 30 * s.double().view(1, H, 1)).to(BF16)
    k[:, :, ::7] = 0
    pages = [torch.full((2, H, page, D), 1.0, device="cuda").to(E4M3) for _ in range(2)]
    slots = torch.arange(T, dtype=torch.int32)
    sq.paged_write(k, k, slots.cuda(), *pages, s, s)
    i = slots.long()
    for x in pages:
        codes = x.cpu().view(torch.uint8)[i // page, :, i % page].view(E4M3)
        ref = k.cpu().to(F64)
        P.assert_codes(codes, ref, torch.zeros_like(ref), s.cpu().to(F64).view(-1, 1))
        assert bool((codes.float()[:, :, ::7] == 0).all())
    out = [torch.empty(1, T, H, D, dtype=BF16, device="cuda") for _ in range(2)]
    sq.paged_read(*pages, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"),
                  torch.tensor([T], dtype=torch.int32, device="cuda"), *out, s, s)
    for x, o in zip(pages, out):
        codes = x.cpu().view(torch.uint8)[i // page, :, i % page].view(E4M3)
        assert torch.equal(o[0].cpu().double(), codes.double() * s.cpu().double().view(1, H, 1))
