"""Masked attention over enough sequences and heads that the rows go in tiles of
128, a wave each 32 of them (fewer take 32, whose waves share the keys): the same
formula, masks and hidden values at sizes around both tiles' edges."""
import pytest
import torch

import block_ref as R
from test_gpu_attention import BF16, F16, check, qkv, run

pytestmark = pytest.mark.gpu
B = 16


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Lq,Lk,D,dtype", [(127, 63, 64, F16), (128, 129, 128, BF16), (129, 257, 72, F16),
                                           (260, 190, 128, F16), (190, 260, 40, BF16)])
def test_lengths(sq, Lq, Lk, D, dtype, causal):
    check(sq, *qkv(B, Lq, Lk, 16, 16, D, dtype), causal=causal)


@pytest.mark.parametrize("Hq,Hkv", [(16, 4), (30, 10)])
def test_grouped_heads_cap_and_slopes(sq, Hq, Hkv):
    q, k, v = qkv(B, 75, 210, Hq, Hkv, 128, BF16)
    sl = torch.logspace(-3, 0, Hq, device="cuda")
    check(sq, 4 * q, k, v, softcap=3.0, causal=True)
    check(sq, q, k, v, slopes=sl)
    check(sq, q, k, v, softcap=20.0, slopes=sl, causal=True)


def test_prefix(sq):
    q, k, v = qkv(B, 200, 230, 16, 16, 64, F16)
    p = torch.arange(0, 17 * B, 17, device="cuda", dtype=torch.int32)
    check(sq, q, k, v, causal=True, prefix=p)


def test_ranges(sq):
    """Unordered, empty, reversed and out-of-range intervals, per batch entry."""
    q, k, v = qkv(B, 200, 300, 16, 16, 128, F16)
    g = torch.Generator().manual_seed(5)
    r = torch.randint(-20, 330, (B, 200, 2), generator=g, dtype=torch.int32).cuda()
    for causal in (False, True):
        check(sq, q, k, v, key_ranges=r, causal=causal)


def test_documents(sq):
    q, k, v = qkv(B, 300, 300, 16, 16, 64, BF16)
    r = torch.from_numpy(sq.document_key_ranges([1, 63, 0, 64, 100, 2], 300)).cuda()
    out = check(sq, q, k, v, key_ranges=r)
    assert bool((out[:, 230:] == 0).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_hidden_infinities_and_nan(sq, dtype):
    """Keys 40 and on are hidden from the first rows of every sequence, and the last
    10 from all: what they hold reaches only the rows that see them."""
    q, k, v = qkv(B, 200, 230, 16, 16, 128, dtype)
    k[:, 220:] = float("nan")
    v[:, 220:] = float("inf")
    v[3, 40, 5, 7] = float("inf")
    v[4, 60, 2, 9] = float("nan")
    r = torch.zeros(1, 200, 2, dtype=torch.int32)
    r[0, :, 1] = torch.arange(21, 221)
    out = check(sq, q, k, v, key_ranges=r.cuda())
    assert bool(torch.isfinite(out[3, :19]).all()) and bool(torch.isinf(out[3, 20:, 5, 7]).all())


def test_both_row_tiles_agree(sq):
    """One sequence alone takes tiles of 32 rows, sixteen together tiles of 128."""
    q, k, v = qkv(B, 200, 230, 16, 16, 128, F16)
    whole = run(sq, q, k, v, causal=True)
    one = run(sq, q[:1], k[:1], v[:1], causal=True)
    ref, bound = R.attention(q[:1], k[:1], v[:1], 128 ** -0.5, causal=True)
    R.assert_within(one, ref, bound)
    R.assert_within(whole[:1], ref, bound)
