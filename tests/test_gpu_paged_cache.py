"""Writing keys and values into pages, 16 bits and e4m3, with and without the norm and the
rotation, and reading them back."""
import pytest
import torch

import block_ref as R
import paged_ref as P
from paged_ref import BF16, E4M3, F16, F64
from test_gpu_norm_rotary import angles, gains, heads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


def pool(pages, Hkv, page, D, dtype, seed=0):
    """(k, v) of random bytes' worth of values, (pages, Hkv, page, D)."""
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(pages, Hkv, page, D, generator=g).to(dtype).cuda() for _ in range(2)]


def slots_of(T, pages, page, seed=0, skip=()):
    g = torch.Generator().manual_seed(seed)
    s = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    for i, x in skip:
        s[i] = x
    return s


def at(pages, slots, page):
    """The rows (tokens x heads x D) of slots in the pool."""
    i = slots.long()
    return pages.cpu()[i // page, :, i % page] if pages.dtype != E4M3 else \
        pages.cpu().view(torch.uint8)[i // page, :, i % page].view(E4M3)


def check_written(pages, before, slots, page, ref, err, scale, dtype):
    """The rows at the slots are ref's, every other byte is what it was."""
    T = len(slots)
    keep = (slots >= 0) & (slots < pages.shape[0] * page)
    got = at(pages, slots[keep], page)
    if scale is not None:
        P.assert_codes(got, ref[keep], err[keep], scale.cpu().to(F64).view(-1, 1))
    else:
        P.assert_rounded(got, ref[keep], err[keep], dtype)
    a, b = pages.cpu().view(torch.uint8).clone(), before.cpu().view(torch.uint8)
    i = slots[keep].long()
    a[i // page, :, i % page] = b[i // page, :, i % page]
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("D,page", [(8, 16), (40, 16), (64, 32), (72, 64), (80, 16), (128, 16), (128, 256), (120, 1024)])
def test_plain_writes(sq, D, page, coded, dtype):
    T, Hkv, pages = 45, 3, 1024 // page + 3
    k, v = heads(T, Hkv, D, dtype, scale=2.0), heads(T, Hkv, D, dtype, 1)
    kp, vp = pool(pages, Hkv, page, D, E4M3 if coded else dtype)
    ks, vs = (torch.tensor([0.01, 0.02, 0.5], device="cuda"), torch.tensor([1.0, 0.011, 0.03], device="cuda")) if coded else (None, None)
    s = slots_of(T, pages, page, skip=[(0, -1), (7, pages * page), (8, 2 ** 31 - 1), (9, -(2 ** 31))])
    before = kp.clone(), vp.clone()
    sq.paged_write(k, v, s.cuda(), kp, vp, ks, vs)
    zero = torch.zeros(T, Hkv, D, dtype=F64)
    check_written(kp, before[0], s, page, k.cpu().to(F64), zero, ks, dtype)
    check_written(vp, before[1], s, page, v.cpu().to(F64), zero, vs, dtype)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,inter,norm", [
    (1, 20, 4, 64, 64, False, False), (8, 32, 8, 128, 128, False, True), (130, 6, 3, 72, 36, True, True),
    (77, 5, 5, 40, 20, False, True), (700, 24, 8, 128, 64, True, False)])
def test_fused_writes(sq, T, Hq, Hkv, D, R, inter, norm, coded, dtype):
    page, pages = 32, T // 32 + 3
    x = heads(T, Hq + 2 * Hkv, D, dtype)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    kp, vp = pool(pages, Hkv, page, D, E4M3 if coded else dtype)
    ks, vs = (0.02 + 0.01 * torch.arange(Hkv, device="cuda"), 0.5 + torch.rand(Hkv, device="cuda")) if coded else (None, None)
    s = slots_of(T, pages, page, skip=[(T - 1, -1)] if T > 1 else [])
    pos, f, a = angles(sq, T, R, scaling="parts", scale=4.0)
    gq, gk = gains(D) if norm else (None, None)
    kw = dict(positions=pos, freqs=f, factor=a, interleaved=inter, q_gain=gq, k_gain=gk, eps=1e-6 if norm else None)
    before = kp.clone(), vp.clone()
    qo = torch.full((T, Hq, D), 9.0, dtype=dtype, device="cuda")
    sq.norm_rotary_write(q, k, v, qo, s.cuda(), kp, vp, ks, vs, **kw)
    ref, err = P.heads(q, pos, f, a, inter, gq, kw["eps"])
    P.assert_rounded(qo, ref, err, dtype)
    ref, err = P.heads(k, pos, f, a, inter, gk, kw["eps"])
    check_written(kp, before[0], s, page, ref, err, ks, dtype)
    check_written(vp, before[1], s, page, v.cpu().to(F64), torch.zeros(T, Hkv, D, dtype=F64), vs, dtype)
    # the queries are those of the pass without pages; in place too
    q2, k2 = torch.empty_like(qo), torch.empty(T, Hkv, D, dtype=dtype, device="cuda")
    sq.norm_rotary(q, k, q2, k2, **kw)
    assert torch.equal(q2, qo)
    sq.norm_rotary_write(q, k, v, q, s.cuda(), kp, vp, ks, vs, **kw)
    assert torch.equal(q, qo)


def test_codes_at_the_edges(sq):
    """Every midpoint of neighbouring codes goes to the even one, beyond 448 is clamped, an
    infinity or NaN is the NaN code."""
    t = torch.from_numpy(R.e4m3_values()[:127])
    mid = ((t[1:] + t[:-1]) / 2).float()
    row = torch.zeros(128)
    row[:126] = mid
    row[126], row[127] = 448.0, 10000.0
    k = torch.stack([row, -row]).view(2, 1, 128).to(BF16)
    assert torch.equal(k[0, 0, :126].float(), mid)                 # midpoints have 5 bits: exact in bf16
    v = torch.tensor([float("inf"), float("-inf"), float("nan"), 500.0, -1e30, 2.0 ** -11, 0.0, -0.0] * 16).view(1, 1, 128)
    v = v.expand(2, 1, 128).to(BF16).contiguous()
    kp, vp = pool(1, 1, 16, 128, E4M3)
    sq.paged_write(k.cuda(), v.cuda(), torch.tensor([3, 4], dtype=torch.int32, device="cuda"), kp, vp)
    code = kp.cpu().view(torch.uint8)[0, 0]
    even = torch.arange(126) + torch.arange(126) % 2
    assert torch.equal(code[3, :126].long(), even) and torch.equal(code[4, :126].long(), even | 0x80)
    assert code[3, 126] == code[3, 127] == 0x7E and code[4, 127] == 0xFE
    code = vp.cpu().view(torch.uint8)[0, 0, 3, :8].tolist()
    assert all(c & 0x7F == 0x7F for c in code[:3]) and code[3:] == [0x7E, 0xFE, 0, 0, 0x80]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("D,page", [(8, 16), (40, 16), (64, 64), (72, 32), (128, 16), (128, 128)])
def test_reads(sq, D, page, coded, dtype):
    lengths = [1, 0, 130, page, page + 1, 77]
    p = P.Pool(lengths, 5, D, dtype, coded, page).cuda()
    L = 131
    k = torch.full((len(lengths), L, 5, D), 3.0, dtype=dtype, device="cuda")
    v = torch.full((len(lengths), 5, L, D), 3.0, dtype=dtype, device="cuda").transpose(1, 2)
    sq.paged_read(p.k, p.v, p.tables, p.lengths, k, v, p.ks, p.vs)
    for b, n in enumerate(lengths):
        n = min(n, L)
        rk, rv, there = p.dense(b, n)
        assert bool(there.all())
        zero = torch.zeros(n, 5, D, dtype=F64)
        for got, ref in ((k, rk), (v, rv)):
            P.assert_rounded(got[b, :n], ref, zero + 2.0 ** -24 * ref.abs(), dtype)
            assert bool((got[b, n:] == 3.0).all())


def test_reads_of_what_is_not_there(sq):
    """Lengths beyond the table or the output, pages outside the pool, no pages at all."""
    p = P.Pool([40, 40, 16], 2, 64, F16, False, 16).cuda()
    p.tables[1, 1] = p.k.shape[0]
    p.tables[2, 0] = -5
    lengths = torch.tensor([1000, 2 ** 31 - 1, 16], dtype=torch.int32, device="cuda")
    p.tables[0, 2] = 0
    k, v = (torch.full((3, 50, 2, 64), 3.0, dtype=F16, device="cuda") for _ in range(2))
    sq.paged_read(p.k, p.v, p.tables, lengths, k, v)
    rk, rv, there = p.dense(0, 48)
    assert torch.equal(k[0, :48].cpu().to(F64), rk) and bool((k[0, 48:] == 3.0).all())
    rk, rv, there = p.dense(1, 48)
    assert there.tolist() == [True] * 16 + [False] * 16 + [True] * 16
    assert torch.equal(v[1, :48].cpu().to(F64)[there], rv[there]) and bool((v[1, 16:32] == 3.0).all())
    assert bool((k[2] == 3.0).all())
    sq.paged_read(p.k[:0], p.v[:0], p.tables, lengths, k, v)
    sq.paged_read(p.k, p.v, p.tables[:, :0].contiguous(), lengths, k, v)
    assert torch.equal(k[0, :48].cpu().to(F64), p.dense(0, 48)[0])


@pytest.mark.parametrize("coded", [False, True])
def test_written_then_read(sq, coded):
    """Pages that hold both operands side by side (a stride of two pages), through a graph whose
    slots change between replays."""
    T, Hkv, D, page = 50, 3, 72, 16
    both = torch.zeros(8, 2, Hkv, page, D, dtype=E4M3 if coded else BF16, device="cuda")
    kp, vp = both[:, 0], both[:, 1]
    k, v = heads(T, Hkv, D, BF16), heads(T, Hkv, D, BF16, 1)
    ks = torch.full((Hkv,), 2.0 ** -6, device="cuda") if coded else None
    slots = torch.zeros(T, dtype=torch.int32, device="cuda")
    tables = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    lengths = torch.tensor([T], dtype=torch.int32, device="cuda")
    ko, vo = (torch.zeros(1, T, Hkv, D, dtype=BF16, device="cuda") for _ in range(2))
    sq.paged_write(k, v, slots.fill_(-1), kp, vp, ks, ks)          # nothing
    assert not bool(both.view(torch.uint8).any())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sq.paged_write(k, v, slots, kp, vp, ks, ks)
        sq.paged_read(kp, vp, tables, lengths, ko, vo, ks, ks)
    for order in ([0, 1, 2, 3], [7, 2, 5, 4], [1, 6, 0, 3]):
        tables.copy_(torch.tensor([order], dtype=torch.int32))
        j = torch.arange(T, device="cuda")
        slots.copy_(tables[0].long()[j // page] * page + j % page)
        for t in (both.view(torch.uint8), ko, vo):
            t.fill_(0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for got, x in ((ko, k), (vo, v)):
            if not coded:
                assert torch.equal(got[0], x)
            else:                                                  # a power of two: the code's error alone
                x = x.double().cpu()
                err = (got[0].double().cpu() - x).abs()
                assert bool((err <= 2.0 ** -4 * x.abs() + 2.0 ** -6 * 2.0 ** -10).all())


def test_rows_beyond_32_bits(sq):
    """A pool whose last pages lie more than 2^32 bytes behind its start."""
    free, _ = torch.cuda.mem_get_info()
    Hkv, D, page = 1, 8, 16
    stride = 1 << 25                                               # bytes from page to page, by strides alone
    pages = 140
    if free < 2 * pages * stride:
        pytest.skip("not enough memory")
    flat = [torch.zeros(pages * stride // 2, dtype=F16, device="cuda") for _ in range(2)]
    kp, vp = (x.as_strided((pages, Hkv, page, D), (stride // 2, page * D, D, 1)) for x in flat)
    k, v = heads(page, Hkv, D, F16), heads(page, Hkv, D, F16, 1)
    slots = torch.arange(page, dtype=torch.int32, device="cuda") + (pages - 1) * page
    sq.paged_write(k, v, slots, kp, vp)
    ko, vo = (torch.zeros(1, page, Hkv, D, dtype=F16, device="cuda") for _ in range(2))
    tables = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([page], dtype=torch.int32, device="cuda")
    sq.paged_read(kp, vp, tables, lengths, ko, vo)
    assert torch.equal(ko[0], k) and torch.equal(vo[0], v)
    q = heads(1, 2, D, F16, 2)
    out = torch.empty_like(q)
    sq.paged_attention(q, kp, vp, tables, lengths, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), out)
    x = (q[0].double() @ k[:, 0].double().t()) * D ** -0.5
    ref = torch.softmax(x, 1) @ v[:, 0].double()
    assert float((out[0].double() - ref).abs().max()) <= 4 * 2.0 ** -11 * float(v.abs().max())
