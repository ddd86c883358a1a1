"""Attention of new tokens over a paged cache against the fp64 formula: sequences of every
length side by side, types, heads, pages, masks, and what must not reach an output."""
import pytest
import torch

import block_ref as R
import paged_ref as P
from paged_ref import BF16, E4M3, F16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


def queries(T, Hq, D, dtype, seed=5):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, Hq, D, generator=g).to(dtype).cuda()


def run(sq, q, p, starts, ws=True, out=None, scale=None, lengths=None, **kw):
    T, Hq, D = q.shape
    out = torch.full_like(q, 9.0, memory_format=torch.contiguous_format) if out is None else out
    need = sq.paged_attention_workspace_bytes(T, len(starts) - 1, p.width * p.page, Hq, p.k.shape[1], D)
    work = torch.full((need // 4,), float("nan"), device="cuda") if ws and need else None
    s = torch.tensor(starts, dtype=torch.int32, device="cuda")
    sq.paged_attention(q, p.k, p.v, p.tables, p.lengths if lengths is None else lengths, s, out, p.ks, p.vs, scale=scale,
                       ws=work, **kw)
    return out


def check(sq, q, p, starts, ws=True, out=None, scale=None, lengths=None, **kw):
    got = run(sq, q, p, starts, ws, out, scale, lengths, **kw)
    held = p.lengths_list if lengths is None else lengths.tolist()
    ref, bound, owned = P.attention(q, p, starts, held, q.shape[2] ** -0.5 if scale is None else scale,
                                    kw.get("softcap", 0.0), kw.get("slopes"), kw.get("causal", True))
    R.assert_within(got[owned], ref[owned], bound[owned])
    if out is None:
        assert bool((got[~owned] == 9.0).all())
    return got


def starts_of(new, first=0):
    s = [first]
    for n in new:
        s.append(s[-1] + n)
    return s


CASES = [("f16", F16, False), ("bf16", BF16, False), ("f16 e4m3", F16, True), ("bf16 e4m3", BF16, True)]


@pytest.fixture(params=CASES, ids=[c[0] for c in CASES])
def kind(request):
    return request.param[1:]


@pytest.mark.parametrize("D", [8, 40, 64, 72, 80, 96, 120, 128])
def test_head_sizes(sq, kind, D):
    dtype, coded = kind
    held, new = [90, 33, 200], [70, 1, 3]
    p = P.Pool(held, 2, D, dtype, coded).cuda()
    check(sq, queries(sum(new), 4, D, dtype), p, starts_of(new))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 1024])
@pytest.mark.parametrize("causal", [True, False])
def test_pages(sq, kind, page, causal):
    """Sequences that end inside a page, at its end and behind it."""
    dtype, coded = kind
    held, new = [page - 1, page, page + 1, 2 * page + 5, 3], [1, 2, page // 2, 40, 3]
    p = P.Pool(held, 2, 64, dtype, coded, page).poison_free().cuda()
    check(sq, queries(sum(new), 2, 64, dtype), p, starts_of(new), causal=causal)


@pytest.mark.parametrize("n", [1, 2, 5, 31, 32, 33, 64, 127, 128, 129, 200])
def test_chunk_lengths(sq, kind, n):
    """Chunks at the end of longer sequences, whole prompts, and single tokens beside them."""
    dtype, coded = kind
    held, new = [n, n + 1, n + 63, n + 300, 500], [n, n, n, n, 1]
    p = P.Pool(held, 1, 128, dtype, coded, 32).poison_free().cuda()
    check(sq, queries(sum(new), 2, 128, dtype), p, starts_of(new))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (6, 2), (8, 1), (5, 1), (16, 4), (40, 1), (71, 1), (130, 1)])
def test_grouped_heads(sq, Hq, Hkv):
    held, new = [50, 77, 300], [20, 1, 1]
    for dtype, coded, D in ((BF16, True, 64), (F16, False, 128)):
        p = P.Pool(held, Hkv, D, dtype, coded, 32).cuda()
        check(sq, queries(sum(new), Hq, D, dtype), p, starts_of(new))


def test_rows_of_no_sequence(sq, kind):
    """Tokens before the first sequence and behind the last, sequences without tokens or keys."""
    dtype, coded = kind
    held, new = [40, 0, 17, 0, 90, 30], [3, 0, 0, 2, 33, 1]
    p = P.Pool(held, 2, 64, dtype, coded).poison_free().cuda()
    s = starts_of(new, 4)
    out = check(sq, queries(s[-1] + 6, 4, 64, dtype), p, s)
    assert bool((out[:4] == 9.0).all()) and bool((out[-6:] == 9.0).all())
    assert bool((out[s[3]:s[4]] == 0).all())           # two tokens of a sequence that holds nothing


def test_more_tokens_than_keys(sq, kind):
    """Rows before a sequence's first key see nothing and come out 0."""
    dtype, coded = kind
    p = P.Pool([5, 3], 2, 64, dtype, coded).cuda()
    out = check(sq, queries(160, 2, 64, dtype), p, [0, 150, 160])
    assert bool((out[:145] == 0).all()) and bool((out[150:157] == 0).all()) and bool((out[145:150] != 0).any())
    check(sq, queries(160, 2, 64, dtype), p, [0, 150, 160], causal=False)


@pytest.mark.parametrize("cap,slopes,scale", [(3.0, False, 0.5), (0.0, True, None), (20.0, True, None), (1e5, False, None),
                                              (0.0, False, 0.0), (0.0, False, -0.3), (30.0, False, 8.0)])
def test_cap_slopes_scale(sq, kind, cap, slopes, scale):
    dtype, coded = kind
    held, new = [333, 150, 64], [4, 140, 1]
    p = P.Pool(held, 2, 128, dtype, coded, 64).cuda()
    sl = torch.tensor([0.5, 0.1, 0.01, 1.0], device="cuda") if slopes else None
    check(sq, queries(sum(new), 4, 128, dtype), p, starts_of(new), scale=scale, softcap=cap, slopes=sl)


@pytest.mark.parametrize("held,new", [([5000], [1]), ([1], [1]), ([4097, 1, 700], [1, 1, 1]), ([3000, 2900], [40, 7]),
                                      ([2000, 10, 900], [300, 4, 1]), ([700] * 33, [1] * 33)])
@pytest.mark.parametrize("ws", [True, False])
def test_long_and_many(sq, kind, held, new, ws):
    """Enough keys that the work is split along them, with and without room for its parts."""
    dtype, coded = kind
    p = P.Pool(held, 2, 128, dtype, coded, 64).poison_free().cuda()
    check(sq, queries(sum(new), 8, 128, dtype), p, starts_of(new), ws=ws)


def test_more_sequences_than_a_wave(sq):
    """150 sequences of all lengths, some without tokens."""
    held = [(37 * i) % 190 + 1 for i in range(150)]
    new = [min(h, (5 * i) % 7 if i % 11 else 60) for i, h in enumerate(held)]
    p = P.Pool(held, 2, 64, BF16, True, 16).poison_free().cuda()
    check(sq, queries(sum(new), 4, 64, BF16), p, starts_of(new))


@pytest.mark.parametrize("B", [65, 130, 1000, 4200])
def test_large_batches(sq, B):
    """Single tokens of many short sequences, some empty, and two chunks among them."""
    held = [(11 * i) % 23 for i in range(B)]
    new = [1 if h and i % 9 else 0 for i, h in enumerate(held)]
    held[B // 2], new[B // 2], held[B - 1], new[B - 1] = 1500, 1, 300, 40
    p = P.Pool(held, 1, 64, BF16, True, 16).cuda()
    check(sq, queries(sum(new), 2, 64, BF16), p, starts_of(new))


def test_a_workspace_too_small_is_not_used(sq):
    p = P.Pool([3000, 900], 2, 64, F16, True, 64).cuda()
    q, s = queries(2, 4, 64, F16), torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    out, ws = torch.empty_like(q), torch.full((1024,), 0x5A, dtype=torch.uint8, device="cuda")
    assert sq.paged_attention_workspace_bytes(2, 2, p.width * 64, 4, 2, 64) > 1024
    sq.paged_attention(q, p.k, p.v, p.tables, p.lengths, s, out, p.ks, p.vs, ws=ws)
    assert torch.equal(out, run(sq, q, p, [0, 1, 2], ws=False)) and bool((ws == 0x5A).all())


@pytest.mark.parametrize("n", [1, 150])
def test_pages_outside_the_pool_are_not_seen(sq, kind, n):
    dtype, coded = kind
    p = P.Pool([400, 300], 2, 64, dtype, coded, 16).poison_free().cuda()
    p.tables[0, 3] = -1
    p.tables[0, 7:9] = p.k.shape[0]
    p.tables[0, 20] = 2 ** 31 - 1
    p.tables[0, 0] = -(2 ** 31)
    p.tables[1, :] = -1
    out = check(sq, queries(2 * n, 4, 64, dtype), p, [0, n, 2 * n])
    assert bool((out[n:] == 0).all())
    p.k, p.v = p.k[:0], p.v[:0]                         # a pool of no pages
    assert bool((run(sq, queries(2 * n, 4, 64, dtype), p, [0, n, 2 * n]) == 0).all())


def test_lengths_beyond_the_table(sq, kind):
    """Cut to the table's pages; below 0: nothing."""
    dtype, coded = kind
    p = P.Pool([64, 64, 64], 1, 64, dtype, coded, 16).cuda()
    q = queries(9, 2, 64, dtype)
    far = torch.tensor([2 ** 31 - 1, -3, 65], dtype=torch.int32, device="cuda")
    got = run(sq, q, p, [0, 3, 6, 9], lengths=far)
    want = run(sq, q, p, [0, 3, 6, 9], lengths=torch.tensor([64, 0, 64], dtype=torch.int32, device="cuda"))
    assert torch.equal(got, want) and bool((got[3:6] == 0).all())
    e = P.Pool([0], 1, 64, dtype, coded, 16).cuda()
    e.tables, e.width = e.tables[:, :0].contiguous(), 0
    assert bool((run(sq, q, e, [0, 9]) == 0).all())


@pytest.mark.parametrize("n", [1, 20, 160])
def test_hidden_keys_do_not_reach_an_output(sq, kind, n):
    """Later tokens of the chunk that are not a number, or infinite, change nothing before them;
    visible ones come out as the formula has them."""
    dtype, coded = kind
    held = 200 + n
    p = P.Pool([held, held], 2, 64, dtype, coded, 16).cuda()
    q = queries(2 * n, 4, 64, dtype)
    clean = run(sq, q, p, [0, n, 2 * n])
    for x in (p.k, p.v):                               # the first sequence's last key
        page, row = int(p.tables[0, (held - 1) // 16]), (held - 1) % 16
        P.Pool.poison(x[page, :, row])
    got = run(sq, q, p, [0, n, 2 * n])
    keep = torch.ones(2 * n, dtype=torch.bool)
    keep[n - 1] = False
    # Not bit for bit: the pass that is repeated for such values raises a row's reference at other
    # keys, and an exponential's argument x - m, |x - m| < 2^7, is rounded to 2^-17 of a base-2 logit
    # against each, which the bound's 4 * 2^-24 (2 + |top|) dx and the weights' half step both hold.
    ref, bound, _ = P.attention(q, p, [0, n, 2 * n], [held, held], 64 ** -0.5)
    R.assert_within(got, ref, bound)
    R.assert_within(clean[keep], ref[keep], bound[keep])
    assert bool(torch.isnan(got[n - 1]).all())
    if not coded:
        p = P.Pool([held], 2, 64, dtype, coded, 16).cuda()
        page, row = int(p.tables[0, (held - 1) // 16]), (held - 1) % 16
        p.v[page, 0, row, 3] = float("inf")
        p.v[page, 1, row, 4] = float("-inf")
        check(sq, q[:n], p, [0, n])


def test_sums_near_the_largest_value(sq):
    """Averages of values whose sum overflows, and weights that span far."""
    p = P.Pool([300], 1, 64, BF16, False, 16).cuda()
    p.v.copy_(3e38 * torch.sign(p.v.float()).to(BF16))
    p.k.zero_()
    for n in (1, 140):
        out = run(sq, queries(n, 2, 64, BF16), p, [0, n], causal=False)
        k, v, _ = p.dense(0)
        ref = v[:, 0].mean(0)
        assert float((out.cpu().double() - ref).abs().max()) <= 2.0 ** -7 * 3e38


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n", [1, 150])
def test_one_value_everywhere(sq, dtype, n):
    """A row's weights add up to 1: equal values average to themselves."""
    for coded in (False, True):
        p = P.Pool([n + 200], 2, 64, dtype, coded, 16, scales=False).cuda()
        p.v.copy_(torch.full(p.v.shape, 1.125).to(p.v.dtype))
        out = run(sq, 4 * queries(n, 4, 64, dtype), p, [0, n])
        assert bool((out.float() == 1.125).all())


def test_strides(sq, kind):
    dtype, coded = kind
    held, new = [70, 300], [60, 1]
    p = P.Pool(held, 2, 72, dtype, coded, 16).cuda()
    T = sum(new)
    x = queries(T, 9, 72, dtype)
    plain = check(sq, x[:, 2:6].contiguous(), p, starts_of(new))
    q = x[:, 2:6]
    out = torch.full((4, T, 80), 9.0, dtype=dtype, device="cuda")
    view = out[..., :72].transpose(0, 1)
    run(sq, q, p, starts_of(new), out=view)
    assert torch.equal(view, plain) and bool((out[..., 72:] == 9.0).all())
    # a pool of two layers
    both = torch.zeros(p.k.shape[0], 2, *p.k.shape[1:], dtype=p.k.dtype, device="cuda")
    both[:, 0].view(torch.uint8).copy_(p.k.view(torch.uint8)) if coded else both[:, 0].copy_(p.k)
    both[:, 1].view(torch.uint8).copy_(p.v.view(torch.uint8)) if coded else both[:, 1].copy_(p.v)
    p.k, p.v = both[:, 0], both[:, 1]
    assert torch.equal(run(sq, q, p, starts_of(new)), plain)


def test_codes_as_bytes(sq):
    p = P.Pool([90], 2, 64, F16, True, 16).cuda()
    q = queries(3, 4, 64, F16)
    want = check(sq, q, p, [0, 3])
    p.k, p.v = p.k.view(torch.uint8), p.v.view(torch.uint8)
    assert torch.equal(run(sq, q, p, [0, 3]), want)


def test_the_dense_operator_agrees(sq):
    """The same sequence through paged_read and attention()."""
    Hq, Hkv, D, n, held = 8, 2, 128, 100, 700
    p = P.Pool([held], Hkv, D, BF16, False, 64).cuda()
    q = queries(n, Hq, D, BF16)
    got = check(sq, q, p, [0, n])
    k, v = (torch.empty(1, held, Hkv, D, dtype=BF16, device="cuda") for _ in range(2))
    sq.paged_read(p.k, p.v, p.tables, p.lengths, k, v)
    out = torch.empty(1, n, Hq, D, dtype=BF16, device="cuda")
    sq.attention(q[None], k, v, out, causal=True)
    _, bound, _ = P.attention(q, p, [0, n], [held], D ** -0.5)
    assert bool(((out[0].double() - got.double()).abs().cpu() <= 2 * bound).all())


@pytest.mark.parametrize("coded", [False, True])
def test_a_graph_of_growing_sequences(sq, coded):
    """One graph, lengths, starts and tables changed between its replays, the workspace's memory
    overwritten, other work between: every replay is the eager call's bits."""
    held, Hkv, D = [2900, 700, 64, 0], 2, 128
    p = P.Pool([3000, 1000, 200, 200], Hkv, D, BF16, coded, 64).cuda()
    q = queries(150, 8, D, BF16)
    lengths = torch.tensor(held, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 1, 2, 3, 3], dtype=torch.int32, device="cuda")
    need = sq.paged_attention_workspace_bytes(150, 4, p.width * p.page, 8, Hkv, D)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    call = lambda o, w: sq.paged_attention(q, p.k, p.v, p.tables, lengths, starts, o, p.ks, p.vs, ws=w)  # noqa: E731
    call(out, ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call(out, ws)
    a = torch.randn(256, 256, device="cuda")
    for new, grown in (([1, 1, 1, 0], held), ([1, 1, 1, 1], [2901, 701, 65, 1]), ([100, 1, 0, 49], [3000, 702, 65, 50]),
                       ([1, 140, 3, 2], [10, 842, 68, 52])):
        lengths.copy_(torch.tensor(grown, dtype=torch.int32))
        starts.copy_(torch.tensor(starts_of(new), dtype=torch.int32))
        want = torch.full_like(q, 9.0)
        call(want, torch.full_like(ws, 0x7F))
        ref, bound, owned = P.attention(q, p, starts_of(new), grown, D ** -0.5)
        R.assert_within(want[owned], ref[owned], bound[owned])
        for _ in range(2):
            out.fill_(9.0)
            ws.fill_(0xA5)
            b = (a @ a).sum()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert bool(torch.isfinite(b)) and torch.equal(out, want)


def test_two_calls_at_once(sq):
    """On two streams with a workspace each."""
    ps = [P.Pool([4000, 900], 2, 128, BF16, True, 64, seed=i).cuda() for i in range(2)]
    qs = [queries(30, 8, 128, BF16, i) for i in range(2)]
    want = [run(sq, q, p, [0, 1, 30]) for q, p in zip(qs, ps)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, q, p in zip(streams, qs, ps):
        with torch.cuda.stream(s):
            got.append([run(sq, q, p, [0, 1, 30]) for _ in range(3)])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for outs, w in zip(got, want) for o in outs)
