"""Calls of the paged cache's operators in other settings: values that are not finite in queries,
another stream by argument, one workspace behind two graphs, tables far wider than their
sequences, slopes of both signs, repeated calls."""
import pytest
import torch

import block_ref as R
import paged_ref as P
from paged_ref import BF16, E4M3, F16
from test_gpu_norm_rotary import angles, heads
from test_gpu_paged_attention import check, kind, queries, run, starts_of  # noqa: F401 (kind: a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_post_quantized_smooth_amd as sq
    return sq


@pytest.mark.parametrize("n", [2, 150])
def test_queries_that_are_not_finite_stay_in_their_rows(sq, kind, n):
    dtype, coded = kind
    held, new = [200, 300], [n, 1]
    p = P.Pool(held, 2, 64, dtype, coded, 16).poison_free().cuda()
    q = queries(n + 1, 4, 64, dtype)
    odd = torch.zeros(n + 1, 4, dtype=torch.bool)
    for i, (t, h, x) in enumerate(((0, 1, float("nan")), (n - 1, 2, float("inf")), (n, 0, float("-inf")))):
        q[t, h, 5 + i] = x
        odd[t, h] = True
    got = run(sq, q, p, starts_of(new))
    # an infinite query meets keys of both signs, and so an infinite score: no average exists
    assert bool(torch.isnan(got.cpu()[odd]).all())
    ref, bound, _ = P.attention(q, p, starts_of(new), held, 64 ** -0.5)
    R.assert_within(got.cpu()[~odd], ref[~odd], bound[~odd])


@pytest.mark.parametrize("width", [7, 128])
def test_wide_tables(sq, kind, width):
    """Tables of 448 and 8192 places for sequences of up to 333: work is laid out for the longest
    that the table could hold, nothing is cut, and the result is the narrow table's."""
    dtype, coded = kind
    held, new = [333, 40, 0, 64], [1, 1, 0, 1]
    p = P.Pool(held, 2, 128, dtype, coded, 64, width=6).poison_free().cuda()
    q = queries(3, 8, 128, dtype)
    want = check(sq, q, p, starts_of(new))
    p.tables = torch.nn.functional.pad(p.tables, (0, width - 6), value=-1).contiguous()
    p.width = width
    assert torch.equal(check(sq, q, p, starts_of(new)), want)


@pytest.mark.parametrize("new", [[1, 3], [140, 3]])
def test_slopes_of_both_signs(sq, kind, new):
    dtype, coded = kind
    p = P.Pool([300, 90], 2, 64, dtype, coded, 16).poison_free().cuda()
    s = torch.tensor([-0.05, 0.0, 0.25, -0.01], device="cuda")
    check(sq, queries(sum(new), 4, 64, dtype), p, starts_of(new), slopes=s)


def test_repeated_calls_are_the_same_bits(sq, kind):
    dtype, coded = kind
    held, new = [3000, 900, 700], [1, 200, 2]
    p = P.Pool(held, 2, 128, dtype, coded, 64).poison_free().cuda()
    q = queries(sum(new), 8, 128, dtype)
    want = run(sq, q, p, starts_of(new))
    for _ in range(5):
        torch.randn(1024, 1024, device="cuda")                     # other memory for the workspace
        assert torch.equal(run(sq, q, p, starts_of(new)), want)


def test_two_graphs_of_one_workspace(sq):
    """Replayed in turn on one stream: each call writes what its join reads."""
    ps = [P.Pool([3000, 700, 90], 2, 128, BF16, c, 64, seed=int(c)).cuda() for c in (True, False)]
    starts = [[0, 1, 2, 3], [0, 1, 41, 43]]
    qs = [queries(s[-1], 8, 128, BF16, i) for i, s in enumerate(starts)]
    need = [sq.paged_attention_workspace_bytes(s[-1], 3, p.width * 64, 8, 2, 128) for s, p in zip(starts, ps)]
    assert min(need) > 0
    ws = torch.zeros(max(need), dtype=torch.uint8, device="cuda")
    want = [run(sq, q, p, s) for q, p, s in zip(qs, ps, starts)]
    dev = [torch.tensor(s, dtype=torch.int32, device="cuda") for s in starts]
    outs = [torch.empty_like(w) for w in want]
    graphs = [torch.cuda.CUDAGraph() for _ in ps]
    for g, q, p, s, o in zip(graphs, qs, ps, dev, outs):
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            sq.paged_attention(q, p.k, p.v, p.tables, p.lengths, s, o, p.ks, p.vs, ws=ws)
    for i in (0, 1, 1, 0, 1, 0, 0):
        for o in outs:
            o.fill_(9.0)
        torch.cuda.synchronize()
        graphs[i].replay()
        graphs[1 - i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("coded", [False, True])
def test_all_four_on_a_given_stream(sq, coded):
    """stream=: the work waits for that stream's, not the current one's."""
    T, Hq, Hkv, D, page = 70, 8, 2, 128, 16
    q, k, v = heads(T, Hq, D, BF16), heads(T, Hkv, D, BF16, 1), heads(T, Hkv, D, BF16, 2)
    pos, f, a = angles(sq, T, D)
    tables = torch.tensor([[4, 1, 3, 0, 2]], dtype=torch.int32, device="cuda")
    lengths, starts = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([T], [0, T]))
    j = torch.arange(T, device="cuda")
    slots = (tables[0].long()[j // page] * page + j % page).to(torch.int32)

    def everything(stream):
        kp, vp = (torch.zeros(5, Hkv, page, D, device="cuda").to(E4M3 if coded else BF16) for _ in range(2))
        qo, ko, out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
        back = [torch.empty(1, T, Hkv, D, dtype=BF16, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        sq.norm_rotary(q, k, qo, ko, pos, f, eps=1e-6, stream=stream)
        sq.norm_rotary_write(q, k, v, qo, slots, kp, vp, positions=pos, freqs=f, eps=1e-6, stream=stream)
        sq.paged_write(ko, v, slots, kp, vp, stream=stream)
        sq.paged_read(kp, vp, tables, lengths, *back, stream=stream)
        sq.paged_attention(qo, kp, vp, tables, lengths, starts, out, stream=stream)
        if stream is None:
            torch.cuda.synchronize()
        else:
            stream.synchronize()
        return [qo, ko, *back, out]

    want = everything(None)
    for a, b in zip(want, everything(torch.cuda.Stream())):
        assert torch.equal(a, b)
