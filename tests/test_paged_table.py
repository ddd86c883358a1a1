"""The page table's bookkeeping and the refusals of the paged cache and its block, without a
GPU."""
import numpy as np
import pytest
import torch

import bit_post_quantized_smooth_amd as sq
from test_block_class import weights


def state(t):
    return [x.clone() for x in (t.tables, t.lengths, t.starts, t.slots, t.positions)] + [t.tokens]


def same(a, b):
    return all(torch.equal(x, y) if isinstance(x, torch.Tensor) else x == y for x, y in zip(a, b))


def check(t):
    """Every page is free or one sequence's; slots and positions are those of the step's tokens."""
    owned = [p for row in t.tables.tolist() for p in row if p >= 0]
    assert len(set(owned)) == len(owned) and not set(owned) & set(t._free) and len(owned) + len(t._free) == t.pages
    starts, lengths = t.starts.tolist(), t.lengths.tolist()
    assert starts[0] == 0 and starts[-1] == t.tokens
    for b in range(t.batch):
        n, held = starts[b + 1] - starts[b], lengths[b]
        assert held == t.length(b)
        row = t.tables[b].tolist()
        assert all(p >= 0 for p in row[:-(-held // t.page_size)]) and all(p == -1 for p in row[-(-held // t.page_size):])
        for i in range(n):
            pos = held - n + i
            assert t.positions[starts[b] + i] == pos
            assert t.slots[starts[b] + i] == row[pos // t.page_size] * t.page_size + pos % t.page_size
    assert bool((t.slots[t.tokens:] == -1).all())


def test_sequences_grow_and_end():
    t = sq.PageTable(3, 100, page_size=16, device="cpu")
    assert t.width == 7 and t.pages == 21 and t.step_tokens == 300
    for counts in ([20, 0, 16], [1, 1, 1], 1, [0, 40, 3], [60, 0, 0]):
        t.begin(counts)
        check(t)
    assert [t.length(b) for b in range(3)] == [82, 42, 21]
    t.release(0)
    t.begin([0, 1, 0])
    check(t)
    assert t.length(0) == 0 and t.starts.tolist() == [0, 0, 1, 1]
    t.begin([100, 57, 79])
    check(t)
    t.begin(0)
    check(t)
    assert t.tokens == 0


def test_what_does_not_fit_changes_nothing():
    t = sq.PageTable(2, 64, page_size=16, pages=5, step_tokens=50, device="cpu")
    t.begin([33, 10])
    before = state(t)
    for counts, match in (([40, 11], "step"), ([32, 0], "sequences of up to 64"), ([1, 30], "pages"), ([1, -1], "counts"),
                          ([1], "counts"), ([1, 2, 3], "counts"), (-1, "counts")):
        with pytest.raises(ValueError, match=match):
            t.begin(counts)
        assert same(before, state(t)) and [t.length(0), t.length(1)] == [33, 10]
    with pytest.raises(TypeError):
        t.begin([1.0, 2.0])
    t.begin([15, 6])
    check(t)


def test_no_step_begins_while_a_graph_is_captured(monkeypatch):
    t = sq.PageTable(2, 64, device="cpu")
    t.begin([3, 4])
    before = state(t)
    t.device = torch.device("cuda")
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="captured"):
        t.begin(1)
    t.device = torch.device("cpu")
    assert same(before, state(t)) and t.length(0) == 3
    t.begin(1)
    check(t)


@pytest.mark.parametrize("a", [dict(batch=0, capacity=5), dict(batch=2, capacity=0), dict(batch=2, capacity=50, page_size=24),
                               dict(batch=2, capacity=50, page_size=8), dict(batch=2, capacity=50, page_size=2048)])
def test_tables_refused(a):
    with pytest.raises(ValueError):
        sq.PageTable(**a, device="cpu")


def test_caches_refused():
    t = sq.PageTable(2, 64, device="cpu")
    c = sq.PagedKeyValueCache(t, 2, 32, torch.float8_e4m3fn, k_scales=[0.5, 1.0])
    assert c.k.shape == (2, 2, 64, 32) and c.k_scales.tolist() == [0.5, 1.0] and c.v_scales is None
    with pytest.raises(ValueError, match="dtype"):
        sq.PagedKeyValueCache(t, 2, 32, torch.float32)
    with pytest.raises(ValueError, match="16-bit"):
        sq.PagedKeyValueCache(t, 2, 32, torch.float16, v_scales=[1.0, 1.0])
    for bad in ([1.0], [1.0, 0.0], [1.0, -1.0], [1.0, float("nan")], [1.0, float("inf")]):
        with pytest.raises(ValueError, match="k_scales"):
            sq.PagedKeyValueCache(t, 2, 32, torch.float8_e4m3fn, k_scales=bad)


def make(**kw):
    return sq.AttentionBlock(np.ones(256, np.float32), *weights(), 4, 2, 32, device="cpu", **kw)


def test_block_refusals():
    X = torch.zeros(1, 3, 256, dtype=torch.float16)
    t = sq.PageTable(2, 64, step_tokens=8, device="cpu")
    c = sq.PagedKeyValueCache(t, 2, 32, torch.float16)
    block = make()
    t.begin([2, 2])
    with pytest.raises(ValueError, match="3 rows, the step has 4"):
        block(X, cache=c)
    with pytest.raises(ValueError, match="of up to 8"):
        block(torch.zeros(3, 3, 256, dtype=torch.float16), cache=c)
    t.begin([1, 1])
    for kw in (dict(prefix=torch.zeros(1, dtype=torch.int32)), dict(key_ranges=torch.zeros(1, 3, 2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="paged"):
            block(X, cache=c, **kw)
    with pytest.raises(ValueError, match="no rotation"):
        block(X, positions=torch.zeros(1, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="on a GPU"):
        block(X, cache=c)
    with pytest.raises(ValueError, match="paged"):
        make(rotary=sq.rotary_frequencies(32))(X, cache=c, positions=torch.zeros(1, 3, dtype=torch.int32))
    for kw, match in ((dict(head_gains=(np.ones(31), None)), "head_gains"), (dict(rotary=sq.rotary_frequencies(34)), "rotary"),
                      (dict(rotary=(np.ones((2, 2)), 1.0)), "rotary")):
        with pytest.raises(ValueError, match=match):
            make(**kw)


def test_positions_are_behind_those_held(monkeypatch):
    """The dense cache's next tokens turn by their places in the sequence."""
    from bit_post_quantized_smooth_amd import block as module
    for f in ("rmsnorm_quantize_fp8", "gemm_fp8", "quantize_act_fp8", "attention"):
        monkeypatch.setattr(module.api, f, lambda *a, **k: None)
    seen = []
    monkeypatch.setattr(module.paged, "norm_rotary", lambda *a, **k: seen.append(k["positions"]))
    block = make(rotary=sq.rotary_frequencies(32))
    cache = sq.KeyValueCache(2, 10, 2, 32, torch.float16, device="cpu")
    X = torch.zeros(2, 3, 256, dtype=torch.float16)
    block(X)
    block(X, cache=cache)
    block(X[:, :2], cache=cache)
    own = torch.arange(6, dtype=torch.int32).view(2, 3)
    block(X, positions=own)
    assert [p.tolist() for p in seen] == [[0, 1, 2] * 2, [0, 1, 2] * 2, [3, 4] * 2, list(range(6))]
    with pytest.raises(ValueError, match="positions"):
        block(X, positions=own[:1])
    make(head_gains=(None, np.ones(32)))(X)
    assert seen[-1] is None
