"""Sequences that a step lists without new tokens: they read nothing, so they neither save
reading nor come between those that do (books only)."""
from long_context_sparse_moba_gb300 import paged
from long_context_sparse_moba_gb300.paged import PagedCache, Pages


def forks(n, tokens=640, page=16):
    p = Pages(1000, page)
    a = p.new()
    p.extend({a: tokens})
    return p, [a] + [p.fork(a) for _ in range(n - 1)]


def test_one_active_fork_shares_with_nobody():
    p, (a, b, c) = forks(3)
    for counts in ({a: 1, b: 0, c: 0}, {a: 0, b: 0, c: 2}, {a: 0, b: 0, c: 0}):
        p.extend(counts)
        assert p.groups(counts) == []


def test_idle_sequences_lie_inside_a_run():
    p, (a, b, c, e) = forks(4)
    other = p.new()
    p.extend({other: 50})
    short = p.fork(a)
    p.truncate(short, 20)
    counts = {other: 0, a: 1, b: 0, short: 0, c: 2, e: 0}
    p.extend(counts)
    assert p.groups(counts) == [(1, 5, 640)]  # from a to c; the idle short one does not cut the prefix


def test_an_idle_stranger_between_forks():
    p, (a, b) = forks(2)
    other = p.new()
    p.extend({other: 300})
    counts = {a: 1, other: 0, b: 1}
    p.extend(counts)
    assert p.groups(counts) == [(0, 3, 640)]
    counts = {a: 1, other: 1, b: 1}
    p.extend(counts)
    assert p.groups(counts) == []


def test_savings_go_by_those_that_read(monkeypatch):
    c = PagedCache(1, 200, 2, 64, page_size=16, block_size=64, device="cpu")
    a = c.new()
    c.extend({a: 640})
    seqs = [a] + [c.fork(a) for _ in range(5)]
    saved = 640 * 2 * 64 * 4  # by each member but one
    monkeypatch.setattr(paged, "SHARED_BYTES", 2 * saved)
    assert c.extend({s: int(i < 2) for i, s in enumerate(seqs)}).cu_groups is None
    batch = c.extend({s: int(i % 2 == 0) for i, s in enumerate(seqs)})
    assert batch.cu_groups.tolist() == [0, 5] and batch.prefix_lens.tolist() == [640]
