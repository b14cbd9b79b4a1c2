"""A step or a compaction whose copies cannot be enqueued leaves the cache as it was
(no GPU: the copies are fakes)."""
import copy
import random

import pytest

from long_context_sparse_moba_gb300 import paged
from long_context_sparse_moba_gb300.paged import OutOfPages, PagedCache, Pages


@pytest.fixture
def cache(monkeypatch):
    c = PagedCache(1, 12, 1, 64, page_size=16, block_size=64, device="cpu")
    c.calls = []

    def page_copy(k, v, kbar, src, dst):
        c.calls.append((src.tolist(), dst.tolist()))
        if c.fail:
            raise RuntimeError("moba_page_copy failed")

    c.fail = False
    monkeypatch.setattr(paged.ops, "page_copy", page_copy)
    return c


def state(books):
    return copy.deepcopy(vars(books))


def test_a_step_whose_copy_fails_changes_nothing(cache):
    a = cache.new()
    cache.extend({a: 40})
    b = cache.fork(a)
    before = state(cache.books)
    cache.fail = True
    with pytest.raises(RuntimeError):
        cache.extend({b: 30, a: 1})
    assert len(cache.calls) == 1 and state(cache.books) == before
    # the same step later is the step that it would have been
    cache.fail = False
    batch = cache.extend({b: 30, a: 1})
    assert cache.calls[0] == cache.calls[1]
    assert batch.cache_lens.tolist() == [70, 41] and cache.books.length(a) == 41


def test_a_step_whose_tables_fail_changes_nothing(cache, monkeypatch):
    a = cache.new()
    cache.extend({a: 5})
    before = state(cache.books)
    monkeypatch.setattr(PagedCache, "_ints", lambda self, x: (_ for _ in ()).throw(MemoryError()))
    with pytest.raises(MemoryError):
        cache.extend({a: 100})
    assert state(cache.books) == before


def test_a_compaction_whose_copy_fails_changes_nothing(cache):
    a, b = cache.new(), cache.new()
    cache.extend({a: 64, b: 40})
    cache.free(a)
    before = state(cache.books)
    cache.fail = True
    with pytest.raises(RuntimeError):
        cache.compact()
    assert cache.calls and state(cache.books) == before
    cache.fail = False
    assert cache.compact() == 3 and cache.books.pages(b) != tuple(before["_pages"][b])
    assert sorted(cache.books.pages(b)) == [0, 1, 2]


@pytest.mark.parametrize("seed", range(4))
def test_growth_taken_back(seed):
    rng = random.Random(seed)
    books = Pages(80, rng.choice([1, 4, 16]))
    for _ in range(300):
        seqs = list(books.sequences())
        what = rng.random()
        if not seqs or what < 0.1:
            books.new()
        elif what < 0.2:
            books.fork(rng.choice(seqs))
        elif what < 0.3:
            books.free(rng.choice(seqs))
        elif what < 0.4:
            s = rng.choice(seqs)
            books.truncate(s, rng.randint(0, books.length(s)))
        elif what < 0.45:
            before = state(books)
            pairs = books.compaction()
            assert state(books) == before and books.compact() == pairs
        else:
            counts = {s: rng.choice([0, 1, 1, 5, 20]) for s in rng.sample(seqs, rng.randint(1, len(seqs)))}
            before = state(books)
            try:
                copies = books.extend(counts)
            except OutOfPages:
                assert state(books) == before
                books.free(rng.choice(seqs))
                continue
            after = state(books)
            books.undo_extend(counts, copies)
            assert state(books) == before
            assert books.extend(counts) == copies and state(books) == after
