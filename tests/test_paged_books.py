"""The books of the paged cache (no GPU): every sequence keeps its tokens through
sharing, copying on write, cutting back, leaving and compaction."""
import random

import pytest

from long_context_sparse_moba_gb300.paged import OutOfPages, Pages


class Model:
    """Pages with their contents: what each token slot holds, moved as the books say."""

    def __init__(self, num_pages, page):
        self.books = Pages(num_pages, page)
        self.page = page
        self.slot = [[None] * page for _ in range(num_pages)]
        self.text = {}
        self.count = 0

    def move(self, pairs):
        src, dst = {a for a, _ in pairs}, [b for _, b in pairs]
        assert not src & set(dst) and len(set(dst)) == len(dst)
        for a, b in pairs:
            self.slot[b] = list(self.slot[a])

    def extend(self, counts):
        before = {s: self.books.length(s) for s in counts}
        self.move(self.books.extend(counts))
        written = set()
        for s, n in counts.items():
            pages = self.books.pages(s)
            for p in range(before[s], before[s] + n):
                self.count += 1
                at = (pages[p // self.page], p % self.page)
                assert at not in written  # no slot is written by two sequences
                written.add(at)
                self.slot[at[0]][at[1]] = self.count
                self.text[s].append(self.count)
        self.check()

    def check(self):
        owners = {}
        for s in self.books.sequences():
            pages, n = self.books.pages(s), self.books.length(s)
            assert len(pages) == -(-n // self.page) and n == len(self.text[s])
            assert [self.slot[pages[p // self.page]][p % self.page] for p in range(n)] == self.text[s]
            for p in pages:
                owners[p] = owners.get(p, 0) + 1
        assert self.books.free_pages == self.books.num_pages - len(owners)


@pytest.mark.parametrize("seed", range(6))
def test_random_lives(seed):
    rng = random.Random(seed)
    m = Model(60, rng.choice([1, 4, 16]))
    for _ in range(400):
        seqs = list(m.books.sequences())
        what = rng.random()
        if not seqs or what < 0.1:
            m.text[m.books.new()] = []
        elif what < 0.55:
            counts = {s: rng.choice([0, 1, 1, 1, 5, 40]) for s in rng.sample(seqs, rng.randint(1, len(seqs)))}
            state = [(s, m.books.pages(s), m.books.length(s)) for s in seqs], m.books.free_pages
            try:
                m.extend(counts)
            except OutOfPages:
                assert state == ([(s, m.books.pages(s), m.books.length(s)) for s in seqs], m.books.free_pages)
                victim = rng.choice(seqs)
                m.books.free(victim)
                del m.text[victim]
        elif what < 0.7:
            s = rng.choice(seqs)
            m.text[m.books.fork(s)] = list(m.text[s])
        elif what < 0.8:
            s = rng.choice(seqs)
            n = rng.randint(0, m.books.length(s))
            m.books.truncate(s, n)
            del m.text[s][n:]
        elif what < 0.9:
            s = rng.choice(seqs)
            m.books.free(s)
            del m.text[s]
        else:
            m.move(m.books.compact())
            live = {p for s in m.books.sequences() for p in m.books.pages(s)}
            assert live == set(range(len(live)))
        m.check()


def test_refusals():
    with pytest.raises(ValueError):
        Pages(0, 16)
    b = Pages(2, 16)
    s = b.new()
    with pytest.raises(ValueError):
        b.extend({s: -1})
    with pytest.raises(OutOfPages):
        b.extend({s: 33})
    assert b.free_pages == 2 and b.length(s) == 0
    assert b.extend({s: 32}) == []
    with pytest.raises(ValueError):
        b.truncate(s, 33)
    with pytest.raises(KeyError):
        b.length(99)
