"""Which sequences of a step share their past (books only), and what the cache makes of it
(no GPU: the calls are fakes)."""
import random

import pytest

from long_context_sparse_moba_gb300 import paged
from long_context_sparse_moba_gb300.paged import PagedCache, Pages


def test_forks_share_whole_pages_before_their_new_tokens():
    p = Pages(100, 16)
    a = p.new()
    p.extend({a: 100})
    b, c = p.fork(a), p.fork(a)
    assert p.shared_pages(a, b) == 7
    counts = {a: 1, b: 5, c: 1}
    p.extend(counts)  # the seventh page is partly filled: two of the three copy it
    assert p.shared_pages(a, b) <= 6 and p.groups(counts) == [(0, 3, 96)]
    d = p.new()
    p.extend({d: 40})
    counts = {a: 1, d: 1, b: 1, c: 1}
    p.extend(counts)
    assert p.groups(counts) == [(2, 4, 96)]  # neighbours only
    p.truncate(c, 50)
    counts = {b: 1, c: 30}
    p.extend(counts)
    assert p.groups(counts) == [(0, 2, 48)]  # c's new tokens begin in its fourth page
    e = p.fork(c)
    p.truncate(e, 10)
    counts = {c: 1, e: 1}
    p.extend(counts)
    assert p.groups(counts) == []


def test_a_group_ends_where_more_would_save_less():
    p = Pages(1000, 16)
    a = p.new()
    p.extend({a: 1600})
    forks = [p.fork(a) for _ in range(3)]
    far = p.fork(a)
    p.truncate(far, 160)
    counts = {s: 1 for s in [a, *forks, far]}
    p.extend(counts)
    assert p.groups(counts) == [(0, 4, 1600)]  # 300 pages saved; with far on 10 pages each, 40
    counts = {s: 1 for s in [far, a, *forks]}
    p.extend(counts)
    assert p.groups(counts)[0][0] == 0 and sum((j - i - 1) * n for i, j, n in p.groups(counts)) >= 160


def test_shared_pages_are_a_common_beginning():
    rng = random.Random(4)
    for _ in range(30):
        p = Pages(400, 16)
        seqs = [p.new()]
        p.extend({seqs[0]: 64})
        for _ in range(40):
            s = rng.choice(seqs)
            what = rng.random()
            if what < 0.3 and len(seqs) < 8:
                seqs.append(p.fork(s))
            elif what < 0.5 and p.length(s):
                p.truncate(s, rng.randrange(p.length(s)))
            else:
                p.extend({s: rng.randrange(1, 40)})
        for a in seqs:
            for b in seqs:
                x, y = p.pages(a), p.pages(b)
                n = p.shared_pages(a, b)
                assert x[:n] == y[:n] and not set(zip(range(n, 999), x[n:])) & set(zip(range(n, 999), y[n:]))


class Fakes:
    def __init__(self, monkeypatch):
        self.seen = []
        for name, result in (("rope", ("q", "k")), ("paged_append", None), ("paged_append_rope", Heads(4)), ("paged_attn", (1, 2, 3)),
                             ("paged_attn_shared", (4, 5))):
            monkeypatch.setattr(paged.ops, name, self.fake(name, result))

    def fake(self, name, result):
        def call(*a, **kw):
            self.seen.append((name, kw))
            return result
        return call


class Heads:
    def __init__(self, n):
        self.shape = (1, n, 64)


def forks(page=16, n=3, length=640):
    c = PagedCache(1, 200, 2, 64, page_size=page, block_size=64, device="cpu")
    a = c.new()
    c.extend({a: length})
    return c, [a] + [c.fork(a) for _ in range(n - 1)]


@pytest.mark.parametrize("stream", [None, "side"])
def test_the_calls_of_a_layer(monkeypatch, stream):
    monkeypatch.setattr(paged, "SHARED_BYTES", 1000)
    c, seqs = forks()
    batch = c.extend({s: 1 for s in seqs})
    assert batch.cu_groups.tolist() == [0, 3] and batch.prefix_lens.tolist() == [640]
    f = Fakes(monkeypatch)
    q, k = Heads(4), Heads(2)
    kw = {} if stream is None else {"stream": stream}
    assert c.attend(0, batch, q, k, "v", 99, freqs="f", norms=("wq", None), eps=1e-5, **kw) == (4, 5, None)
    assert [s[0] for s in f.seen] == ["paged_append_rope", "paged_attn_shared"]
    assert f.seen[0][1]["q_weight"] == "wq" and f.seen[0][1]["k_weight"] is None and f.seen[0][1]["eps"] == 1e-5
    assert all(s[1]["stream"] == stream for s in f.seen)
    # selection, an idx asked for, or many rows of a sequence: each by itself
    for args, more in (((3,), {}), ((99,), {"with_idx": True}), ((99,), {"workspace": "w"}), ((99,), {"shared": False})):
        f.seen.clear()
        assert c.attend(0, batch, q, k, "v", *args, **more, **kw) == (1, 2, 3)
        assert [s[0] for s in f.seen] == ["paged_append", "paged_attn"]
    f.seen.clear()
    assert c.attend(0, batch, Heads(130), k, "v", 99, **kw) == (1, 2, 3) and f.seen[-1][0] == "paged_attn"
    with pytest.raises(ValueError):
        c.attend(0, batch, q, k, "v", 99, norms=("wq", "wk"))


def test_batches_that_share_little_say_nothing():
    c, seqs = forks()
    assert c.extend({s: 1 for s in seqs}).cu_groups is None  # 1280 tokens of two heads of 64
    assert c.extend({seqs[0]: 1}).cu_groups is None


def test_sequences_between_groups(monkeypatch):
    monkeypatch.setattr(paged, "SHARED_BYTES", 1)
    c, seqs = forks()
    alone, more = c.new(), c.new()
    batch = c.extend({alone: 5, seqs[0]: 1, seqs[1]: 1, more: 2, seqs[2]: 1})
    assert batch.cu_groups.tolist() == [0, 1, 3] and batch.prefix_lens.tolist() == [0, 640]
