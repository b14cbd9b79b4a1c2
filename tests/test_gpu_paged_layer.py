"""A server's life with normalised queries and keys, and forks that are attended together:
PagedCache against the definition in 64 bits (tolerances as in test_gpu_paged_attn)."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops, paged
from long_context_sparse_moba_gb300.paged import PagedCache

from .test_gpu_paged_attn import compare, expect
from .test_gpu_paged_cache import BF, built, i32, normal  # noqa: F401  (built: a fixture)
from .test_gpu_paged_run import Layer

pytestmark = pytest.mark.gpu


class Server:
    """Two layers, one that selects blocks and one that attends to all, beside the plain
    history of every sequence."""

    def __init__(self, num_pages, hq, hkv, d, page, block, interleaved, norms):
        self.c = PagedCache(2, num_pages, hkv, d, page, block)
        for p in (self.c.k_pages, self.c.v_pages, self.c.kbar_pages):
            p.fill_(float("nan"))
        self.hq, self.hkv, self.d, self.block, self.interleaved = hq, hkv, d, block, interleaved
        self.freqs = ops.rope_frequencies(d // 2, 10000.0, ops.ROPE_BANDS, factor=4.0, original_length=512)
        self.norms = norms and tuple((1 + 0.3 * normal(s, d).float()).to(BF) for s in (1, 2))
        self.hist, self.seed, self.shared = {}, 10, 0

    def new(self):
        s = self.c.new()
        for layer in range(2):
            self.hist[s, layer] = [torch.empty(0, self.hkv, self.d, dtype=BF, device="cuda") for _ in range(2)]
        return s

    def fork(self, s):
        t = self.c.fork(s)
        for layer in range(2):
            self.hist[t, layer] = list(self.hist[s, layer])
        return t

    def truncate(self, s, n):
        self.c.truncate(s, n)
        for layer in range(2):
            self.hist[s, layer] = [x[:n] for x in self.hist[s, layer]]

    def step(self, counts):
        batch = self.c.extend(counts)
        self.shared += batch.cu_groups is not None
        nq, lens = [counts[s] for s in batch.seqs], [self.c.books.length(s) for s in batch.seqs]
        kw = dict(interleaved=self.interleaved, magnitude=1.1)
        for layer, topk in ((0, 3), (1, 1000)):
            self.seed += 1
            x = normal(self.seed, batch.total, self.hq + 2 * self.hkv, self.d)  # one projection
            q, k, v = x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:]
            if self.norms:
                got = self.c.attend(layer, batch, q, k, v, topk, freqs=self.freqs, norms=self.norms, eps=1e-5, **kw)
                q, k = ops.qk_norm_rope(q, k, *self.norms, batch.positions, self.freqs, eps=1e-5, **kw)
            else:
                got = self.c.attend(layer, batch, q, k, v.contiguous(), topk, freqs=self.freqs, **kw)
                q, k = ops.rope(q, k, batch.positions, self.freqs, self.interleaved, 1.1)
            row = 0
            for s, n in zip(batch.seqs, nq):
                h = self.hist[s, layer]
                self.hist[s, layer] = [torch.cat((h[0], k[row:row + n])), torch.cat((h[1], v[row:row + n]))]
                row += n
            ks, vs = ([self.hist[s, layer][i] for s in batch.seqs] for i in range(2))
            compare(got, expect(q, ks, vs, Layer(self.c, layer, batch), nq, lens, self.block, topk))
        assert ops.get_status() == ops.MOBA_OK


@pytest.mark.parametrize("norms", [True, False])
@pytest.mark.parametrize("hq,hkv,d,page,block,interleaved", [(8, 2, 128, 16, 64, False), (6, 2, 64, 32, 128, True)])
def test_a_server_with_forks(monkeypatch, hq, hkv, d, page, block, interleaved, norms):
    monkeypatch.setattr(paged, "SHARED_BYTES", 1 << 16)
    s = Server(3200 // page, hq, hkv, d, page, block, interleaved, norms)
    a, b = s.new(), s.new()
    s.step({a: 300, b: 77})
    s.step({a: 213, b: 1})
    c, e = s.fork(a), s.fork(a)
    s.step({a: 1, c: 1, e: 1, b: 1})            # three of them together, the last page copied by two
    s.step({b: 1, a: 2, c: 5, e: 1})
    f = s.fork(c)
    s.truncate(e, 400)
    s.step({a: 1, e: 3, c: 1, f: 1})
    s.step({c: 1, f: 9, a: 1, e: 1, b: 60})     # (more rows than pay: each by itself)
    s.c.free(a)
    assert s.c.compact() > 0
    s.step({e: 1, c: 1, f: 1, b: 1})
    assert s.shared >= 4


def test_a_captured_step_of_forks(monkeypatch):
    """Whose page table is rewritten between replays: each by itself, unless the graph is asked to
    take them together, with groups that are rewritten too."""
    monkeypatch.setattr(paged, "SHARED_BYTES", 1)
    c = PagedCache(1, 64, 2, 64, 16, 64)
    a, b = c.new(), c.new()
    lens = {a: 128, b: 160}
    hist = {}

    def step(counts, seed, run):
        batch = c.extend(counts)
        q, k, v = (normal(seed + i, batch.total, h, 64) for i, h in ((0, 8), (1, 2), (2, 2)))
        row = 0
        for s in batch.seqs:
            n = counts[s]
            old = hist.get(s, (k[:0], v[:0]))
            hist[s] = tuple(torch.cat((o, x[row:row + n])) for o, x in zip(old, (k, v)))
            row += n
        got = run(batch, q, k, v)
        ks, vs = ([hist[s][i] for s in batch.seqs] for i in range(2))
        compare(got, expect(q, ks, vs, Layer(c, 0, batch), [counts[s] for s in batch.seqs],
                            [c.books.length(s) for s in batch.seqs], 64, 1000))
        return batch

    eager = lambda batch, q, k, v: c.attend(0, batch, q, k, v, 1000)
    step(lens, 1, eager)
    forks = [c.fork(s) for s in (a, a, b, b)]
    for f, s in zip(forks, (a, a, b, b)):
        hist[f] = hist[s]
    pairs = [forks[:2], forks[2:]]
    first = step({s: 1 for s in pairs[0]}, 11, eager)
    assert first.cu_groups is not None
    for shared in (None, True):
        batch = c.extend({s: 1 for s in pairs[0]})
        assert batch.cu_groups is not None
        batch.page_table = torch.nn.functional.pad(batch.page_table, (0, 4), value=-1).contiguous()
        q, k, v = (normal(21 + i, 2, h, 64) for i, h in ((0, 8), (1, 2), (2, 2)))
        for i, s in enumerate(batch.seqs):
            hist[s] = tuple(torch.cat((o, x[i:i + 1])) for o, x in zip(hist[s], (k, v)))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = c.attend(0, batch, q, k, v, 1000, shared=shared)
        g.replay()

        def replay(new, q2, k2, v2):
            for x, y in ((q, q2), (k, k2), (v, v2), (batch.cu_new, new.cu_new), (batch.cache_lens, new.cache_lens)):
                x.copy_(y)
            batch.page_table.fill_(-1)
            batch.page_table[:, :new.page_table.shape[1]] = new.page_table
            if shared:
                batch.cu_groups.copy_(new.cu_groups)
                batch.prefix_lens.copy_(new.prefix_lens)
            g.replay()
            return got

        for i, pair in enumerate((pairs[1], pairs[0], pairs[1])):
            step({s: 1 for s in pair}, 31 + 3 * i, replay)
        assert ops.get_status() == ops.MOBA_OK
