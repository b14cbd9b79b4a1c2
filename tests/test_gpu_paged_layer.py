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
