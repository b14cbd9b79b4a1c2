"""The paged operators together, as a server uses them, and beside the contiguous
paths of the library.  Tolerances as in test_gpu_paged_attn."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops
from long_context_sparse_moba_gb300.paged import OutOfPages, PagedCache

from .parity import LSE_MAX, OUT_MAX, OUT_MEAN
from .test_gpu_paged_attn import compare, expect
from .test_gpu_paged_cache import built, i32, normal  # noqa: F401  (built: a fixture)

pytestmark = pytest.mark.gpu


class Layer:
    """A cache's layer as `expect` reads it."""

    def __init__(self, cache, layer, batch):
        self.page, self.table, self.kbar = cache.books.page_size, batch.page_table, cache.kbar_pages[layer]


class Server:
    """A paged cache of two layers beside the plain history of every sequence."""

    def __init__(self, num_pages, hq, hkv, d, page, block, interleaved, topks):
        self.c = PagedCache(2, num_pages, hkv, d, page, block)
        for p in (self.c.k_pages, self.c.v_pages, self.c.kbar_pages):
            p.fill_(float("nan"))
        self.hq, self.hkv, self.d, self.block, self.topks = hq, hkv, d, block, topks
        self.interleaved = interleaved
        self.freqs = ops.rope_frequencies(d // 2, 10000.0, ops.ROPE_BANDS, factor=4.0, original_length=512)
        self.hist = {}  # (sequence, layer): [k rotated, v]
        self.seed = 0

    def new(self):
        s = self.c.new()
        for layer in range(2):
            self.hist[s, layer] = [torch.empty(0, self.hkv, self.d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
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
        nq, lens = [counts[s] for s in batch.seqs], [self.c.books.length(s) for s in batch.seqs]
        for layer in range(2):
            self.seed += 3
            q, k, v = (normal(self.seed + i, batch.total, h, self.d) for i, h in enumerate((self.hq, self.hkv, self.hkv)))
            topk = self.topks[layer]
            got = self.c.attend(layer, batch, q, k, v, topk, freqs=self.freqs, interleaved=self.interleaved,
                                magnitude=1.1, with_idx=True)
            q, k = ops.rope(q, k, batch.positions, self.freqs, self.interleaved, 1.1)
            row = 0
            for s, n in zip(batch.seqs, nq):
                h = self.hist[s, layer]
                self.hist[s, layer] = [torch.cat((h[0], k[row:row + n])), torch.cat((h[1], v[row:row + n]))]
                row += n
            ks, vs = ([self.hist[s, layer][i] for s in batch.seqs] for i in range(2))
            compare(got, expect(q, ks, vs, Layer(self.c, layer, batch), nq, lens, self.block, topk))
        assert ops.get_status() == ops.MOBA_OK


@pytest.mark.parametrize("hq,hkv,d,page,block,interleaved", [(8, 2, 128, 16, 64, False), (6, 2, 64, 32, 128, True)])
def test_a_server(hq, hkv, d, page, block, interleaved):
    # one layer selects blocks, the other attends to all of them
    s = Server(2400 // page, hq, hkv, d, page, block, interleaved, (3, 1000))
    a, b = s.new(), s.new()
    s.step({a: 300, b: 77})                     # prompts in chunks
    s.step({a: 213, b: 1})
    c, e = s.fork(a), s.fork(a)                 # the last page is partly filled
    s.step({c: 1, b: 1, a: 1})                  # everyone writes on
    s.step({a: 5, e: 70, c: 1})
    s.truncate(c, 400)                          # a rejected speculation, into a shared page
    s.step({c: 120, a: 1, b: 1})
    s.c.free(a)
    moved = s.c.compact()
    assert moved > 0
    s.step({b: 100, c: 1, e: 64})
    with pytest.raises(OutOfPages):
        s.step({b: 3000})
    s.step({b: 1, c: 1, e: 1})
    for x in (b, c, e):
        s.c.free(x)
    assert s.c.books.free_pages == s.c.books.num_pages


@pytest.mark.parametrize("topk", [1, 3, 64])
def test_a_prompt_beside_the_contiguous_forward(topk):
    """A prompt through the paged path in two chunks, and through moba_attn_fwd.  The
    two order scores alike but for near ties of fp32: rows whose selections are equal
    are compared, and nearly all are."""
    n, h, d, block = 1500, 4, 128, 128
    q, k, v = (normal(i, n, h, d) for i in range(3))
    idx = torch.empty(1, n, h, topk, dtype=torch.int32, device="cuda")
    out, lse = ops.attn_fwd(q[None], k[None], v[None], block, topk, idx_out=idx)
    c = PagedCache(1, 40, h, d, 64, block)
    s = c.new()
    got = []
    for lo, hi in ((0, 700), (700, n)):
        batch = c.extend({s: hi - lo})
        # (the page table is cut to the pages in use: topk stands for the same blocks)
        got.append(c.attend(0, batch, q[lo:hi].contiguous(), k[lo:hi].contiguous(), v[lo:hi].contiguous(), topk,
                            with_idx=True))
    o, z, sel = (torch.cat([g[i] for g in got]) for i in range(3))
    same = (sel == idx[0]).all(-1)
    assert same.float().mean() > 0.999
    err = (o.float() - out[0].float()).abs()[same]
    assert err.max() <= OUT_MAX and err.mean() <= OUT_MEAN
    assert (z - lse[0].T)[same].abs().max() <= LSE_MAX


def test_a_decode_step_beside_the_contiguous_decode():
    lens, h, d, block, topk = [1000, 333, 64, 1], 4, 128, 128, 4
    S = 1024
    kc, vc, q = normal(1, 4, S, h, d), normal(2, 4, S, h, d), normal(3, 4, h, d)
    out, lse, idx = ops.decode_fwd(q, kc, vc, ops.kpool(kc, block), i32(lens), block, topk)
    c = PagedCache(1, 100, h, d, 32, block)
    seqs = [c.new() for _ in lens]
    pack = lambda x: torch.cat([x[b, :n] for b, n in enumerate(lens)])
    batch = c.extend(dict(zip(seqs, lens)))
    ops.paged_append(pack(kc), pack(vc), c.k_pages[0], c.v_pages[0], c.kbar_pages[0], batch.page_table, batch.cu_new,
                     batch.cache_lens, batch.max_new, block)
    o, z, sel = ops.paged_attn(q, c.k_pages[0], c.v_pages[0], c.kbar_pages[0], batch.page_table, i32(range(5)),
                               batch.cache_lens, 1, block, topk, with_idx=True)
    assert torch.equal(sel, idx)
    err = (o.float() - out.float()).abs()
    assert err.max() <= OUT_MAX and err.mean() <= OUT_MEAN and (z - lse).abs().max() <= LSE_MAX


def test_a_captured_decode_step_follows_the_tables():
    """One graph of rotation, append and attention, replayed as the sequences grow."""
    hq, hkv, d, page, block = 8, 2, 64, 16, 64
    c = PagedCache(1, 64, hkv, d, page, block)
    a, b = c.new(), c.new()
    first = c.extend({a: 100, b: 62})
    freqs = ops.rope_frequencies(d)
    ks, vs = normal(1, 162, hkv, d), normal(2, 162, hkv, d)
    _, _, _ = c.attend(0, first, normal(0, 162, hq, d), ks, vs, 3, freqs=freqs)
    table = torch.full((2, 12), -1, dtype=torch.int32, device="cuda")
    cu, lens, pos = i32([0, 1, 2]), i32([1, 1]), i32([0, 0])
    q, k, v = (torch.zeros(2, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    pools = c.k_pages[0], c.v_pages[0], c.kbar_pages[0]
    out, lse = torch.empty_like(q), torch.empty(2, hq, device="cuda")
    ws = torch.empty(ops.paged_attn_workspace_size(2, 2, 1, hq, hkv, d, page, 12, block, 3), dtype=torch.uint8,
                     device="cuda")
    qr, kr = torch.empty_like(q), torch.empty_like(k)

    def step():
        ops.rope(q, k, pos, freqs, q_out=qr, k_out=kr)
        ops.paged_append(kr, v, *pools, table, cu, lens, 1, block)
        ops.paged_attn(qr, *pools, table, cu, lens, 1, block, 3, out=out, lse=lse, workspace=ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    ref = PagedCache(1, 64, hkv, d, page, block)
    ra, rb = ref.new(), ref.new()
    ref.attend(0, ref.extend({ra: 100, rb: 62}), normal(0, 162, hq, d), ks, vs, 3, freqs=freqs)
    for i in range(40):
        batch = c.extend({a: 1, b: 1})
        table[:, :batch.page_table.shape[1]] = batch.page_table
        lens.copy_(batch.cache_lens)
        pos.copy_(batch.positions)
        for x, h, j in ((q, hq, 0), (k, hkv, 1), (v, hkv, 2)):
            x.copy_(normal(1000 + 3 * i + j, 2, h, d))
        g.replay()
        o, z, _ = ref.attend(0, ref.extend({ra: 1, rb: 1}), q, k, v, 3, freqs=freqs)
        assert torch.equal(out, o) and torch.equal(lse, z), i
    assert ops.get_status() == ops.MOBA_OK
