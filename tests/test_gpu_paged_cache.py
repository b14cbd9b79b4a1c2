"""Appending to a paged cache and copying its pages.

Stored keys and values and copied pages are exact.  A pooled key is a
compensated fp32 sum of bf16 values in three levels and one division: each level
errs by at most 2 u of the sum of magnitudes (u = 2^-24), the division by u, so
|error| <= 8 u mean|k|."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_sparse_moba_gb300 import build
    build.build()
    ops.lib()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Cache:
    """Pools with shuffled pages for sequences of up to `most` tokens, NaN wherever nothing is written."""

    def __init__(self, seqs, most, hkv, d, page, block, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.page, self.block = page, block
        self.mp = -(-most // page)
        self.P = seqs * self.mp + 3
        order = torch.randperm(self.P, generator=g)[:seqs * self.mp]
        self.table = order.view(seqs, self.mp).to("cuda", torch.int32)
        self.k = torch.full((self.P, hkv, page, d), float("nan"), dtype=BF, device="cuda")
        self.v = self.k.clone()
        self.kbar = torch.full((self.P, hkv, d), float("nan"), device="cuda")

    def append(self, k, v, cu, lens, pooling=ops.POOL_MEAN, **kw):
        ops.paged_append(k, v, self.k, self.v, self.kbar, self.table, i32(cu), i32(lens),
                         max(b - a for a, b in zip(cu, cu[1:])) or 1, self.block, pooling=pooling, **kw)

    def read(self, pool, b, length):
        p = torch.arange(length, device="cuda")
        return pool[self.table[b, p // self.page].long(), :, p % self.page]


def normal(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(BF)


@pytest.mark.parametrize("hkv,d,page,block", [(1, 64, 16, 64), (3, 128, 32, 128), (2, 64, 64, 64),
                                              (4, 128, 128, 512), (2, 128, 16, 192)])
@pytest.mark.parametrize("pooling", [ops.POOL_MEAN, ops.POOL_MAX])
def test_append_in_uneven_chunks(hkv, d, page, block, pooling):
    lens = [700, 1, 64, 513, 0, 1024]
    steps = [[1, 1, 0, 200, 0, 63], [299, 0, 64, 1, 0, 1], [0, 0, 0, 310, 0, 449], [400, 0, 0, 2, 0, 511]]
    ks, vs = [normal(b, L, hkv, d) for b, L in enumerate(lens)], [normal(50 + b, L, hkv, d) for b, L in enumerate(lens)]
    c = Cache(len(lens), 1024, hkv, d, page, block)
    at = [0] * len(lens)
    for step in steps:
        k = torch.cat([ks[b][at[b]:at[b] + n] for b, n in enumerate(step)])
        v = torch.cat([vs[b][at[b]:at[b] + n] for b, n in enumerate(step)])
        cu = [0]
        for b, n in enumerate(step):
            at[b] += n
            cu.append(cu[-1] + n)
        c.append(k, v, cu, at, pooling)
    assert at == lens and ops.get_status() == ops.MOBA_OK
    one = Cache(len(lens), 1024, hkv, d, page, block)
    cu = [0]
    for L in lens:
        cu.append(cu[-1] + L)
    one.append(torch.cat(ks), torch.cat(vs), cu, lens, pooling)
    written = torch.zeros(c.P, page, dtype=torch.bool, device="cuda")
    slots = torch.zeros(c.P, dtype=torch.bool, device="cuda")
    for b, L in enumerate(lens):
        if L:
            assert torch.equal(c.read(c.k, b, L), ks[b]) and torch.equal(c.read(c.v, b, L), vs[b])
            p = torch.arange(L, device="cuda")
            written[c.table[b, p // page].long(), p % page] = True
        for blk in range(L // block):
            slot = int(c.table[b, (blk + 1) * block // page - 1])
            slots[slot] = True
            x = ks[b][blk * block:(blk + 1) * block].double()
            if pooling == ops.POOL_MAX:
                assert torch.equal(c.kbar[slot].double(), x.amax(0))
            else:
                err = (c.kbar[slot].double() - x.mean(0)).abs()
                assert (err <= 8 * 2.0 ** -24 * x.abs().mean(0)).all()
    # nothing else was written, and the cuts made no difference
    for pool in (c.k, c.v):
        assert pool.transpose(1, 2)[~written].isnan().all()
    assert c.kbar[~slots].isnan().all()
    for x, y in ((c.k, one.k), (c.v, one.v)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert torch.equal(c.kbar.view(torch.int32), one.kbar.view(torch.int32))


@pytest.mark.parametrize("where", [0, 17, 39])
def test_append_of_steps_beside_a_long_chunk(where):
    n, block = 40, 64
    lens = [63 + 7 * b for b in range(n)]
    nq = [1 + b % 2 for b in range(n)]
    lens[where], nq[where] = 1500, 1401
    c, page = Cache(n, 1536, 2, 64, 16, block), 16
    cu = [0]
    for m in nq:
        cu.append(cu[-1] + m)
    old = [normal(b, L, 2, 64) for b, L in enumerate(lens)]
    start = [0]
    for L, m in zip(lens, nq):
        start.append(start[-1] + L - m)
    before = torch.cat([k[:L - m] for k, L, m in zip(old, lens, nq)])
    c.append(before, before, start, [L - m for L, m in zip(lens, nq)])
    new = torch.cat([k[L - m:] for k, L, m in zip(old, lens, nq)])
    c.append(new, -new, cu, lens)
    assert ops.get_status() == ops.MOBA_OK
    one = Cache(n, 1536, 2, 64, page, block)
    full = [0]
    for L in lens:
        full.append(full[-1] + L)
    one.append(torch.cat(old), torch.cat(old), full, lens)
    assert torch.equal(c.k.view(torch.int16), one.k.view(torch.int16))
    assert torch.equal(c.kbar.view(torch.int32), one.kbar.view(torch.int32))
    for b, (L, m) in enumerate(zip(lens, nq)):
        assert torch.equal(c.read(c.v, b, L)[L - m:], -old[b][L - m:])
    # a refused sequence beside them is recorded, the others stand
    wrong = list(lens)
    wrong[3 if where else 4] = 0
    c.append(new, new, cu, wrong)
    assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    for b, (L, m) in enumerate(zip(wrong, nq)):
        if L:
            assert torch.equal(c.read(c.v, b, L)[L - m:], old[b][L - m:])
    # offsets that decrease are recorded too
    c.append(new, new, [0] * 5 + [-1] * (n - 4), [9] * n)
    assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG


def test_append_without_pooled_keys_and_padding_rows():
    c = Cache(2, 128, 2, 64, 16, 64)
    k, v = normal(1, 200, 2, 64), normal(2, 200, 2, 64)
    ops.paged_append(k, v, c.k, c.v, None, c.table, i32([0, 100, 130]), i32([100, 30]), 100, 64)
    assert torch.equal(c.read(c.k, 0, 100), k[:100]) and torch.equal(c.read(c.v, 1, 30), v[100:130])
    assert int((~c.k.isnan()).all(-1).sum()) == 130 * 2 and c.kbar.isnan().all()
    assert ops.get_status() == ops.MOBA_OK


def test_append_refuses_bad_sequences_and_pages_on_the_device():
    c = Cache(4, 128, 1, 64, 16, 64)
    k, v = normal(3, 40, 1, 64), normal(4, 40, 1, 64)
    # the first: more new tokens than its length; the third: longer than its pages; the others stand
    ops.paged_append(k, v, c.k, c.v, c.kbar, c.table, i32([0, 10, 20, 30, 40]), i32([9, 10, 129, 64]), 10, 64)
    assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    assert torch.equal(c.read(c.k, 1, 10), k[10:20]) and torch.equal(c.read(c.k, 3, 64)[54:], k[30:])
    assert int((~c.k.isnan()).all(-1).sum()) == 20
    # rows outside the tensors, decreasing offsets, more than max_new
    before = c.k.clone()
    for cu in ([0, 10, 50, 50, 50], [-5, 0, 0, 0, 0], [30, 20, 20, 20, 20], [0, 11, 11, 11, 11]):
        ops.paged_append(k, v, c.k, c.v, c.kbar, c.table, i32(cu), i32([0 if cu[0] == 30 else 20, 64, 64, 64]), 10, 64)
        assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    changed = (c.k.view(torch.int16) != before.view(torch.int16)).any(-1).sum()
    assert int(changed) <= 10  # the one good first sequence of the first table
    # a page outside the pool: its tokens are left out, and its block is not pooled
    c = Cache(1, 64, 1, 64, 16, 64)
    for wrong in (-1, c.P, 2 ** 31 - 1):
        table = c.table.clone()
        table[0, 2] = wrong
        ops.paged_append(normal(5, 64, 1, 64), normal(6, 64, 1, 64), c.k, c.v, c.kbar, table, i32([0, 64]), i32([64]),
                         64, 64)
        assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
        assert int((~c.k.isnan()).all(-1).sum()) == 48 and c.kbar.isnan().all()


@pytest.mark.parametrize("layers,hkv,d,page,n,bar", [(None, 1, 64, 16, 1, True), (3, 2, 128, 64, 17, True),
                                                     (1, 8, 128, 16, 300, True), (2, 3, 64, 32, 5, False)])
def test_page_copy(layers, hkv, d, page, n, bar):
    P = 3 * n + 2
    lead = () if layers is None else (layers,)
    k, v = normal(1, *lead, P, hkv, page, d), normal(2, *lead, P, hkv, page, d)
    kbar = torch.randn(*lead, P, hkv, d, device="cuda") if bar else None
    order = torch.randperm(P, generator=torch.Generator().manual_seed(3)).to("cuda", torch.int32)
    src, dst = order[:n].contiguous(), order[n:2 * n].contiguous()
    src[-1] = src[0]  # one page may go to several
    want = [None if x is None else x.clone() for x in (k, v, kbar)]
    for w in want:
        if w is not None:
            w[(slice(None),) * len(lead) + (dst.long(),)] = w[(slice(None),) * len(lead) + (src.long(),)]
    ops.page_copy(k, v, kbar, src, dst)
    assert ops.get_status() == ops.MOBA_OK
    for x, w in zip((k, v, kbar), want):
        assert w is None or torch.equal(x, w)


def test_page_copy_refuses_pairs_that_clash():
    k, v = normal(1, 12, 2, 16, 64), normal(2, 12, 2, 16, 64)
    kbar = torch.randn(12, 2, 64, device="cuda")
    want = [x.clone() for x in (k, v, kbar)]
    #      good    outside                    same dst twice    src is a dst   onto itself
    src = [0,      1,  12, -1, 2,  2 ** 30,   3, 4,             7,             9]
    dst = [6,      12, 7,  8,  -7, 10,        11, 11,           5,             9]
    ops.page_copy(k, v, kbar, i32(src), i32(dst))
    assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    for x, w in zip((k, v, kbar), want):
        w[6] = w[0]
        assert torch.equal(x, w)
