"""Branches of the paged kernels that only large counts take.  Tolerances as in
test_gpu_paged_attn and test_gpu_paged_cache."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_attn import case
from .test_gpu_paged_cache import Cache, built, normal  # noqa: F401  (built: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("topk", [8, 15, 16, 17, 32])
@pytest.mark.parametrize("hq,hkv,d,page,block", [(4, 2, 64, 16, 64), (6, 2, 128, 32, 128)])
def test_many_selected_blocks_in_a_chunk(hq, hkv, d, page, block, topk):
    """Seven to 31 past blocks a row, of up to 70."""
    case([300, 1, 131], [70 * block + 17, 40 * block, 33 * block - 1], hq, hkv, d, page, block, topk, seed=topk)


@pytest.mark.parametrize("n", [2, 300])
def test_more_past_blocks_than_are_counted_in_shared_memory(n):
    case([n], [64 * 1100 + 30], 4, 1, 64, 64, 64, 3, seed=n)


@pytest.mark.parametrize("pooling", [ops.POOL_MEAN, ops.POOL_MAX])
@pytest.mark.parametrize("seqs", [1, 12])
def test_appending_to_blocks_of_many_pages(pooling, seqs):
    """516 pages to a block: more than a CTA looks up at once."""
    page, block, hkv, d = 16, 16 * 516, 1, 64
    n = 2 * block + 5
    k, v = normal(1, n, hkv, d), normal(2, n, hkv, d)
    c, one = Cache(seqs, 3 * block, hkv, d, page, block), Cache(seqs, 3 * block, hkv, d, page, block)
    for cache, cuts in ((c, [0, 100, block - 1, block + 7, n]), (one, [0, n])):
        for lo, hi in zip(cuts, cuts[1:]):
            m = hi - lo
            cache.append(k[lo:hi].repeat(seqs, 1, 1), v[lo:hi].repeat(seqs, 1, 1), [i * m for i in range(seqs + 1)],
                         [hi] * seqs, pooling)
    assert ops.get_status() == ops.MOBA_OK
    assert torch.equal(c.kbar.view(torch.int32), one.kbar.view(torch.int32))
    for b in range(seqs):
        assert torch.equal(c.read(c.k, b, n), k) and torch.equal(c.read(c.v, b, n), v)
        for blk in range(2):
            got = c.kbar[int(c.table[b, (blk + 1) * block // page - 1])].double()
            x = k[blk * block:(blk + 1) * block].double()
            if pooling == ops.POOL_MAX:
                assert torch.equal(got, x.amax(0))
            else:
                assert ((got - x.mean(0)).abs() <= 8 * 2.0 ** -24 * x.abs().mean(0)).all()
