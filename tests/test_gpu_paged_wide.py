"""Page tables much wider than the sequences are long, as a captured step has them,
and many sequences: results as ever, at a cost that goes by the lengths.  Tolerances
as in test_gpu_paged_attn."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_attn import case, compare, expect, filled
from .test_gpu_paged_cache import built, i32, normal  # noqa: F401  (built: a fixture)

pytestmark = pytest.mark.gpu


def best_time(fn, n=20):
    """The fastest of n runs, in us."""
    for _ in range(3):
        fn()
    times = []
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        fn()
        b.record()
        b.synchronize()
        times.append(1e3 * a.elapsed_time(b))
    return min(times)


def test_a_wide_table_changes_neither_results_nor_cost():
    """64 decode steps beside a chunk; tables as wide as the sequences, and 2048 blocks wide
    (a million lists of a block and kv head, few of them in use)."""
    hq, hkv, d, page, block, topk = 8, 8, 64, 64, 64, 4
    lens = [300 + 11 * i for i in range(64)] + [1500]
    nq = [1] * 64 + [600]
    c, ks, vs = filled(lens, hkv, d, page, block, seed=1)
    q = normal(2, sum(nq), hq, d)
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    cu, ln = i32(cu), i32(lens)
    wide = torch.full((65, 2048), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    want = expect(q, ks, vs, c, nq, lens, block, topk)
    took = []
    for table in (c.table, wide):
        size = ops.paged_attn_workspace_size(65, q.shape[0], 600, hq, hkv, d, page, table.shape[1], block, topk)
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        call = lambda: ops.paged_attn(q, c.k, c.v, c.kbar, table, cu, ln, 600, block, topk, with_idx=True, workspace=ws)
        compare(call(), want)
        took.append(best_time(call))
    assert ops.get_status() == ops.MOBA_OK
    # the wide one has 4 MB of counters to clear, which is a few us
    assert took[1] <= 1.5 * took[0] + 20, took


@pytest.mark.parametrize("topk", [1, 3, 1000])
@pytest.mark.parametrize("where", [0, 1023, 1024, 1299])
def test_more_sequences_than_the_plan_has_threads(where, topk):
    n = 1300
    lens = [65 + (37 * i) % 200 for i in range(n)]
    nq = [(i * 7) % 3 for i in range(n)]
    lens[where], nq[where] = 900, 300
    case(nq, lens, 2, 1, 64, 16, 64, topk, seed=where, with_idx=topk < 100)


@pytest.mark.parametrize("hkv,block,length", [(1, 64, 64 * 4600 + 5), (3, 128, 128 * 1500 + 100)])
def test_more_lists_than_the_plan_takes_at_a_time(hkv, block, length):
    """Over 4096 lists of one sequence, and lists of several tiles beside it."""
    case([130, 1, 40], [length, 500, 20000], hkv, hkv, 64, 64, block, 5, seed=hkv)
