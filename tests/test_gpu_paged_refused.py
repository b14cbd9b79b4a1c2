"""Every row of a refused sequence that lies inside the tensors is cleared (zero
outputs, -inf lse, -1 idx), however many rows its offsets give it, and the other
sequences stand.  Tolerances as in test_gpu_paged_attn."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_attn import compare, expect, filled
from .test_gpu_paged_cache import BF, built, i32, normal  # noqa: F401  (built: a fixture)

pytestmark = pytest.mark.gpu

# (new tokens, lengths, offsets as given, max_new as given, refused sequence)
FEW = {
    "more than max_new": ([3, 9, 1, 4], [200, 300, 150, 64], [0, 3, 12, 13, 17], 4, 1),
    "many more than max_new": ([1, 150, 1], [70, 300, 129], [0, 1, 151, 152], 1, 1),
    "from before the rows": ([7, 4, 2], [90, 200, 65], [-1000, 7, 11, 13], 4, 0),
    "to behind the rows": ([2, 4, 9], [90, 200, 65], [0, 2, 6, 5000], 4, 2),
    "length below its tokens": ([3, 4, 1], [90, 2, 65], [0, 3, 7, 8], 4, 1),
}
MANY = {
    "more than max_new": ([200, 700, 1, 130], [300, 1000, 1500, 900], [0, 200, 900, 901, 1031], 200, 1),
    "one more than max_new": ([130, 401, 90], [300, 1000, 640], [0, 130, 531, 621], 400, 1),
    "from before the rows": ([300, 200], [300, 1000], [-1000, 300, 500], 200, 0),
    "to behind the rows": ([200, 300], [900, 300], [0, 200, 9000], 200, 1),
    "length below its tokens": ([200, 90, 150], [300, 89, 900], [0, 200, 290, 440], 200, 1),
}


@pytest.mark.parametrize("topk", [1, 3, 100])
@pytest.mark.parametrize("hq,hkv,d,page,block", [(4, 2, 64, 16, 64), (12, 2, 128, 32, 128)])
@pytest.mark.parametrize("what,sizes", [(w, s) for s in (FEW, MANY) for w in s],
                         ids=lambda x: x.replace(" ", "_") if isinstance(x, str) else ("few" if x is FEW else "many"))
def test_all_rows_of_a_refused_sequence_are_cleared(what, sizes, hq, hkv, d, page, block, topk):
    nq, lens, cu, max_new, bad = sizes[what]
    real = [max(n, x) for n, x in zip(nq, lens)]
    c, ks, vs = filled(real, hkv, d, page, block, seed=len(what))
    total = sum(nq)
    q = normal(5, total + 30, hq, d)  # (30 rows of padding)
    want = expect(q[:total], ks, vs, c, nq, real, block, topk)
    if cu[-1] > total:  # the padding belongs to the refused sequence too
        clear = torch.arange(total + 30, device="cuda") >= cu[bad]
    else:
        clear = torch.zeros(total + 30, dtype=torch.bool, device="cuda")
        clear[max(cu[bad], 0):cu[bad + 1]] = True
    good = ~clear
    good[total:] = False
    out, lse = torch.full_like(q, 7.0), torch.full((total + 30, hq), 7.0, device="cuda")
    idx = torch.full((total + 30, hq, topk), 7, dtype=torch.int32, device="cuda")
    ops.paged_attn(q, c.k, c.v, c.kbar, c.table, i32(cu), i32(lens), max_new, block, topk, out=out, lse=lse, idx=idx)
    assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    assert (out[clear] == 0).all() and (lse[clear] == -float("inf")).all() and (idx[clear] == -1).all()
    compare((out[good], lse[good], idx[good]), [t[good[:total]] for t in want])
    rest = ~clear
    rest[:total] = False
    assert (out[rest] == 7).all() and (lse[rest] == 7).all() and (idx[rest] == 7).all()
