"""Offsets that lead out of the tensors, or nowhere, in the attention of shared prefixes: what
becomes of every row, by the rules that the header states for them (tolerances as in
test_gpu_paged_shared)."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_attn import expect
from .test_gpu_paged_cache import BF, built, normal  # noqa: F401  (built: a fixture)
from .test_gpu_paged_shared import Forks

pytestmark = pytest.mark.gpu
GUARD = 70  # rows before and behind the results


def claims(cu, lens, rows, most):
    """Of each sequence the rows that it claims, and whether it is refused."""
    for lo, hi, length in zip(cu, cu[1:], lens):
        fine = 0 <= lo <= hi <= rows and hi - lo <= most
        if fine:
            yield range(lo, hi), hi - lo > length
        else:
            first = min(max(lo, 0), rows)
            yield range(first, min(max(hi, first), rows)), True


@pytest.mark.parametrize("scale", [1, 50])
@pytest.mark.parametrize("cu", [
    [-5, 2, 9, 10, 11, 15],                                   # out in front
    [9, 8, 7, 6, 5, 4],                                       # backwards: no rows at all
    [0, 10 ** 6, 3, 2 ** 31 - 1, -2 ** 31, 7],                # out behind, everything claimed
    [0, 2, 5, 6, 7, 10 ** 6],                                 # the last one alone
    [0, 2, 5, 4, 5, 8],                                       # backwards once, rows claimed twice
    [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0, 1, 4],
    [3, 3, 3, 3, 3, 3]])                                      # nobody has any: nothing is refused either
def test_every_row(cu, scale):
    groups = [(256, [(2 * scale, 150), (3 * scale, 200), (1, 1)]), (128, [(1, 30), (4, 9)])]
    f = Forks(groups, 2, 128, 32, seed=31, slack=1)
    rows, most = sum(f.nq) + 20, max(f.nq)
    q = normal(1, rows, 8, 128)
    outs = torch.full((rows + 2 * GUARD, 8, 128), 7.0, dtype=BF, device="cuda")
    lses = torch.full((rows + 2 * GUARD, 8), 7.0, device="cuda")
    out, lse = outs[GUARD:-GUARD], lses[GUARD:-GUARD]
    f.call(q, cu=cu, out=out, lse=lse)
    got = list(claims(cu, f.lens, rows, most))
    refused = any(bad for _, bad in got)
    assert ops.get_status() == (ops.MOBA_ERR_INVALID_ARG if refused else ops.MOBA_OK)
    for x in (outs, lses):
        assert (x[:GUARD] == 7).all() and (x[-GUARD:] == 7).all()
    backwards = any(a > b for a, b in zip(cu, cu[1:]))
    owners = [[b for b, (r, _) in enumerate(got) if i in r] for i in range(rows)]
    want = {}
    for b, (r, bad) in enumerate(got):
        if not bad and len(r):
            o, z, _, tol, ltol = expect(q[r.start:r.stop], [f.ks[b]], [f.vs[b]], f, [len(r)], [f.lens[b]], 1 << 20, 1)
            for i, row in enumerate(r):
                want[b, row] = o[i], z[i], tol[i], ltol[i]
    for i, who in enumerate(owners):
        untouched = bool((out[i] == 7).all() and (lse[i] == 7).all())
        cleared = bool((out[i] == 0).all() and (lse[i] == -float("inf")).all())
        if not who:
            assert untouched, i
        elif all(got[b][1] for b in who):
            assert cleared, i
        elif len(who) == 1:
            o, z, tol, ltol = want[who[0], i]
            right = bool(((out[i].double() - o).abs() <= tol).all() and ((lse[i].double() - z).abs() <= ltol).all())
            assert right or (backwards and untouched), i
        # (of rows that several claim the header promises nothing but that they are theirs)
