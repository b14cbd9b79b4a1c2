"""Shared prefixes where scratch and groups are at their ends (tolerances as in
test_gpu_paged_shared)."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_cache import BF, built, i32, normal  # noqa: F401  (built: a fixture)
from .test_gpu_paged_shared import Forks, case, compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("members", [16, 17, 18])
def test_as_many_groups_for_the_tensor_cores_as_rows_allow(members):
    """Groups of one more row than a small span holds, each of them in a workspace of exactly
    the bytes asked for."""
    f = Forks([(4096, [(1, 1 + i % 3) for i in range(members)])] * 10, 8, 64, 64, seed=21)
    n = len(f.nq)
    q = normal(1, n, 8, 64)
    need = ops.paged_attn_shared_workspace_size(n, 10, n, 1, 8, 8, 64, 64, f.table.shape[1])
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    got = f.call(q, workspace=ws[:need])
    assert ops.get_status() == ops.MOBA_OK and (ws[need:] == 255).all()
    compare(got, f.expect(q))


def test_many_pairs_beside_one_large_group():
    case([(512, [(1, 1 + i % 5)] * 2) for i in range(120)] + [(16384, [(1, 2)] * 40)], 8, 8, 64, 64, seed=22)


@pytest.mark.parametrize("new", [1, 40])
def test_idle_members_inside_a_group(new):
    """Sequences without new tokens between the members, of other pages and lengths."""
    f = Forks([(512, [(new, new + 8), (0, 30), (new, new + 60)]), (64, [(0, 5)]), (512, [(1, 9)])], 2, 64, 16, seed=23)
    # behind the idle stranger another member of the first prefix
    f.rows[4] = f.rows[0][:32] + f.rows[4][32:]
    f.ks[4], f.vs[4] = (torch.cat((a[0][:512], a[4][512:])) for a in (f.ks, f.vs))
    f.table = i32([r + [-1] * (f.table.shape[1] - len(r)) for r in f.rows])
    q = normal(1, sum(f.nq), 8, 64)
    got = f.call(q, cu_groups=[0, 5], prefixes=[512])
    assert ops.get_status() == ops.MOBA_OK
    compare(got, f.expect(q))
