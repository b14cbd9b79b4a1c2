"""Steps without new tokens and copies of no page: nothing is done, results are empty."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops
from long_context_sparse_moba_gb300.paged import PagedCache

from .test_gpu_paged_cache import BF, built, i32, normal  # noqa: F401  (built: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("before", [0, 70])
def test_a_step_of_no_tokens(before):
    c = PagedCache(1, 16, 2, 64, 16, 64)
    a, b = c.new(), c.new()
    freqs = ops.rope_frequencies(64)
    step = lambda batch, **kw: c.attend(0, batch, normal(1, batch.total, 4, 64), normal(2, batch.total, 2, 64),
                                        normal(3, batch.total, 2, 64), 3, freqs=freqs, **kw)
    if before:
        step(c.extend({a: before}))
    pools = [x.clone() for x in (c.k_pages, c.v_pages, c.kbar_pages)]
    batch = c.extend({a: 0, b: 0})
    assert batch.total == 0 and c.books.length(a) == before and c.books.length(b) == 0
    out, lse, idx = step(batch, with_idx=True)
    assert out.shape == (0, 4, 64) and out.dtype == BF and lse.shape == (0, 4) and idx.shape == (0, 4, 3)
    assert step(batch)[2] is None
    given = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    assert step(batch, out=given)[0] is given
    with pytest.raises(ValueError):  # arguments are checked all the same
        step(batch, out=torch.empty(1, 4, 64, dtype=BF, device="cuda"))
    for x, y in zip(pools, (c.k_pages, c.v_pages, c.kbar_pages)):
        assert torch.equal(x, y)
    assert ops.get_status() == ops.MOBA_OK
    # the cache goes on
    out, _, _ = step(c.extend({a: 1, b: 2}))
    assert out.shape == (3, 4, 64) and out.isfinite().all() and ops.get_status() == ops.MOBA_OK


def test_the_calls_on_nothing():
    q, k = normal(1, 0, 4, 64), normal(2, 0, 2, 64)
    freqs, none = ops.rope_frequencies(64), i32([])
    for fn, name in ((ops.rope, "q_out"), (ops.rope_bwd, "dq")):
        qo, ko = fn(q, k, none, freqs)
        assert qo.shape == q.shape and ko.shape == k.shape
        assert fn(q, None, none, freqs, **{name: q})[0] is q
    pools = [normal(3, 5, 2, 16, 64), normal(4, 5, 2, 16, 64), torch.randn(5, 2, 64, device="cuda")]
    want = [x.clone() for x in pools]
    ops.page_copy(*pools, none, none)
    ops.paged_append(k, k, *pools, i32([[-1], [0]]), i32([0, 0, 0]), i32([0, 16]), 1, 64)
    for x, w in zip(pools, want):
        assert torch.equal(x, w)
    with pytest.raises(ValueError):
        ops.page_copy(*pools, none, i32([1]))
    assert ops.get_status() == ops.MOBA_OK
