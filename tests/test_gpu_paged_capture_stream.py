"""A layer captured on a stream that is named and not the current one: forks are attended each
by itself there too, since a replay's page table may hold others."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops, paged
from long_context_sparse_moba_gb300.paged import PagedCache

from .test_gpu_paged_cache import built, normal  # noqa: F401  (built: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("named", [False, True])
def test_forks_of_a_captured_stream(monkeypatch, named):
    monkeypatch.setattr(paged, "SHARED_BYTES", 1)
    c = PagedCache(1, 64, 2, 64, 16, 64)
    a = c.new()
    batch = c.extend({a: 128})
    q, k, v = (normal(i, 128, h, 64) for i, h in ((1, 8), (2, 2), (3, 2)))
    c.attend(0, batch, q, k, v, 1000)
    b = c.fork(a)
    batch = c.extend({a: 1, b: 1})
    assert batch.cu_groups is not None
    q, k, v = (normal(i, 2, h, 64) for i, h in ((4, 8), (5, 2), (6, 2)))
    names = []
    for name in ("paged_attn", "paged_attn_shared"):
        def call(*args, name=name, real=getattr(ops, name), **kw):
            names.append(name)
            return real(*args, **kw)
        monkeypatch.setattr(ops, name, call)
    want = c.attend(0, batch, q, k, v, 1000)[0]
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = torch.cuda.current_stream()
        if named:
            with torch.cuda.stream(side):
                got = c.attend(0, batch, q, k, v, 1000, stream=captured)
        else:
            got = c.attend(0, batch, q, k, v, 1000)
    assert names == ["paged_attn_shared", "paged_attn"]
    g.replay()
    torch.cuda.synchronize()
    assert (got[0].double() - want.double()).abs().max() <= 2e-2 and ops.get_status() == ops.MOBA_OK
