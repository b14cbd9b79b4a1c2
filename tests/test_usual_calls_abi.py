"""The binding of the calls in one step, without a GPU: what it leaves alone, and its absence."""
import sys

import pytest
import torch

from long_context_sparse_moba_gb300 import ops


def test_tensors_of_the_host_are_left_to_the_other_steps():
    t = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    n = ops._native()
    for f, args in ((n.qk_norm_rope, 11), (n.qk_norm_rope_bwd, 16), (n.paged_append_rope, 19), (n.paged_attn_shared, 12)):
        assert f(*[t] * args) is None and f(*[None] * args) is None and f(*[1] * args) is None
        assert f() is None and f(t) is None


def test_a_binding_that_is_missing_says_so(monkeypatch):
    monkeypatch.setattr(ops, "_calls", None)
    monkeypatch.setitem(sys.modules, "long_context_sparse_moba_gb300.moba_calls", None)
    import long_context_sparse_moba_gb300 as package
    monkeypatch.delattr(package, "moba_calls", raising=False)
    with pytest.raises(RuntimeError, match="build"):
        ops._native()


def test_a_cuda_error_raises():
    with pytest.raises(RuntimeError, match="moba_x"):
        ops._usual(ops.MOBA_ERR_CUDA, "moba_x")
    assert ops._usual((1, 2), "moba_x") == (1, 2)
