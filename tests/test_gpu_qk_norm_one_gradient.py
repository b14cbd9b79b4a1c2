"""One gradient handed over for both outputs of the norms (tolerances as in
test_gpu_qk_norm): taken where the results are elsewhere, refused where one side's would be
written over what the other still reads."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_cache import BF, built, normal  # noqa: F401  (built: a fixture)
from .test_gpu_qk_norm import check_gradient, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,h,d", [(3, 1, 64), (700, 6, 128)])
def test_one_gradient_for_both(tokens, h, d):
    g, q, k = (normal(i, tokens, h, d) for i in range(3))
    wq, wk = weights(3, d, BF), weights(4, d, BF)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    freqs = ops.rope_frequencies(d)
    kept = g.clone()
    for kw in (dict(dq=g), dict(dk=g), dict(dq=q), dict(dk=k), dict(dq=k)):
        with pytest.raises(RuntimeError):
            ops.qk_norm_rope_bwd(g, g, q, k, wq, wk, pos, freqs, **kw)
    one = torch.empty(d, device="cuda")
    with pytest.raises(RuntimeError):
        ops.qk_norm_rope_bwd(g, g, q, k, wq, wk, pos, freqs, dq_weight=one, dk_weight=one)
    dq, dk, dwq, dwk = ops.qk_norm_rope_bwd(g, g, q, k, wq, wk, pos, freqs)
    assert torch.equal(g, kept) and ops.get_status() == ops.MOBA_OK
    check_gradient(dq, dwq, g, q, wq, pos, freqs, 1e-6, False)
    check_gradient(dk, dwk, g, k, wk, pos, freqs, 1e-6, False)
    # in place where each side has a gradient of its own
    g2 = g.clone()
    again = ops.qk_norm_rope_bwd(g, g2, q, k, wq, wk, pos, freqs, dq=g, dk=g2)
    assert again[0] is g and again[1] is g2
    for a, b in zip(again, (dq, dk, dwq, dwk)):
        assert torch.equal(a, b)
