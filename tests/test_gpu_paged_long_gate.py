"""A selection that takes longer than the attention kernel's waits for its next job may:
the kernel, which starts as the first CTAs of the gate leave, has to sit it out."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_cache import BF, built, i32, normal  # noqa: F401  (built: a fixture)

pytestmark = pytest.mark.gpu


def test_ties_over_a_very_long_cache():
    """Every score of every second tile of 128 rows ties, so each of those rows is decided by 64-bit
    scores of 65535 blocks: some seconds on some SMs while others are done at once."""
    blocks, block, d, n = 65535, 64, 128, 456 * 128
    length = blocks * block + 30
    k = torch.zeros(blocks + 1, 1, block, d, dtype=BF, device="cuda")
    v = normal(2, blocks + 1, 1, block, d)
    kbar = torch.randn(blocks + 1, 1, d, generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    table = torch.arange(blocks + 1, dtype=torch.int32, device="cuda").view(1, -1)
    q = normal(4, n, 1, d)
    tied = torch.arange(n, device="cuda") // 128 % 2 == 0
    q[tied] = 0
    out, lse, idx = ops.paged_attn(q, k, v, kbar, table, i32([0, n]), i32([length]), n, block, 2, with_idx=True)
    assert ops.get_status() == ops.MOBA_OK
    own = torch.arange(length - n, length, device="cuda") // block
    assert (idx[tied, 0, 0] == 0).all() and (idx[:, 0, 1] == own).all()
    some = torch.arange(128, n, 997, device="cuda")
    some = some[~tied[some]]
    score = torch.stack([(kbar[:, 0].double() * q[i, 0].double()).sum(-1) for i in some.tolist()])
    score.masked_fill_(torch.arange(blocks + 1, device="cuda") >= own[some, None], -float("inf"))
    assert torch.equal(idx[some, 0, 0].long(), score.argmax(-1))
    # keys of zeros: the mean of the values that a row sees, and the logarithm of their number
    seen = block + 1 + torch.arange(length - n, length, device="cuda") % block
    assert ((lse[:, 0].double() - seen.double().log()).abs() <= 2.0 ** -20 * (1 + seen.double().log())).all()
    for i in some[:16].tolist():
        keys = torch.cat((v[idx[i, 0, 0], 0], v[own[i], 0, :int(seen[i]) - block])).double()
        # weights of a power of two would be exact; P, the partials and the result are rounded
        tol = 2.0 ** -8 * (keys.abs().mean(0) + keys.mean(0).abs()) + 2.0 ** -10 * keys.abs().mean(0)
        assert ((out[i, 0].double() - keys.mean(0)).abs() <= tol).all()
