"""Calls right behind calls of the framework whose results they read: such a call's first
kernel is there while the kernel that writes its operands still runs.  The same bits as with
copies of the operands and nothing running beside."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_cache import BF, Cache, built, i32, normal  # noqa: F401  (built: a fixture)
from .test_gpu_paged_rope import same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
def test_weights_that_the_call_before_wrote(captured):
    """The norms' and the append's weights are the weights' gradient of the call before."""
    T, h, d, steps = 300, 6, 64, 40
    x = normal(1, T, 3 * h, d)
    w = 1 + 0.3 * normal(2, d).float()
    pos, freqs = torch.arange(T, dtype=torch.int32, device="cuda"), ops.rope_frequencies(d)
    dy = [normal(3 + i, T, h, d) for i in range(steps)]
    c = Cache(1, 512, h, d, 32, 64)
    tables = c.k, c.v, c.kbar, c.table, i32([0, T]), i32([T]), T, c.block, freqs
    dw, dx = torch.empty(d, device="cuda"), torch.empty(T, h, d, dtype=BF, device="cuda")
    want = []
    ws = torch.empty(ops.qk_norm_rope_bwd_workspace_size(T, h, 0, d), dtype=torch.uint8, device="cuda")

    def step(i):
        ops.qk_norm_rope_bwd(dy[i], None, x[:, :h], None, w, None, pos, freqs, dq=dx, dq_weight=dw, workspace=ws)
        y, _ = ops.qk_norm_rope(dx, None, dw, None, pos, freqs)
        ops.qk_norm_rope_bwd(dy[-1 - i], None, x[:, :h], None, w, None, pos, freqs, dq=dx, dq_weight=dw, workspace=ws)
        z = ops.paged_append_rope(dx, x[:, h:2 * h], x[:, 2 * h:], *tables, q_weight=dw, k_weight=dw)
        return y, z, c.k.clone(), c.kbar.clone()

    for i in range(steps):
        made = []
        for g in (dy[i], dy[-1 - i]):
            r = ops.qk_norm_rope_bwd(g, None, x[:, :h], None, w, None, pos, freqs)
            torch.cuda.synchronize()
            made.append((r[0].clone(), r[2].clone()))
            torch.cuda.synchronize()
        (x1, w1), (x2, w2) = made
        y = ops.qk_norm_rope(x1, None, w1, None, pos, freqs)[0]
        z = ops.paged_append_rope(x2, x[:, h:2 * h], x[:, 2 * h:], *tables, q_weight=w2, k_weight=w2)
        torch.cuda.synchronize()
        want.append((y, z, c.k.clone(), c.kbar.clone()))
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = [step(i) for i in range(steps)]
        for _ in range(2):
            g.replay()
    else:
        out = [step(i) for i in range(steps)]
    for a, b in zip(out, want):
        assert all(same(x, y) for x, y in zip(a, b))
    assert ops.get_status() == ops.MOBA_OK
