"""Pages whose offsets pass 32 bits: appending with norms and rotation, and shared prefixes,
at the end of pools of 5 G values."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_attn import expect
from .test_gpu_paged_cache import BF, built, i32, normal  # noqa: F401  (built: a fixture)
from .test_gpu_qk_norm import weights
from .test_gpu_paged_shared import compare

pytestmark = pytest.mark.gpu


def test_far_pages():
    P, hq, hkv, page, d, block = 5 << 20, 8, 1, 16, 64, 64
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    k_pages, v_pages = (torch.empty(P, hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
    kbar = torch.empty(P, hkv, d, device="cuda")
    assert k_pages.numel() > 1 << 32
    # three sequences of 320 tokens, 256 of them on the same pages, near the pools' end and start
    head, own = [P - 1 - i for i in range(16)], [[P // 2 + 8 * b + i for i in range(4)] for b in range(3)]
    table = i32([head + own[b] for b in range(3)])
    w, freqs = weights(1, d, BF), ops.rope_frequencies(d)
    k0, v0 = normal(2, 256, hkv, d), normal(3, 256, hkv, d)
    kw = dict(q_weight=w, k_weight=w)
    q0 = normal(4, 256, hq, d)
    ops.paged_append_rope(q0, k0, v0, k_pages, v_pages, kbar, table[:1], i32([0, 256]), i32([256]), 256, block, freqs, **kw)
    q, k, v = (normal(s, 192, h, d) for s, h in ((5, hq), (6, hkv), (7, hkv)))
    cu, lens = i32([0, 64, 128, 192]), i32([320, 320, 320])
    qr = ops.paged_append_rope(q, k, v, k_pages, v_pages, kbar, table, cu, lens, 64, block, freqs, **kw)
    assert ops.get_status() == ops.MOBA_OK
    pos0 = torch.arange(256, dtype=torch.int32, device="cuda")
    pos = torch.arange(256, 320, dtype=torch.int32, device="cuda").repeat(3)
    kr0, kr = ops.qk_norm_rope(k0, None, w, None, pos0, freqs)[0], ops.qk_norm_rope(k, None, w, None, pos, freqs)[0]
    assert torch.equal(qr, ops.qk_norm_rope(q, None, w, None, pos, freqs)[0])
    ks, vs = [], []
    for b in range(3):
        rows = table[b].long()
        stored = k_pages[rows].transpose(1, 2).reshape(320, hkv, d)
        ks.append(torch.cat((kr0, kr[64 * b:64 * b + 64])))
        vs.append(torch.cat((v0, v[64 * b:64 * b + 64])))
        assert torch.equal(stored, ks[-1])
        mean = stored[256:].double().mean(0)
        assert ((kbar[rows[19]].double() - mean).abs() <= 8 * 2.0 ** -24 * stored[256:].double().abs().mean(0)).all()
    # few new tokens (the stream) and many (the tensor cores)
    for n in (1, 64):
        rows = [r for b in range(3) for r in range(64 * b + 64 - n, 64 * b + 64)]
        qn = qr[rows].contiguous()
        got = ops.paged_attn_shared(qn, k_pages, v_pages, table, i32([0, n, 2 * n, 3 * n]), lens, n, i32([0, 3]), i32([256]))
        assert ops.get_status() == ops.MOBA_OK
        compare(got, expect(qn, ks, vs, None, [n] * 3, [320] * 3, 1 << 20, 1))
