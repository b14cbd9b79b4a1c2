"""Appending keys that are not finite: a pooled key is what the mean in 64 bits is,
and a block whose score is infinite is selected first or last.

Finite pooled keys err by at most 8 u mean|k| (u = 2^-24): a compensated sum in
three levels of at most 2 u each, and the division; or a sum in 64 bits, rounded once."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_attn import attend
from .test_gpu_paged_cache import Cache, built, normal  # noqa: F401  (built: a fixture)

pytestmark = pytest.mark.gpu
INF = float("inf")


def keys(n, hkv, d, block):
    """Infinities in some columns of some blocks: one, several, both signs, beside a NaN."""
    k = normal(3, n, hkv, d)
    k[5, 0, 0] = INF                       # block 0: the first group of tokens
    k[block - 1, 0, 1] = -INF              # its last token
    k[:block:7, -1, 2] = INF               # several of one sign
    k[block + 3, 0, 3], k[block + 40, 0, 3] = INF, -INF   # block 1: both signs, of different groups
    k[block + 3, 0, 4], k[block + 4, 0, 4] = -INF, INF
    k[2 * block:3 * block, 0, 5] = -INF    # block 2: every key
    k[2 * block + 9, 0, 6], k[2 * block + 10, 0, 6] = INF, float("nan")
    k[:block, 0, 7] = 3e38                 # finite, the sum is not
    k[block:2 * block, 0, 8] = 3e38 * (1 - 2 * (torch.arange(block, device="cuda") // 3 % 2))
    k[2 * block + 1:2 * block + 3, 0, 9] = -3e38
    return k


@pytest.mark.parametrize("seqs", [1, 40])  # (few and many blocks take clusters of different sizes)
@pytest.mark.parametrize("hkv,d,page,block", [(1, 64, 16, 64), (2, 128, 32, 128), (8, 128, 64, 512), (3, 64, 64, 192)])
def test_the_mean_of_infinite_keys(hkv, d, page, block, seqs):
    n = 3 * block + 11
    k = keys(n, hkv, d, block)
    c = Cache(seqs, 4 * block, hkv, d, page, block)
    cut = 2 * block + 10
    for lo, hi in ((0, cut), (cut, n)):
        part = k[lo:hi].repeat(seqs, 1, 1)
        c.append(part, part, [i * (hi - lo) for i in range(seqs + 1)], [hi] * seqs)
    assert ops.get_status() == ops.MOBA_OK
    x = k[:3 * block].double().view(3, block, hkv, d)
    want, size = x.mean(1), x.abs().mean(1)
    assert want.isposinf().any() and want.isneginf().any() and want.isnan().any()
    slots = c.table[:, [(b + 1) * block // page - 1 for b in range(3)]].long()
    got = c.kbar[slots].double()
    want = want.expand_as(got)
    finite = want.isfinite()
    assert torch.equal(got.nan_to_num(nan=7.0, posinf=8.0, neginf=9.0)[~finite],
                       want.nan_to_num(nan=7.0, posinf=8.0, neginf=9.0)[~finite])
    assert ((got - want).abs() <= 8 * 2.0 ** -24 * size)[finite].all()


@pytest.mark.parametrize("n", [1, 200])  # few rows, and a chunk
def test_a_block_with_an_infinite_key_is_selected_by_its_score(n):
    d, block, page, length = 64, 64, 16, 64 * 9 + 30
    k = normal(1, length, 1, d)
    k[2 * block + 7, 0, 0] = INF
    k[5 * block + 1, 0, 0] = -INF
    c = Cache(1, 640, 1, d, page, block)
    c.append(k, normal(2, length, 1, d), [0, length], [length])
    q = normal(4, n, 4, d)
    q[:, :2, 0] = q[:, :2, 0].abs() + 0.1   # these heads score +inf with block 2
    q[:, 2:, 0] = -q[:, 2:, 0].abs() - 0.1  # these with block 5
    _, _, idx = attend(c, q, [n], [length], block, 2, with_idx=True)
    assert ops.get_status() == ops.MOBA_OK
    own = torch.arange(length - n, length, device="cuda") // block
    for heads, first in ((slice(0, 2), 2), (slice(2, 4), 5)):
        rows = own > first
        assert (idx[rows][:, heads, 0] == first).all() and rows.any()
