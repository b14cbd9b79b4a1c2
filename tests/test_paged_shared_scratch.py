"""Scratch of the shared-prefix attention where there are many groups of few rows (no GPU)."""
import pytest

from long_context_sparse_moba_gb300 import ops

from .test_paged_abi import lib  # noqa: F401  (a fixture)


def size(n_groups, num_seqs=1024, total=None, max_new=1, Hq=32, Hkv=32, D=128, page_size=64, max_pages=512):
    n = ops.paged_attn_shared_workspace_size(num_seqs, n_groups, total or num_seqs * max_new, max_new, Hq, Hkv, D, page_size, max_pages)
    assert n > 0
    return n


def big_spans(n, Hkv, D):
    """Partial sums of n spans of 256 rows on every kv head."""
    return n * Hkv * 256 * (4 * D + 8)


@pytest.mark.parametrize("seqs,hq,hkv", [(1024, 32, 32), (4096, 32, 8), (60, 8, 2)])
def test_only_groups_of_more_than_16_rows_have_big_spans(lib, seqs, hq, hkv):
    rows = seqs * hq // hkv
    one = size(1, seqs, Hq=hq, Hkv=hkv)
    many = size(seqs // 2, seqs, Hq=hq, Hkv=hkv)
    spans = rows // 256 + min(seqs // 2, rows // 17)
    # beside those, a group has a small span on every kv head and a few numbers
    small = seqs // 2 * hkv * 16 * (4 * 128 + 8)
    assert many - one <= big_spans(spans - rows // 256 - 1, hkv, 128) + small + (1 << 20)


def test_few_rows_have_none(lib):
    a, b = (size(n, num_seqs=16, Hq=1, Hkv=1, max_pages=1 << 16, page_size=16) for n in (1, 8))
    assert a < big_spans(2, 1, 128) * 100 and b - a < big_spans(1, 1, 128)
    # a chunk's groups are big whatever their rows
    assert size(8, num_seqs=8, max_new=100, Hq=1, Hkv=1) - size(1, num_seqs=8, max_new=100, Hq=1, Hkv=1) >= big_spans(7, 1, 128)
