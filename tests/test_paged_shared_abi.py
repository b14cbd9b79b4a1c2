"""Refusals of the shared-prefix attention that need no GPU (the fake pointers are never
dereferenced)."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_paged_abi import INV, MB, SHARED, UNS, WSP, lib  # noqa: F401  (lib: a fixture)


@pytest.mark.parametrize("want,kw", [x for x in SHARED if not {"kbar", "block_size"} & set(x[1])] + [
    (INV, dict(q=0)), (INV, dict(out=0)), (INV, dict(lse=0)), (INV, dict(groups=0)), (INV, dict(prefixes=0)),
    (INV, dict(n_groups=-1)), (UNS, dict(n_groups=65536)), (INV, dict(Hq=3)), (INV, dict(Hq=0)), (UNS, dict(Hq=130)),
    (INV, dict(q=1 * MB + 4)), (INV, dict(out=8 * MB + 8)), (INV, dict(lse=9 * MB + 2)), (INV, dict(groups=11 * MB + 1)),
    (INV, dict(prefixes=12 * MB + 2)), (UNS, dict(total=1 << 25, Hq=4)), (WSP, dict(bytes=1000)), (WSP, dict(ws=256 * MB + 64))])
def test_it_refuses(lib, want, kw):
    a = dict(q=1 * MB, k=2 * MB, v=3 * MB, table=5 * MB, cu=6 * MB, lens=7 * MB, groups=11 * MB, prefixes=12 * MB, out=8 * MB,
             lse=9 * MB, num_seqs=2, n_groups=1, total=8, max_new=4, Hq=4, Hkv=2, D=64, num_pages=100, page_size=16, max_pages=40,
             ws=256 * MB, bytes=1 << 40)
    a.update(kw)
    assert lib.moba_paged_attn_shared(*a.values(), None) == want


def test_workspace_size(lib):
    size = lambda **kw: ops.paged_attn_shared_workspace_size(**{**dict(num_seqs=2, n_groups=1, total=8, max_new=4, Hq=4, Hkv=2, D=64,
                                                                       page_size=16, max_pages=40), **kw})
    assert size() > 0 and size(n_groups=0) > 0 and size(max_new=100, total=300) > 0
    assert size(D=32) == size(Hq=3) == size(page_size=48) == size(n_groups=-1) == size(n_groups=70000) == 0


def test_the_binding_refuses(monkeypatch):
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    pools = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.paged_attn_shared(q, pools, pools, i.view(2, 2), i, i, 1, i, i)
    monkeypatch.setattr(ops, "_device", lambda t, name: -1)
    for groups, prefixes in ((i, i), (i, i[:2])):
        with pytest.raises(ValueError):
            ops.paged_attn_shared(q, pools, pools, torch.zeros(2, 2, dtype=torch.int32), i[:3], i[:2], 1, groups, prefixes)
