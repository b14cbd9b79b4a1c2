"""Refusals of the rotary and paged-cache entry points that need no GPU: bad
arguments are rejected on the host before anything is launched (the fake
pointers are never dereferenced)."""
import ctypes
import math
import os
import shutil

import pytest
import torch

from long_context_sparse_moba_gb300 import ops

INV, UNS, WSP = ops.MOBA_ERR_INVALID_ARG, ops.MOBA_ERR_UNSUPPORTED, ops.MOBA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ops.LIB_PATH):
        if not shutil.which("nvcc") and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("nvcc not available to build the library")
        from long_context_sparse_moba_gb300 import build
        build.build()
    return ops.lib()


MB = 1 << 20


def rope(lib, name="moba_rope", **kw):
    a = dict(q=1 * MB, k=8 * MB, qo=16 * MB, ko=24 * MB, pos=32 * MB, freqs=33 * MB, tokens=4, Hq=4, Hk=2, D=64, rot=64,
             inter=0, mag=1.0, qs=0, ks=0, qos=0, kos=0)
    a.update(kw)
    return getattr(lib, name)(*a.values(), None)


@pytest.mark.parametrize("name", ["moba_rope", "moba_rope_bwd"])
@pytest.mark.parametrize("want,kw", [
    (INV, dict(q=0)), (INV, dict(qo=0)), (INV, dict(k=0)), (INV, dict(ko=0)), (INV, dict(pos=0)), (INV, dict(freqs=0)),
    (INV, dict(tokens=0)), (INV, dict(tokens=-1)), (INV, dict(Hq=0)), (INV, dict(Hk=-1)), (UNS, dict(D=96)),
    (UNS, dict(D=256)), (INV, dict(rot=0)), (INV, dict(rot=8)), (INV, dict(rot=80)), (INV, dict(rot=24)),
    (INV, dict(inter=2)), (INV, dict(mag=math.inf)), (INV, dict(mag=math.nan)), (INV, dict(q=1 * MB + 8)),
    (INV, dict(ko=24 * MB + 2)), (INV, dict(pos=32 * MB + 2)), (INV, dict(freqs=33 * MB + 4)), (INV, dict(qs=255)),
    (INV, dict(qs=260)), (INV, dict(kos=64)), (UNS, dict(Hq=70000)), (UNS, dict(qs=1 << 40)),
    # overlaps: an output over another operand, shifted in place, in place with another stride
    (INV, dict(qo=8 * MB)), (INV, dict(ko=1 * MB)), (INV, dict(qo=1 * MB + 64)), (INV, dict(qo=1 * MB, qos=512)),
    (INV, dict(ko=16 * MB + 256)), (INV, dict(qo=1 * MB + 512, qs=512, qos=512, Hk=0, k=0, ko=0, Hq=5))])
def test_rope_refuses(lib, name, want, kw):
    assert rope(lib, name, **kw) == want


def test_rope_frequencies(lib):
    def f(rot=8, base=10000.0, kind=ops.ROPE_PLAIN, factor=1.0, orig=0.0, slow=1.0, fast=4.0, out=True):
        buf = (ctypes.c_double * max(1, rot // 2))()
        return lib.moba_rope_frequencies(buf if out else None, rot, base, kind, factor, orig, slow, fast), list(buf)

    for bad in (dict(out=False), dict(rot=0), dict(rot=7), dict(base=1.0), dict(base=math.inf), dict(base=math.nan),
                dict(kind=4), dict(kind=-1), dict(kind=ops.ROPE_LINEAR, factor=0.5),
                dict(kind=ops.ROPE_LINEAR, factor=math.nan), dict(kind=ops.ROPE_BASE, rot=2, factor=2.0),
                dict(kind=ops.ROPE_BANDS, factor=2.0), dict(kind=ops.ROPE_BANDS, factor=2.0, orig=100.0, slow=4.0),
                dict(kind=ops.ROPE_BANDS, factor=2.0, orig=100.0, fast=math.inf)):
        assert f(**bad)[0] == INV, bad
    plain = [10000.0 ** (-i / 4) for i in range(4)]
    near = lambda x, y: all(abs(a - b) <= 4e-16 * abs(b) for a, b in zip(x, y))  # a few roundings of 64 bits
    assert near(f()[1], plain)
    assert near(f(kind=ops.ROPE_LINEAR, factor=4.0)[1], [p / 4 for p in plain])
    # the larger base leaves the fastest pair alone and slows the slowest by the factor
    got = f(kind=ops.ROPE_BASE, factor=4.0)[1]
    assert got[0] == 1.0 and abs(got[3] - plain[3] / 4) < 1e-15
    # bands: 1000 positions make 159.2, 15.9, 1.59 and 0.159 turns
    got = f(kind=ops.ROPE_BANDS, factor=4.0, orig=1000.0)[1]
    keep = (1000 * plain[2] / (2 * math.pi) - 1.0) / 3.0
    assert near(got, [plain[0], plain[1], plain[2] * keep + plain[2] / 4 * (1 - keep), plain[3] / 4])
    assert ops.rope_frequencies(64, device="cpu").dtype == torch.float64
    with pytest.raises(RuntimeError):
        ops.rope_frequencies(0, device="cpu")


def attn(lib, **kw):
    a = dict(q=1 * MB, k=2 * MB, v=3 * MB, kbar=4 * MB, table=5 * MB, cu=6 * MB, lens=7 * MB, out=8 * MB, lse=9 * MB,
             idx=10 * MB, num_seqs=2, total=8, max_new=4, Hq=4, Hkv=2, D=64, num_pages=100, page_size=16, max_pages=40,
             block_size=64, topk=3, ws=256 * MB, bytes=1 << 40)
    a.update(kw)
    return lib.moba_paged_attn(*a.values(), None)


SHARED = [(INV, dict(k=0)), (INV, dict(v=0)), (INV, dict(table=0)), (INV, dict(cu=0)), (INV, dict(lens=0)),
          (INV, dict(num_seqs=0)), (INV, dict(total=0)), (INV, dict(max_new=0)), (INV, dict(Hkv=0)),
          (INV, dict(num_pages=0)), (INV, dict(max_pages=0)), (INV, dict(page_size=8)), (INV, dict(page_size=48)),
          (INV, dict(block_size=32)), (INV, dict(block_size=96)), (INV, dict(block_size=64, page_size=128)),
          (UNS, dict(D=32)), (INV, dict(k=2 * MB + 8)), (INV, dict(v=3 * MB + 2)), (INV, dict(kbar=4 * MB + 4)),
          (INV, dict(table=5 * MB + 2)), (INV, dict(cu=6 * MB + 1)), (INV, dict(lens=7 * MB + 3)),
          (UNS, dict(total=1 << 26)), (UNS, dict(num_seqs=70000)), (UNS, dict(max_pages=1 << 26)),
          (UNS, dict(num_pages=1 << 27))]


@pytest.mark.parametrize("want,kw", SHARED + [
    (INV, dict(q=0)), (INV, dict(out=0)), (INV, dict(lse=0)), (INV, dict(kbar=0)), (INV, dict(topk=0)),
    (INV, dict(Hq=3)), (INV, dict(Hq=0)), (UNS, dict(Hq=130)), (INV, dict(q=1 * MB + 4)), (INV, dict(out=8 * MB + 8)),
    (INV, dict(lse=9 * MB + 2)), (INV, dict(idx=10 * MB + 1)), (UNS, dict(max_pages=400, topk=34)),
    (UNS, dict(max_pages=1 << 20)), (WSP, dict(bytes=1000)), (WSP, dict(ws=256 * MB + 64))])
def test_attention_refuses(lib, want, kw):
    assert attn(lib, **kw) == want


def test_attention_workspace_size(lib):
    size = lambda **kw: ops.paged_attn_workspace_size(**{**dict(num_seqs=2, total=8, max_new=4, Hq=4, Hkv=2, D=64,
                                                                page_size=16, max_pages=40, block_size=64, topk=3), **kw})
    assert size() > 0 and size(topk=100) > 0
    assert size(D=32) == size(Hq=3) == size(topk=0) == size(page_size=48) == 0


@pytest.mark.parametrize("want,kw", SHARED + [(INV, dict(nk=0)), (INV, dict(nv=0)), (INV, dict(nk=1 * MB + 2)),
                                              (INV, dict(pooling=7))])
def test_append_refuses(lib, want, kw):
    a = dict(nk=1 * MB, nv=11 * MB, k=2 * MB, v=3 * MB, kbar=4 * MB, table=5 * MB, cu=6 * MB, lens=7 * MB, num_seqs=2,
             total=8, max_new=4, Hkv=2, D=64, num_pages=100, page_size=16, max_pages=40, block_size=64)
    kw = dict(kw)
    o = ops.Options()
    o.pooling = kw.pop("pooling", 0)
    a.update(kw)
    assert lib.moba_paged_append(*a.values(), ctypes.byref(o), None) == want


@pytest.mark.parametrize("want,kw", [
    (INV, dict(k=0)), (INV, dict(v=0)), (INV, dict(src=0)), (INV, dict(dst=0)), (INV, dict(n=0)), (INV, dict(layers=0)),
    (INV, dict(pages=0)), (INV, dict(hkv=0)), (INV, dict(page=8)), (INV, dict(page=20)), (INV, dict(k=2 * MB + 8)),
    (INV, dict(kbar=4 * MB + 8)), (INV, dict(src=5 * MB + 2)), (INV, dict(dst=6 * MB + 1)), (UNS, dict(d=96)),
    (UNS, dict(page=1 << 21)), (UNS, dict(pages=1 << 30, layers=100)), (UNS, dict(n=65537)), (UNS, dict(layers=70000))])
def test_page_copy_refuses(lib, want, kw):
    a = dict(k=2 * MB, v=3 * MB, kbar=4 * MB, src=5 * MB, dst=6 * MB, n=3, layers=1, pages=100, hkv=2, d=64, page=16)
    a.update(kw)
    assert lib.moba_page_copy(*a.values(), None) == want


def test_binding_refuses_host_tensors():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    pools = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.rope(q, None, i, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        ops.paged_attn(q, pools, pools, None, i.view(2, 2), i, i, 1, 64, 1)
    with pytest.raises(ValueError):
        ops.paged_append(q, q, pools, pools, None, i.view(2, 2), i, i, 1, 64)
    with pytest.raises(ValueError):
        ops.page_copy(pools, pools, None, i, i)
