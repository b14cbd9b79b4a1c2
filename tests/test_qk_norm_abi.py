"""Refusals of the norms' and the rotating append's entry points that need no GPU: bad
arguments are rejected on the host before anything is launched (the fake pointers are
never dereferenced)."""
import ctypes
import math

import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_paged_abi import INV, MB, SHARED, UNS, WSP, lib  # noqa: F401  (lib: a fixture)

COMMON = [(INV, dict(q=0)), (INV, dict(k=0)), (INV, dict(wq=0)), (INV, dict(wk=0)), (INV, dict(pos=0)), (INV, dict(freqs=0)),
          (INV, dict(tokens=0)), (INV, dict(tokens=-1)), (INV, dict(Hq=0)), (INV, dict(Hk=-1)), (UNS, dict(D=96)),
          (UNS, dict(D=256)), (INV, dict(rot=0)), (INV, dict(rot=8)), (INV, dict(rot=80)), (INV, dict(inter=2)),
          (INV, dict(mag=math.inf)), (INV, dict(mag=math.nan)), (INV, dict(eps=0.0)), (INV, dict(eps=1e-13)),
          (INV, dict(eps=-1.0)), (INV, dict(eps=math.nan)), (INV, dict(eps=math.inf)), (INV, dict(bits=8)), (INV, dict(bits=0)),
          (INV, dict(q=1 * MB + 8)), (INV, dict(pos=32 * MB + 2)), (INV, dict(freqs=33 * MB + 4)), (INV, dict(wq=34 * MB + 1)),
          (INV, dict(wk=35 * MB + 2, bits=32)), (INV, dict(qs=255)), (INV, dict(qs=260)), (INV, dict(ks=64)),
          (UNS, dict(Hq=70000)), (UNS, dict(qs=1 << 40))]


def forward(lib, **kw):
    a = dict(q=1 * MB, k=8 * MB, qo=16 * MB, ko=24 * MB, wq=34 * MB, wk=35 * MB, bits=16, eps=1e-6, pos=32 * MB, freqs=33 * MB,
             tokens=4, Hq=4, Hk=2, D=64, rot=64, inter=0, mag=1.0, qs=0, ks=0, qos=0, kos=0)
    a.update(kw)
    return lib.moba_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("want,kw", COMMON + [
    (INV, dict(qo=0)), (INV, dict(ko=0)), (INV, dict(ko=24 * MB + 2)), (INV, dict(kos=64)),
    # overlaps: an output over another operand, shifted in place, in place with another stride
    (INV, dict(qo=8 * MB)), (INV, dict(ko=1 * MB)), (INV, dict(qo=1 * MB + 64)), (INV, dict(qo=1 * MB, qos=512)),
    (INV, dict(ko=16 * MB + 256)), (INV, dict(qo=1 * MB + 512, qs=512, qos=512, Hk=0, k=0, ko=0, Hq=5))])
def test_norms_refuse(lib, want, kw):
    assert forward(lib, **kw) == want


def gradient(lib, **kw):
    a = dict(dqo=40 * MB, dko=48 * MB, q=1 * MB, k=8 * MB, wq=34 * MB, wk=35 * MB, dq=16 * MB, dk=24 * MB, dwq=36 * MB,
             dwk=37 * MB, bits=16, eps=1e-6, pos=32 * MB, freqs=33 * MB, tokens=4, Hq=4, Hk=2, D=64, rot=64, inter=0, mag=1.0,
             dqos=0, dkos=0, qs=0, ks=0, dqs=0, dks=0, ws=256 * MB, bytes=1 << 30)
    a.update(kw)
    return lib.moba_qk_norm_rope_bwd(*a.values(), None)


@pytest.mark.parametrize("want,kw", COMMON + [
    (INV, dict(dqo=0)), (INV, dict(dko=0)), (INV, dict(dq=0)), (INV, dict(dk=0)), (INV, dict(dwq=0)), (INV, dict(dwk=0)),
    (INV, dict(dwq=36 * MB + 2)), (INV, dict(dkos=64)), (INV, dict(dqs=250)),
    (INV, dict(dq=1 * MB)), (INV, dict(dq=8 * MB)), (INV, dict(dk=40 * MB)), (INV, dict(dq=40 * MB, dqs=512)),
    (INV, dict(dk=16 * MB)), (INV, dict(dk=48 * MB + 64)), (WSP, dict(bytes=64)), (WSP, dict(ws=256 * MB + 64))])
def test_the_norms_gradient_refuses(lib, want, kw):
    assert gradient(lib, **kw) == want


def test_workspace_size(lib):
    size = ops.qk_norm_rope_bwd_workspace_size
    assert size(4, 4, 2, 64) > 0 and size(4, 4, 0, 64) > 0
    assert size(0, 4, 2, 64) == size(4, 0, 2, 64) == size(4, 4, -1, 64) == size(4, 4, 2, 96) == size(4, 70000, 2, 64) == 0


@pytest.mark.parametrize("want,kw", [(w, {("kp" if n == "k" else "vp" if n == "v" else n): x for n, x in kw.items()})
                                     for w, kw in SHARED] + [
    (INV, dict(q=0)), (INV, dict(nk=0)), (INV, dict(nv=0)), (INV, dict(qo=0)), (INV, dict(freqs=0)), (INV, dict(Hq=0)),
    (UNS, dict(Hq=70000)), (INV, dict(rot=8)), (INV, dict(rot=80)), (INV, dict(inter=-1)), (INV, dict(mag=math.nan)),
    (INV, dict(eps=0.0)), (INV, dict(bits=0)), (INV, dict(wq=0, bits=7)), (INV, dict(wq=34 * MB + 1)), (INV, dict(pos=32 * MB + 1)),
    (INV, dict(freqs=33 * MB + 4)), (INV, dict(q=12 * MB + 2)), (INV, dict(nk=1 * MB + 8)), (INV, dict(nv=11 * MB + 4)),
    (INV, dict(qo=13 * MB + 8)), (INV, dict(qs=100)), (INV, dict(ks=64)), (INV, dict(vs=132)), (INV, dict(qos=255)),
    (INV, dict(qo=1 * MB)), (INV, dict(qo=11 * MB)), (INV, dict(qo=12 * MB + 128)), (INV, dict(qo=12 * MB, qos=512)),
    (INV, dict(pooling=7))])
def test_the_rotating_append_refuses(lib, want, kw):
    a = dict(q=12 * MB, nk=1 * MB, nv=11 * MB, qo=13 * MB, kp=2 * MB, vp=3 * MB, kbar=4 * MB, table=5 * MB, cu=6 * MB, lens=7 * MB,
             pos=32 * MB, freqs=33 * MB, wq=34 * MB, wk=35 * MB, bits=16, eps=1e-6, num_seqs=2, total=8, max_new=4, Hq=4, Hkv=2,
             D=64, rot=64, inter=0, mag=1.0, qs=0, ks=0, vs=0, qos=0, num_pages=100, page_size=16, max_pages=40, block_size=64)
    kw = dict(kw)
    o = ops.Options()
    o.pooling = kw.pop("pooling", 0)
    a.update(kw)
    assert lib.moba_paged_append_rope(*a.values(), ctypes.byref(o), None) == want


def test_the_binding_refuses():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i, f, w = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64), torch.ones(64)
    pools = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.qk_norm_rope(q, None, w, None, i, f)
    with pytest.raises(ValueError):
        ops.qk_norm_rope_bwd(q, None, q, None, w, None, i, f)
    with pytest.raises(ValueError):
        ops.paged_append_rope(q, q, q, pools, pools, None, i.view(2, 2), i, i, 1, 64, f)


@pytest.mark.parametrize("a,b,bits", [(torch.float32, torch.float32, 32), (torch.bfloat16, None, 16), (None, None, 0),
                                      (torch.bfloat16, torch.float32, None), (torch.float16, None, None)])
def test_weights_are_of_one_type(monkeypatch, a, b, bits):
    monkeypatch.setattr(ops, "_tensor", lambda *x: None)
    w = [None if t is None else torch.ones(64, dtype=t) for t in (a, b)]
    if bits is None:
        with pytest.raises(ValueError):
            ops._weights(0, 64, *w)
    else:
        assert ops._weights(0, 64, *w) == bits
    if w[0] is not None:
        with pytest.raises(ValueError):
            ops._weights(0, 128, *w)
