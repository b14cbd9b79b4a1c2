"""Overlaps that the norms' entry points refuse, with as many heads of k as of q, so that
operands differ by what they are and not by their width (fake pointers; the host's checks
come before anything is launched).  The gradient's scratch is too small here: a call whose
operands pass gets no further than that."""
import pytest

from .test_paged_abi import INV, MB, WSP, lib  # noqa: F401  (lib: a fixture)
from .test_qk_norm_abi import forward, gradient


@pytest.mark.parametrize("kw", [
    # one gradient handed over for both outputs, written in place by either side
    dict(dko=40 * MB, dq=40 * MB), dict(dqo=48 * MB, dk=48 * MB),
    # an output in place of its own gradient, which is the other side's input too
    dict(k=40 * MB, dq=40 * MB), dict(q=48 * MB, dk=48 * MB),
    dict(q=40 * MB, dq=40 * MB), dict(k=48 * MB, dk=48 * MB),
    # an output over the other side's gradient or input
    dict(dq=48 * MB), dict(dk=40 * MB), dict(dq=8 * MB), dict(dk=1 * MB), dict(dq=16 * MB, dk=16 * MB),
    # the weights' gradients: over each other, an output, an input, the weights
    dict(dwk=36 * MB), dict(dwk=36 * MB + 252), dict(dwq=37 * MB + 4), dict(dwq=16 * MB + 1024), dict(dwk=24 * MB),
    dict(dwq=1 * MB), dict(dwq=8 * MB + 4 * 512 - 4), dict(dwk=40 * MB), dict(dwk=48 * MB - 252), dict(dwq=34 * MB),
    dict(dwq=34 * MB + 252, bits=32), dict(dwk=34 * MB + 124), dict(dwk=35 * MB, bits=32), dict(dwq=32 * MB + 12), dict(dwk=33 * MB),
    # an output over the weights, the positions or the frequencies
    dict(wq=16 * MB), dict(wk=16 * MB + 512), dict(wq=24 * MB - 252, bits=32), dict(pos=24 * MB + 2044), dict(freqs=16 * MB + 8)])
def test_the_gradient_refuses(lib, kw):
    assert gradient(lib, **{**dict(Hk=4, bytes=64), **kw}) == INV


@pytest.mark.parametrize("kw", [
    dict(), dict(dq=40 * MB), dict(dk=48 * MB), dict(dq=40 * MB, dk=48 * MB), dict(dko=40 * MB), dict(k=1 * MB),
    dict(wk=34 * MB), dict(dwk=36 * MB + 256), dict(dwq=16 * MB + 2048), dict(wq=16 * MB - 128), dict(Hk=0, dk=0, dwk=0, k=0, wk=0, dko=0),
    # slices of one projection, and a weight between the rows
    dict(q=1 * MB, k=1 * MB + 512, qs=1024, ks=1024, dq=16 * MB, dk=16 * MB + 512, dqs=1024, dks=1024),
    dict(dqs=512, wq=16 * MB + 512, wk=16 * MB + 1024 + 512, dwq=16 * MB + 512 + 256)])
def test_the_gradient_takes(lib, kw):
    assert gradient(lib, **{**dict(Hk=4, bytes=64), **kw}) == WSP


@pytest.mark.parametrize("kw", [
    dict(qo=8 * MB), dict(ko=1 * MB), dict(qo=16 * MB, ko=16 * MB), dict(k=1 * MB, qo=1 * MB), dict(k=1 * MB, ko=1 * MB),
    dict(wq=16 * MB), dict(wk=16 * MB + 2046), dict(wq=24 * MB - 126), dict(pos=24 * MB + 512), dict(freqs=16 * MB + 2040),
    dict(qos=512, wq=16 * MB + 1024 - 126)])
def test_the_norms_refuse(lib, kw):
    assert forward(lib, **{**dict(Hk=4), **kw}) == INV
