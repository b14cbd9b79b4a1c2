"""Rotary positions and their gradient against the formula in 64 bits.

Tolerance: a result is rounded once to bf16 (half a step, 2^-8 of it); before
that fp32 holds cos and sin of a phase that is itself rounded to 24 bits.  The
phase error is at most pi 2^-24, the functions' and the two products' roundings
less than 2^-21 together, so |error| <= 2^-8 |r| + 2^-20 m (|a| + |b|) for a pair
(a, b) and magnitude m."""
import math

import numpy as np
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_sparse_moba_gb300 import build
    build.build()
    ops.lib()


def turn64(x, pos, freqs, interleaved, mag, sign=1.0):
    """(rotated x, m (|a| + |b|) of each value's pair; 0 for copied values), fp64."""
    x = x.double()
    r = 2 * freqs.numel()
    ang = pos.double().reshape(-1, 1) * freqs
    shape = x.shape[:-2] + (1, r // 2)
    c, s = (ang.cos() * mag).view(shape), (sign * ang.sin() * mag).view(shape)
    ia = torch.arange(r // 2, device=x.device) * 2 if interleaved else torch.arange(r // 2, device=x.device)
    ib = ia + 1 if interleaved else ia + r // 2
    y, w = x.clone(), torch.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    w[..., ia] = w[..., ib] = mag * (a.abs() + b.abs())
    return y, w


def check(got, x, pos, freqs, interleaved, mag, sign=1.0):
    want, pair = turn64(x, pos, freqs, interleaved, mag, sign)
    err = (got.double() - want).abs()
    tol = want.abs() * 2.0 ** -8 + pair * 2.0 ** -20
    assert (err <= tol).all(), float((err - tol).max())
    rest = 2 * freqs.numel()
    assert torch.equal(got[..., rest:], x[..., rest:])


def normal(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("tokens,hq,hk,d,rot,interleaved", [
    (1, 1, 1, 64, 64, False), (1, 32, 8, 128, 128, True), (7, 5, 3, 64, 16, False),
    (129, 6, 2, 128, 64, True), (1000, 9, 1, 128, 48, False), (3333, 33, 8, 64, 32, True),
    (2500, 32, 32, 128, 128, False)])
def test_rope_and_gradient_match_the_formula(tokens, hq, hk, d, rot, interleaved):
    q, k = normal(1, tokens, hq, d), normal(2, tokens, hk, d)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda") * 17 + 3
    freqs = ops.rope_frequencies(rot, 10000.0)
    for fn, sign in ((ops.rope, 1.0), (ops.rope_bwd, -1.0)):
        qo, ko = fn(q, k, pos, freqs, interleaved=interleaved, magnitude=1.25)
        check(qo, q, pos, freqs, interleaved, 1.25, sign)
        check(ko, k, pos, freqs, interleaved, 1.25, sign)
    qo, ko = ops.rope(q, None, pos, freqs, interleaved=interleaved)
    assert ko is None
    check(qo, q, pos, freqs, interleaved, 1.0)


def test_rope_far_and_negative_positions():
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 1, 2 ** 24 + 3, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32,
                       device="cuda")
    freqs = ops.rope_frequencies(128, 500000.0, ops.ROPE_BANDS, factor=8.0, original_length=8192)
    q = normal(3, pos.numel(), 4, 128)
    qo, _ = ops.rope(q, None, pos, freqs)
    check(qo, q, pos, freqs, False, 1.0)
    # any table: turning backwards, several turns per position, no turn at all
    odd = torch.tensor([-0.5, 7.0, 0.0, 2 * math.pi, 100.25, -1e-9, 3.0, 1.0], dtype=torch.float64, device="cuda")
    x = normal(4, pos.numel(), 2, 64)
    near = torch.tensor([0, 1, -1, 5, 1000, -77, 12345], dtype=torch.int32, device="cuda")
    xo, _ = ops.rope(x, None, near, odd, interleaved=True)
    check(xo, x, near, odd, True, 1.0)


def test_rope_strided_and_in_place():
    T, hq, hk, d = 77, 8, 2, 128
    qkv = normal(5, T, hq + 2 * hk, d)
    ref = qkv.clone()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freqs = ops.rope_frequencies(d)
    qo, ko = ops.rope(q, k, pos, freqs)
    check(qo, ref[:, :hq], pos, freqs, False, 1.0)
    check(ko, ref[:, hq:hq + hk], pos, freqs, False, 1.0)
    ops.rope(q, k, pos, freqs, q_out=q, k_out=k)  # in the projection itself
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, ref[:, hq + hk:])
    # a batch, every second token of a longer one
    x = normal(6, 2, 50, 3, 64)
    p2 = torch.arange(50, dtype=torch.int32, device="cuda")
    part = x[:, ::2]
    y, _ = ops.rope(part, None, p2, ops.rope_frequencies(64))
    check(y, part, p2, ops.rope_frequencies(64), False, 1.0)


def test_gradient_against_differences():
    """rope is linear in x: the gradient of <w, rope(x)> along any direction is
    the central difference of the 64-bit formula, up to the gradient's bf16
    rounding (2^-8 of each value) and the difference's own rounding."""
    T, h, d = 5, 2, 64
    pos = torch.tensor([0, 9, 100, 5000, 70000], dtype=torch.int32, device="cuda")
    freqs = ops.rope_frequencies(32)
    x, w, direction = (normal(s, T, h, d) for s in (7, 8, 9))
    for interleaved in (False, True):
        dx, _ = ops.rope_bwd(w, None, pos, freqs, interleaved=interleaved, magnitude=1.5)
        f = lambda t: (turn64(x.double() + t * direction.double(), pos, freqs, interleaved, 1.5)[0] * w.double()).sum()
        diff = float((f(0.5) - f(-0.5)))
        got = float((dx.double() * direction.double()).sum())
        tol = float((dx.double().abs() * direction.double().abs()).sum()) * 2.0 ** -8 + 1e-9
        tol += float(direction.double().abs().sum()) * 1.5 * 12 * 2.0 ** -20  # |a| + |b| < 12 here
        assert w.abs().max() < 6 and abs(got - diff) <= tol


def test_rope_on_a_side_stream_and_in_a_graph():
    q, k = normal(10, 300, 8, 128), normal(11, 300, 2, 128)
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    freqs = ops.rope_frequencies(128)
    want = ops.rope(q, k, pos, freqs)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = ops.rope(q, k, pos, freqs, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.rope(q, k, pos, freqs, q_out=qo, k_out=ko)
    pos.add_(1000)
    g.replay()
    torch.cuda.synchronize()
    again = ops.rope(q, k, pos, freqs)
    assert torch.equal(qo, again[0]) and torch.equal(ko, again[1])
    assert np.isfinite(qo.float().cpu().numpy()).all()
