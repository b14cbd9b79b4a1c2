"""Norms of queries and keys with the rotation in the same pass, and their gradient,
against the formula in 64 bits.

Tolerances, with u = 2^-24.  A sum of D squares (exact products, nineteen additions or
fewer on its way) errs by 19 u of itself, the mean's eps by u, so its inverse root by 10 u
and rsqrtf's own 4 u: r by 2^-20.  A normalised value has two more roundings.  The rotation
errs by 2^-20 m (|a| + |b|) for a pair (a, b) and magnitude m (see test_gpu_rope).  With
the rounding to bf16 (half a step, 2^-8):
  forward    2^-8 |y| + 2^-18 m (|a| + |b|) of the normalised pair (|y| where not rotated)
  gradient   let P = w m (|a| + |b|) of the incoming pair, n = x r, M = mean(P |n|).  g w errs
             by 2^-20 P, the mean by M (2^-20 + 2^-20 + 20 u), dx = r (g w - n mean) has three
             more roundings: 2^-8 |dx| + 2^-17 r (P + |n| M)
  weights    g n errs by 2^-19 of its magnitude A (P without w); a thread sums fewer than 64
             of them, then the sums of the lanes' groups (3 additions), 8 warps, ten CTAs or
             fewer and a tree of 32 (5): (2^-19 + 90 u) sum A, within 2^-17 sum A."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_cache import BF, built, i32, normal  # noqa: F401  (built: a fixture)
from .test_gpu_rope import turn64

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -134  # half a step of the smallest bf16 values


def norm64(x, w, eps):
    """x over its root mean square (fp64), one over that root, and the weights."""
    x = x.double()
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    return x * r, r, w.double()


def check_forward(got, x, w, pos, freqs, eps, interleaved, mag=1.0):
    n, _, wd = norm64(x, w, eps)
    want, pair = turn64(n * wd, pos, freqs, interleaved, mag)
    tol = want.abs() * 2.0 ** -8 + torch.maximum(pair, want.abs()) * 2.0 ** -18 + TINY
    err = (got.double() - want).abs()
    assert (err <= tol).all(), float((err - tol).max())


def gradient64(dy, x, w, pos, freqs, eps, interleaved, mag=1.0):
    n, r, wd = norm64(x, w, eps)
    g, pair = turn64(dy, pos, freqs, interleaved, mag, -1.0)
    A = torch.maximum(pair, g.abs())
    P = A * wd.abs()
    M = (P * n.abs()).mean(-1, keepdim=True)
    dx = r * (g * wd - n * (g * wd * n).mean(-1, keepdim=True))
    tol = dx.abs() * 2.0 ** -8 + (P + n.abs() * M) * r * 2.0 ** -17 + TINY
    over = tuple(range(dx.dim() - 1))
    return dx, tol, (g * n).sum(over), (A * n.abs()).sum(over) * 2.0 ** -17 + 1e-38


def check_gradient(got, got_w, *args):
    dx, tol, dw, wtol = gradient64(*args)
    err = (got.double() - dx).abs()
    assert (err <= tol).all(), float((err - tol).max())
    err = (got_w.double() - dw).abs()
    assert (err <= wtol).all(), float((err - wtol).max())


def weights(seed, d, dtype):
    return (1 + 0.3 * normal(seed, d).float()).to(dtype)


SIZES = [(1, 1, 1, 64, 64, False), (1, 32, 8, 128, 128, True), (7, 5, 3, 64, 16, False), (129, 6, 2, 128, 64, True),
         (1000, 9, 1, 128, 48, False), (3333, 33, 8, 64, 32, True), (2500, 32, 32, 128, 128, False), (64, 1, 70, 128, 16, False)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,hq,hk,d,rot,interleaved", SIZES)
def test_forward_and_gradient_match_the_formula(tokens, hq, hk, d, rot, interleaved, dtype):
    q, k = normal(1, tokens, hq, d) * 3, normal(2, tokens, hk, d)
    wq, wk = weights(3, d, dtype), weights(4, d, dtype)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda") * 17 + 3
    freqs = ops.rope_frequencies(rot, 10000.0)
    kw = dict(eps=1e-5, interleaved=interleaved, magnitude=1.25)
    qo, ko = ops.qk_norm_rope(q, k, wq, wk, pos, freqs, **kw)
    check_forward(qo, q, wq, pos, freqs, 1e-5, interleaved, 1.25)
    check_forward(ko, k, wk, pos, freqs, 1e-5, interleaved, 1.25)
    gq, gk = normal(5, tokens, hq, d), normal(6, tokens, hk, d)
    dq, dk, dwq, dwk = ops.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, pos, freqs, **kw)
    assert dwq.dtype == dwk.dtype == torch.float32
    check_gradient(dq, dwq, gq, q, wq, pos, freqs, 1e-5, interleaved, 1.25)
    check_gradient(dk, dwk, gk, k, wk, pos, freqs, 1e-5, interleaved, 1.25)
    qo, ko = ops.qk_norm_rope(q, None, wq, None, pos, freqs, **kw)
    assert ko is None
    check_forward(qo, q, wq, pos, freqs, 1e-5, interleaved, 1.25)
    again, dk, dw2, dwk = ops.qk_norm_rope_bwd(gq, None, q, None, wq, None, pos, freqs, **kw)
    assert dk is None and dwk is None and torch.equal(again, dq)
    check_gradient(again, dw2, gq, q, wq, pos, freqs, 1e-5, interleaved, 1.25)


def test_values_at_the_ends_of_the_range():
    """Rows of zeros, tiny and huge values (squares out of fp32's range), infinities and NaN."""
    d = 128
    x = normal(1, 9, 2, d)
    x[0] = 0
    x[1] *= 2.0 ** -40
    x[2] *= 2.0 ** 100
    x[3] *= 2.0 ** 125
    x[4] *= 2.0 ** -130
    x[5, :, ::2] *= 2.0 ** 120
    w = weights(2, d, torch.float32)
    pos, freqs = i32(list(range(9))), ops.rope_frequencies(64)
    y, _ = ops.qk_norm_rope(x, None, w, None, pos, freqs)
    check_forward(y, x, w, pos, freqs, 1e-6, False)
    dy = normal(3, 9, 2, d)
    dx, _, dw, _ = ops.qk_norm_rope_bwd(dy, None, x, None, w, None, pos, freqs)
    check_gradient(dx, dw, dy, x, w, pos, freqs, 1e-6, False)
    # an infinite value makes a NaN of itself and its pair, and zeros of the rest of its head
    x[6, 0, 3] = float("inf")
    x[7, 1, 100] = float("nan")
    z, _ = ops.qk_norm_rope(x, None, w, None, pos, freqs)
    odd = torch.zeros_like(z, dtype=torch.bool)
    odd[6, 0, 3] = odd[6, 0, 35] = True
    odd[7, 1] = True
    assert z[odd].isnan().all() and (z[6, 0][~odd[6, 0]] == 0).all()
    keep = torch.ones(9, 2, dtype=torch.bool)
    keep[6, 0] = keep[7, 1] = False
    assert torch.equal(z[keep], y[keep])


def test_far_and_negative_positions():
    pos = i32([0, 1, -1, 2 ** 20 + 1, 2 ** 24 + 3, 2 ** 31 - 1, -2 ** 31])
    freqs = ops.rope_frequencies(128, 500000.0, ops.ROPE_BANDS, factor=8.0, original_length=8192)
    q, w = normal(3, pos.numel(), 4, 128), weights(4, 128, BF)
    check_forward(ops.qk_norm_rope(q, None, w, None, pos, freqs)[0], q, w, pos, freqs, 1e-6, False)
    g = normal(5, pos.numel(), 4, 128)
    dq, _, dw, _ = ops.qk_norm_rope_bwd(g, None, q, None, w, None, pos, freqs)
    check_gradient(dq, dw, g, q, w, pos, freqs, 1e-6, False)


def test_slices_of_a_projection_and_in_place():
    T, hq, hk, d = 77, 8, 2, 128
    qkv = normal(5, T, hq + 2 * hk, d)
    ref = qkv.clone()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    wq, wk = weights(6, d, BF), weights(7, d, BF)
    pos, freqs = torch.arange(T, dtype=torch.int32, device="cuda"), ops.rope_frequencies(d)
    qo, ko = ops.qk_norm_rope(q, k, wq, wk, pos, freqs)
    check_forward(qo, ref[:, :hq], wq, pos, freqs, 1e-6, False)
    check_forward(ko, ref[:, hq:hq + hk], wk, pos, freqs, 1e-6, False)
    # gradients into slices of the projection's gradient, in place over the incoming ones
    grad = normal(8, T, hq + 2 * hk, d)
    gq, gk, gv = grad[:, :hq].clone(), grad[:, hq:hq + hk].clone(), grad[:, hq + hk:].clone()
    want = ops.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, pos, freqs)
    check_gradient(want[0], want[2], gq, q, wq, pos, freqs, 1e-6, False)
    check_gradient(want[1], want[3], gk, k, wk, pos, freqs, 1e-6, False)
    got = ops.qk_norm_rope_bwd(grad[:, :hq], grad[:, hq:hq + hk], q, k, wq, wk, pos, freqs, dq=grad[:, :hq],
                               dk=grad[:, hq:hq + hk])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(grad[:, hq + hk:], gv)
    assert torch.equal(qkv, ref)
    ops.qk_norm_rope(q, k, wq, wk, pos, freqs, q_out=q, k_out=k)  # in the projection itself
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, ref[:, hq + hk:])
    # a batch, every second token of a longer one
    x = normal(9, 2, 50, 3, 64)
    p2, f2, w2 = torch.arange(50, dtype=torch.int32, device="cuda"), ops.rope_frequencies(64), weights(10, 64, BF)
    part = x[:, ::2]
    check_forward(ops.qk_norm_rope(part, None, w2, None, p2, f2)[0], part, w2, p2, f2, 1e-6, False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_operands_aligned_to_sixteen_bytes(interleaved):
    T, hq, d = 33, 3, 64
    w, pos, freqs = weights(1, d, BF), torch.arange(T, dtype=torch.int32, device="cuda"), ops.rope_frequencies(d)
    wide, off = hq * d + 8, 8  # rows of 200 values, from the eighth on

    def rows(seed):
        return normal(seed, T * wide + off)[off:].view(T, wide)[:, :hq * d].view(T, hq, d)

    q, g, out = rows(2), rows(3), rows(4)
    assert q.data_ptr() % 32 == 16 and q.stride(0) * 2 % 32 == 16
    for operands in ((q, g, out), (q.contiguous(), g, None), (q, g.contiguous(), None), (q.contiguous(), g.contiguous(), out)):
        x, dy, dq = operands
        got, _, dw, _ = ops.qk_norm_rope_bwd(dy, None, x, None, w, None, pos, freqs, interleaved=interleaved, dq=dq)
        check_gradient(got, dw, dy, x, w, pos, freqs, 1e-6, interleaved)
        y, _ = ops.qk_norm_rope(x, None, w, None, pos, freqs, interleaved=interleaved, q_out=dq)
        check_forward(y, x, w, pos, freqs, 1e-6, interleaved)


def test_gradient_against_differences():
    """Along a direction in q and one in the weights, against central differences of the
    64-bit formula (step 1e-5, whose own error is far below 1e-6 of the magnitudes here)."""
    T, h, d, eps, step = 5, 2, 64, 1e-3, 1e-5
    pos = i32([0, 9, 100, 5000, 70000])
    freqs = ops.rope_frequencies(32)
    x, dy, along = (normal(s, T, h, d) for s in (7, 8, 9))
    w, turn = weights(10, d, torch.float32), normal(11, d)
    for interleaved in (False, True):
        dx, _, dw, _ = ops.qk_norm_rope_bwd(dy, None, x, None, w, None, pos, freqs, eps=eps, interleaved=interleaved,
                                            magnitude=1.5)

        def f(s, t):
            n, _, wd = norm64(x.double() + s * along.double(), w.double() + t * turn.double(), eps)
            return float((turn64(n * wd, pos, freqs, interleaved, 1.5)[0] * dy.double()).sum())

        _, tol, _, wtol = gradient64(dy, x, w, pos, freqs, eps, interleaved, 1.5)
        size = float(dy.double().abs().sum()) * 1e-6
        got = float((dx.double() * along.double()).sum())
        assert abs(got - (f(step, 0) - f(-step, 0)) / (2 * step)) <= float((tol * along.double().abs()).sum()) + size
        got = float((dw.double() * turn.double()).sum())
        assert abs(got - (f(0, step) - f(0, -step)) / (2 * step)) <= float((wtol * turn.double().abs()).sum()) + size


def test_equal_calls_give_equal_bits_and_workspaces_hold():
    T, hq, hk, d = 4001, 12, 3, 64
    q, k, gq, gk = (normal(s, T, h, d) for s, h in ((1, hq), (2, hk), (3, hq), (4, hk)))
    w = weights(5, d, BF)
    pos, freqs = torch.arange(T, dtype=torch.int32, device="cuda"), ops.rope_frequencies(d)
    want = ops.qk_norm_rope_bwd(gq, gk, q, k, w, w, pos, freqs)
    need = ops.qk_norm_rope_bwd_workspace_size(T, hq, hk, d)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")  # (NaN sums, were they read)
    got = ops.qk_norm_rope_bwd(gq, gk, q, k, w, w, pos, freqs, workspace=ws[:need])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and (ws[need:] == 255).all()
    with pytest.raises(RuntimeError):
        ops.qk_norm_rope_bwd(gq, gk, q, k, w, w, pos, freqs, workspace=ws[:need - 256])
    check_gradient(want[1], want[3], gk, k, w, pos, freqs, 1e-6, False)


def test_a_side_stream_and_a_graph():
    T, hq, hk, d = 300, 8, 2, 128
    q, k, gq, gk = (normal(s, T, h, d) for s, h in ((1, hq), (2, hk), (3, hq), (4, hk)))
    wq, wk = weights(5, d, BF), weights(6, d, BF)
    pos, freqs = torch.arange(T, dtype=torch.int32, device="cuda"), ops.rope_frequencies(128)

    def both(stream=None):
        return (*ops.qk_norm_rope(q, k, wq, wk, pos, freqs, stream=stream),
                *ops.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, pos, freqs, stream=stream))

    want = both()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = both(st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.empty_like(x) for x in want]
    ws = torch.empty(ops.qk_norm_rope_bwd_workspace_size(T, hq, hk, d), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.qk_norm_rope(q, k, wq, wk, pos, freqs, q_out=outs[0], k_out=outs[1])
        ops.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, pos, freqs, dq=outs[2], dk=outs[3], dq_weight=outs[4],
                             dk_weight=outs[5], workspace=ws)
    pos.add_(1000)
    q.mul_(2).add_(1)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, both()))


def test_one_token_of_an_odd_stride():
    """A single token's stride does not matter."""
    q = normal(1, 203).as_strided((1, 3, 64), (203, 64, 1))
    assert q.stride(0) % 8
    w, pos, freqs = weights(2, 64, BF), i32([9]), ops.rope_frequencies(64)
    check_forward(ops.qk_norm_rope(q, None, w, None, pos, freqs)[0], q, w, pos, freqs, 1e-6, False)
    assert torch.equal(ops.rope(q, None, pos, freqs)[0], ops.rope(q.contiguous(), None, pos, freqs)[0])
    dq, _, dw, _ = ops.qk_norm_rope_bwd(q, None, q, None, w, None, pos, freqs)
    check_gradient(dq, dw, q, q, w, pos, freqs, 1e-6, False)


def test_no_tokens():
    q, k = normal(1, 0, 4, 64), normal(2, 0, 2, 64)
    w, pos, freqs = weights(3, 64, BF), i32([]), ops.rope_frequencies(64)
    qo, ko = ops.qk_norm_rope(q, k, w, w, pos, freqs)
    assert qo.shape == q.shape and ko.shape == k.shape
    dq, dk, dwq, dwk = ops.qk_norm_rope_bwd(q, k, q, k, w, w, pos, freqs)
    assert dq.shape == q.shape and dk.shape == k.shape and (dwq == 0).all() and (dwk == 0).all()


def test_a_training_step_through_the_attention():
    """Projection slices -> norms and rotation -> attention, and back: the calls of a
    layer's step fit together.  The gradient that reaches q and k is checked against the
    formula applied to the attention's own gradients."""
    B, S, H, D = 2, 256, 2, 128
    x = normal(1, B, S, 3 * H, D)
    q, k, v = x[:, :, :H], x[:, :, H:2 * H], x[:, :, 2 * H:]
    wq, wk = weights(2, D, BF), weights(3, D, BF)
    pos = torch.arange(S, dtype=torch.int32, device="cuda").repeat(B)
    freqs = ops.rope_frequencies(D)
    qr, kr = ops.qk_norm_rope(q, k, wq, wk, pos, freqs)
    assert qr.is_contiguous() and qr.shape == q.shape
    vc = v.contiguous()
    out, lse = ops.attn_fwd(qr, kr, vc, 64, 2)
    dout = normal(4, B, S, H, D)
    gq, gk, _ = ops.attn_bwd(qr, kr, vc, out, lse, dout, 64, 2)
    dx = torch.zeros_like(x)
    dq, dk, dwq, dwk = ops.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, pos, freqs, dq=dx[:, :, :H], dk=dx[:, :, H:2 * H])
    assert ops.get_status() == ops.MOBA_OK and gq.abs().max() > 0
    flat = lambda t: t.reshape(B * S, H, D)
    check_gradient(flat(dq), dwq, flat(gq), flat(q), wq, pos, freqs, 1e-6, False)
    check_gradient(flat(dk), dwk, flat(gk), flat(k), wk, pos, freqs, 1e-6, False)


@pytest.mark.parametrize("hq,hk,d,interleaved", [(32, 8, 128, False), (9, 64, 64, True)])
def test_calls_of_several_waves(hq, hk, d, interleaved):
    """Tokens enough for CTAs in waves.  A thread of the gradient sums 24 products or fewer here, and
    40 CTAs or fewer on its way: 2^-19 + (24 + 3 + 8 + 40 + 5) u, within 2^-17 as above."""
    tokens = 104000000 // ((hq + hk) * d)
    q, k = normal(1, tokens, hq, d), normal(2, tokens, hk, d)
    wq, wk, freqs = weights(3, d, BF), weights(4, d, BF), ops.rope_frequencies(d)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda") * 3
    a, b = ops.qk_norm_rope(q, k, wq, wk, pos, freqs, interleaved=interleaved)
    dq, dk = normal(5, tokens, hq, d), normal(6, tokens, hk, d)
    got = ops.qk_norm_rope_bwd(dq, dk, q, k, wq, wk, pos, freqs, interleaved=interleaved)
    assert ops.get_status() == ops.MOBA_OK
    for x, y, dy, w, dx, dw in ((q, a, dq, wq, got[0], got[2]), (k, b, dk, wk, got[1], got[3])):
        check_forward(y, x, w, pos, freqs, 1e-6, interleaved)
        check_gradient(dx, dw, dy, x, w, pos, freqs, 1e-6, interleaved)
