"""Appending with norms and rotation on the way: the same bits as the norms (or the
rotation) and the append one after the other, whose own tests hold them to 64 bits
(test_gpu_qk_norm, test_gpu_rope, test_gpu_paged_cache)."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_cache import BF, Cache, built, i32, normal  # noqa: F401  (built: a fixture)
from .test_gpu_qk_norm import check_forward, weights

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a.view(torch.int16 if a.dtype == BF else torch.int32), b.view(torch.int16 if b.dtype == BF else torch.int32))


def offsets(nq):
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    return cu


def fused(c, q, k, v, cu, lens, freqs, max_new=None, **kw):
    most = max_new or max(b - a for a, b in zip(cu, cu[1:])) or 1
    return ops.paged_append_rope(q, k, v, c.k, c.v, c.kbar, c.table, i32(cu), i32(lens), most, c.block, freqs, **kw)


def apart(c, q, k, v, cu, lens, freqs, positions=None, q_weight=None, k_weight=None, pooling=ops.POOL_MEAN, **kw):
    """The same by the calls for each step, positions made on the host."""
    if positions is None:
        positions = i32([p for a, b, n in zip(cu, cu[1:], lens) for p in range(n - (b - a), n)])
    rot = {n: kw[n] for n in ("interleaved", "magnitude") if n in kw}
    turned = []
    for x, w in ((q, q_weight), (k, k_weight)):
        if w is None:
            turned.append(ops.rope(x, None, positions, freqs, **rot)[0])
        else:
            turned.append(ops.qk_norm_rope(x, None, w, None, positions, freqs, eps=kw.get("eps", 1e-6), **rot)[0])
    c.append(turned[1], v.contiguous(), cu, lens, pooling)
    return turned[0]


@pytest.mark.parametrize("hq,hkv,d,rot,page,block,inter,wq,wk,pooling", [
    (4, 2, 64, 64, 16, 64, False, True, True, ops.POOL_MEAN), (8, 8, 128, 128, 32, 128, True, True, True, ops.POOL_MAX),
    (5, 1, 128, 48, 64, 64, False, False, False, ops.POOL_MEAN), (40, 8, 128, 64, 128, 512, False, True, False, ops.POOL_MEAN),
    (3, 3, 64, 16, 16, 192, True, False, True, ops.POOL_MEAN)])
def test_uneven_chunks(hq, hkv, d, rot, page, block, inter, wq, wk, pooling):
    lens = [700, 1, 64, 513, 0, 1024]
    steps = [[1, 1, 0, 200, 0, 63], [299, 0, 64, 1, 0, 1], [0, 0, 0, 310, 0, 449], [400, 0, 0, 2, 0, 511]]
    one, two = (Cache(len(lens), 1024, hkv, d, page, block) for _ in range(2))
    freqs = ops.rope_frequencies(rot)
    kw = dict(interleaved=inter, magnitude=1.1, pooling=pooling, eps=1e-5,
              q_weight=weights(1, d, torch.float32) if wq else None, k_weight=weights(2, d, torch.float32) if wk else None)
    at = [0] * len(lens)
    for i, step in enumerate(steps):
        at = [a + n for a, n in zip(at, step)]
        x = normal(10 + i, sum(step), hq + 2 * hkv, d)  # slices of one projection
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        cu = offsets(step)
        got = fused(one, q, k, v, cu, at, freqs, **kw)
        assert got.is_contiguous() and same(got, apart(two, q, k, v, cu, at, freqs, **kw))
    assert at == lens and ops.get_status() == ops.MOBA_OK
    assert same(one.k, two.k) and same(one.v, two.v) and same(one.kbar, two.kbar)


def test_against_the_formula():
    nq, lens, hq, hkv, d = [130, 1, 70], [300, 64, 128], 6, 2, 128
    c = Cache(3, 320, hkv, d, 32, 64)
    old = [n - m for n, m in zip(lens, nq)]
    c.append(normal(1, sum(old), hkv, d), normal(2, sum(old), hkv, d), offsets(old), old)
    q, k, v = (normal(s, sum(nq), h, d) for s, h in ((3, hq), (4, hkv), (5, hkv)))
    wq, wk, freqs = weights(6, d, BF), weights(7, d, BF), ops.rope_frequencies(64)
    pos = i32([p for n, m in zip(lens, nq) for p in range(n - m, n)])
    out = fused(c, q, k, v, offsets(nq), lens, freqs, q_weight=wq, k_weight=wk, interleaved=True)
    assert ops.get_status() == ops.MOBA_OK
    check_forward(out, q, wq, pos, freqs, 1e-6, True)
    row = 0
    for b, (n, m) in enumerate(zip(lens, nq)):
        stored = c.read(c.k, b, n)
        check_forward(stored[n - m:], k[row:row + m], wk, pos[row:row + m], freqs, 1e-6, True)
        assert same(c.read(c.v, b, n)[n - m:].contiguous(), v[row:row + m])
        for blk in range((n - m) // 64, n // 64):  # (the mean's tolerance: test_gpu_paged_cache)
            x = stored[blk * 64:(blk + 1) * 64].double()
            slot = int(c.table[b, (blk + 1) * 64 // 32 - 1])
            assert ((c.kbar[slot].double() - x.mean(0)).abs() <= 8 * 2.0 ** -24 * x.abs().mean(0)).all()
        row += m


@pytest.mark.parametrize("where", [0, 17, 39])
def test_steps_beside_a_long_chunk(where):
    n = 40
    lens, nq = [63 + 7 * b for b in range(n)], [1 + b % 2 for b in range(n)]
    lens[where], nq[where] = 1500, 1401
    one, two = (Cache(n, 1536, 2, 64, 16, 64) for _ in range(2))
    old = [a - b for a, b in zip(lens, nq)]
    before = normal(1, sum(old), 2, 64)
    for c in (one, two):
        c.append(before, before, offsets(old), old)
    q, k, v = (normal(s, sum(nq), h, 64) for s, h in ((2, 6), (3, 2), (4, 2)))
    freqs, w = ops.rope_frequencies(64), weights(5, 64, BF)
    got = fused(one, q, k, v, offsets(nq), lens, freqs, q_weight=w, k_weight=w)
    assert same(got, apart(two, q, k, v, offsets(nq), lens, freqs, q_weight=w, k_weight=w))
    assert same(one.k, two.k) and same(one.v, two.v) and same(one.kbar, two.kbar) and ops.get_status() == ops.MOBA_OK


def test_positions_of_the_callers_and_in_place():
    nq, lens = [3, 70], [3, 200]
    one, two = (Cache(2, 256, 2, 64, 32, 64) for _ in range(2))
    x = normal(1, 73, 8, 64)
    ref = x.clone()
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    pos, freqs, w = i32([(7 * i) % 5000 - 9 for i in range(73)]), ops.rope_frequencies(32), weights(2, 64, BF)
    want = apart(two, q, k, v, offsets(nq), lens, freqs, positions=pos, q_weight=w)
    got = fused(one, q, k, v, offsets(nq), lens, freqs, positions=pos, q_weight=w, q_out=q)
    assert got.data_ptr() == x.data_ptr() and same(got.contiguous(), want)
    assert torch.equal(x[:, 4:], ref[:, 4:]) and same(one.k, two.k) and same(one.v, two.v)


def test_without_pooled_keys():
    c = Cache(1, 128, 2, 64, 16, 64)
    q, k, v = (normal(s, 100, h, 64) for s, h in ((1, 4), (2, 2), (3, 2)))
    freqs = ops.rope_frequencies(64)
    ops.paged_append_rope(q, k, v, c.k, c.v, None, c.table, i32([0, 100]), i32([100]), 100, 64, freqs)
    assert c.kbar.isnan().all() and same(c.read(c.k, 0, 100), ops.rope(k, None, torch.arange(100, dtype=torch.int32, device="cuda"), freqs)[0])


def test_rows_of_nothing_stay():
    """Padding behind the last sequence, empty sequences, refused sequences and bad pages."""
    c = Cache(5, 256, 2, 64, 16, 64)
    page = c.table[3, 1].clone()
    c.table[3, 1] = c.P  # a page outside the pool: tokens 16 to 31 of the fourth sequence
    nq, lens = [5, 0, 9, 20, 70], [5, 17, 9, 40, 130]
    q, k, v = (normal(s, 130, h, 64) for s, h in ((1, 4), (2, 2), (3, 2)))
    cu, freqs, w = [0, 5, 5, 14, 34, 104], ops.rope_frequencies(64), weights(4, 64, BF)
    lens[2] = 8  # fewer than its new tokens: refused
    out = torch.full_like(q, 7.0)
    fused(c, q, k, v, cu, lens, freqs, q_weight=w, k_weight=w, q_out=out)
    assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    c.table[3, 1] = page  # (read below, as it was before)
    assert c.read(c.k, 3, 32).isnan().all() and c.read(c.v, 3, 32).isnan().all()
    pos = i32([p for n, m in zip(lens, nq) for p in range(n - m, n)] + [0] * 26)
    want = ops.qk_norm_rope(q, k, w, w, pos, freqs)
    good = torch.zeros(130, dtype=torch.bool, device="cuda")
    good[:5] = good[14:104] = True
    assert (out[~good] == 7).all() and same(out[good], want[0][good])
    assert c.read(c.k, 2, 9).isnan().all() and c.read(c.v, 2, 9).isnan().all()
    for b, lo, hi, row in ((0, 0, 5, 0), (3, 32, 40, 26), (4, 60, 130, 34)):
        assert same(c.read(c.k, b, hi)[lo:].contiguous(), want[1][row:row + hi - lo])
        assert same(c.read(c.v, b, hi)[lo:].contiguous(), v[row:row + hi - lo])
    assert not c.kbar[c.table[4, 7].long()].isnan().any()  # its block of tokens 64 to 127 is complete
    # every offset wrong: nothing is touched
    before = c.k.clone()
    for cu in ([-9, 200, 3, 90, -1, 5000], [90, 80, 70, 60, 50, 40]):
        out.fill_(7.0)
        fused(c, q, k, v, cu, [0] * 5, freqs, max_new=20, q_out=out)
        assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
        assert (out == 7).all() and same(c.k, before)


def test_infinite_and_nan_keys():
    """They are stored as the formula gives them, and reach the pooled keys only."""
    one, two = (Cache(1, 128, 1, 64, 16, 64) for _ in range(2))
    q, k, v = (normal(s, 128, 1, 64) for s in (1, 2, 3))
    k[3, 0, 5], k[100, 0, 60], v[7] = float("inf"), float("nan"), float("-inf")
    freqs = ops.rope_frequencies(32)
    for w in (None, weights(4, 64, BF)):
        got = fused(one, q, k, v, [0, 128], [128], freqs, k_weight=w)
        assert same(got, apart(two, q, k, v, [0, 128], [128], freqs, k_weight=w))
        assert torch.equal(one.k.isnan(), two.k.isnan()) and same(one.k.nan_to_num(), two.k.nan_to_num())
        assert same(one.v, two.v) and same(one.kbar.nan_to_num(), two.kbar.nan_to_num())


def test_many_sequences():
    """More sequences than lanes look up at once, some of them empty."""
    n = 1500
    nq = [(b * 7) % 4 for b in range(n)]
    lens = [b % 60 + m for b, m in enumerate(nq)]
    one, two = (Cache(n, 64, 1, 64, 16, 64) for _ in range(2))
    q, k, v = (normal(s, sum(nq), h, 64) for s, h in ((1, 2), (2, 1), (3, 1)))
    freqs = ops.rope_frequencies(64)
    got = fused(one, q, k, v, offsets(nq), lens, freqs)
    assert same(got, apart(two, q, k, v, offsets(nq), lens, freqs)) and ops.get_status() == ops.MOBA_OK
    assert same(one.k, two.k) and same(one.v, two.v)


def test_a_side_stream_and_a_graph():
    """Captured with tables that are rewritten in place; the pooling waits for its pages."""
    one, two = (Cache(3, 512, 2, 128, 32, 64) for _ in range(2))
    q, k, v = (normal(s, 3, h, 128) for s, h in ((1, 4), (2, 2), (3, 2)))
    freqs, w = ops.rope_frequencies(128), weights(4, 128, BF)
    cu, lens, out = i32([0, 1, 2, 3]), i32([1, 1, 1]), torch.empty_like(q)
    g = torch.cuda.CUDAGraph()

    def call(c, **kw):
        return ops.paged_append_rope(q, k, v, c.k, c.v, c.kbar, c.table, cu, lens, 1, 64, freqs, q_weight=w, k_weight=w, **kw)

    for c in (one, two):
        call(c, q_out=out)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call(one, q_out=out)
    st = torch.cuda.Stream()
    for n in range(1, 200):
        lens.copy_(i32([n, 2 * n, n + 64]))
        q.copy_(normal(n, 3, 4, 128))
        k.copy_(normal(1000 + n, 3, 2, 128))
        st.wait_stream(torch.cuda.current_stream())
        got = call(two, stream=st)
        torch.cuda.current_stream().wait_stream(st)
        g.replay()
        assert same(out, got)
    assert same(one.k, two.k) and same(one.v, two.v) and same(one.kbar, two.kbar)
    assert ops.get_status() == ops.MOBA_OK


def test_no_tokens():
    c = Cache(1, 64, 2, 64, 16, 64)
    out = fused(c, normal(1, 0, 4, 64), normal(2, 0, 2, 64), normal(3, 0, 2, 64), [0, 0], [5], ops.rope_frequencies(64), max_new=1)
    assert out.shape == (0, 4, 64) and c.k.isnan().all()


@pytest.mark.parametrize("hkv,d,page,block,pooling", [(8, 64, 16, 64, ops.POOL_MEAN), (8, 128, 32, 128, ops.POOL_MAX),
                                                      (3, 128, 16, 192, ops.POOL_MEAN)])
@pytest.mark.parametrize("seqs", [7, 150])
def test_blocks_completed_by_few_sequences_and_by_many(seqs, hkv, d, page, block, pooling):
    """Blocks that one new token, several or all of them complete, in calls of few candidates for
    pooling and in calls of more than the GPU takes at once."""
    lens = [block * (1 + b % 3) - (b % 5) * (b % 2) for b in range(seqs)]
    new = [1 + 7 * b % 13 if b % 4 else min(n, block + 5) for b, n in enumerate(lens)]
    old = [n - m for n, m in zip(lens, new)]
    one, two = (Cache(seqs, 3 * block, hkv, d, page, block) for _ in range(2))
    x = normal(1, sum(old), 2 * hkv, d)
    for c in (one, two):
        c.append(x[:, :hkv].contiguous(), x[:, hkv:].contiguous(), offsets(old), old, pooling)
    q, k, v = (normal(s, sum(new), hkv, d) for s in (2, 3, 4))
    kw = dict(pooling=pooling, k_weight=weights(5, d, BF))
    freqs = ops.rope_frequencies(d)
    got = fused(one, q, k, v, offsets(new), lens, freqs, **kw)
    assert same(got, apart(two, q, k, v, offsets(new), lens, freqs, **kw))
    assert same(one.k, two.k) and same(one.v, two.v) and same(one.kbar, two.kbar) and ops.get_status() == ops.MOBA_OK
