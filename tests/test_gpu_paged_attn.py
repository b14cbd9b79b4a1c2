"""Attention of new tokens over a paged cache against the definition in 64 bits.

Selections are equal to the 64-bit ones.  For an output value let w be the row's
softmax weights, A = sum w |v| and d the largest error of a logit; a logit is an
fp32 sum of D bf16 products, so d <= D 2^-23 sum |q||k| / sqrt(D).  Rounding P
to bf16 adds at most 2^-8 A, errors of the logits (in numerator and sum) 2 d A,
fp32 exponentials and sums less than 2^-18 A, the rounding of the result 2^-8 of
it.  lse errs by at most d, and 2^-20 (1 + |lse|) for its own arithmetic."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_cache import BF, Cache, built, i32, normal  # noqa: F401  (built: a fixture)

pytestmark = pytest.mark.gpu


def filled(lens, hkv, d, page, block, seed=0, slack=0, offset=0.5):
    """A cache holding the sequences, and their keys and values."""
    most = max(lens) + slack
    c = Cache(len(lens), -(-most // block) * block, hkv, d, page, block, seed)
    ks, vs = [], []
    for b, n in enumerate(lens):
        k = normal(seed + 7 * b + 1, n, hkv, d)
        off = offset * normal(seed + 7 * b + 2, n // block + 1, hkv, d)
        ks.append((k + off[torch.arange(n, device="cuda") // block]).to(BF))
        vs.append(normal(seed + 7 * b + 3, n, hkv, d))
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    c.append(torch.cat(ks), torch.cat(vs), cu, lens)
    return c, ks, vs


def expect(q, ks, vs, c, nq, lens, block, topk):
    """out, lse, idx, and the tolerances of out and lse, all fp64, by the definition."""
    hq, d = q.shape[1:]
    dev = q.device
    out = torch.zeros(*q.shape, dtype=torch.float64, device=dev)
    lse = torch.full(q.shape[:2], -float("inf"), dtype=torch.float64, device=dev)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    idx = torch.full((*q.shape[:2], topk), -1, dtype=torch.int64, device=dev)
    row = 0
    for b, (n, length) in enumerate(zip(nq, lens)):
        if n == 0:
            continue
        group = hq // ks[b].shape[1]
        k, v = (x[b].double().repeat_interleave(group, 1).transpose(0, 1) for x in (ks, vs))
        x = q[row:row + n].double().transpose(0, 1)  # [hq][n][d]
        at = torch.arange(length - n, length, device=dev)
        mine = at // block
        blocks = torch.arange(length // block + 1, device=dev)
        chosen = blocks == mine[:, None]  # [n][blocks]
        chosen = chosen.expand(hq, -1, -1).clone()
        past = length // block
        if topk > 1 and past:
            if topk > past:
                chosen |= blocks < mine[:, None]
            else:
                slot = c.table[b, torch.arange(past, device=dev) * (block // c.page) + block // c.page - 1].long()
                kb = c.kbar[slot].double().repeat_interleave(group, 1).permute(1, 2, 0)
                s = (x @ kb).nan_to_num(nan=-float("inf"), posinf=float("inf"), neginf=-float("inf"))
                order = torch.where(blocks[:past] < mine[:, None], 0, 1).expand_as(s)
                # past blocks by score, ties low; then the others
                first = torch.sort(s, dim=-1, descending=True, stable=True).indices
                second = torch.sort(order.gather(-1, first), dim=-1, stable=True).indices
                best = first.gather(-1, second)[..., :topk - 1]
                keep = best < mine[:, None]
                chosen.scatter_(-1, torch.where(keep, best, mine[:, None].expand_as(best)), True)
        logit = x @ k.transpose(1, 2) * d ** -0.5
        key = torch.arange(length, device=dev)
        seen = (key <= at[:, None]) & chosen[..., key // block]
        logit = logit.masked_fill(~seen, -float("inf"))
        z = torch.logsumexp(logit, -1)
        w = torch.exp(logit - z[..., None])
        o = w @ v
        # (a key whose logit is -inf has weight 0 with or without errors)
        size = (x.abs() @ k.abs().transpose(1, 2)).masked_fill(~seen | logit.isneginf(), 0)
        err = d * 2.0 ** -23 * d ** -0.5 * size.amax(-1)
        A = w @ v.abs()
        out[row:row + n], lse[row:row + n] = o.transpose(0, 1), z.T
        tol[row:row + n] = (2.0 ** -8 * o.abs() + A * (2.0 ** -8 + 2.0 ** -18 + 2 * err[..., None])).transpose(0, 1)
        ltol[row:row + n] = (err + 2.0 ** -20 * (1 + z.abs())).T
        m = min(topk, blocks.numel())
        got = torch.where(chosen, blocks, blocks.numel()).sort(-1).values[..., :m]
        idx[row:row + n, :, :m] = torch.where(got < blocks.numel(), got, -1).transpose(0, 1)
        row += n
    return out, lse, idx, tol, ltol


def compare(got, want):
    out, lse, idx, tol, ltol = want
    if got[2] is not None:
        assert torch.equal(got[2].long(), idx)
    err = (got[0].double() - out).abs()
    assert (err <= tol).all(), float((err - tol).max())
    err = (got[1].double() - lse).abs()
    assert (err <= ltol).all(), float((err - ltol).max())


def attend(c, q, nq, lens, block, topk, **kw):
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    return ops.paged_attn(q, c.k, c.v, c.kbar, c.table, i32(cu), i32(lens), max(nq), block, topk, **kw)


def case(nq, lens, hq, hkv, d, page, block, topk, seed=0, q=None, slack=0, with_idx=True):
    c, ks, vs = filled(lens, hkv, d, page, block, seed, slack)
    if q is None:
        q = normal(seed + 99, sum(nq), hq, d)
    got = attend(c, q, nq, lens, block, topk, with_idx=with_idx)
    assert ops.get_status() == ops.MOBA_OK
    compare(got, expect(q, ks, vs, c, nq, lens, block, topk))
    return got


@pytest.mark.parametrize("topk", [1, 2, 3, 5, 9, 32, 100])
@pytest.mark.parametrize("hq,hkv,d,page,block", [(4, 4, 64, 16, 64), (8, 2, 128, 32, 128), (5, 1, 128, 64, 64)])
def test_one_new_token(hq, hkv, d, page, block, topk):
    lens = [2500, 1, 64, 65, 700, 128, 1999]
    case([1] * len(lens), lens, hq, hkv, d, page, block, topk, seed=topk)


@pytest.mark.parametrize("topk", [1, 3, 6, 64])
@pytest.mark.parametrize("hq,hkv,d,page,block", [(2, 2, 64, 16, 64), (6, 2, 128, 32, 128), (16, 1, 128, 128, 256),
                                                 (64, 1, 64, 16, 64), (14, 2, 64, 64, 192)])
def test_chunks_of_uneven_sizes(hq, hkv, d, page, block, topk):
    nq = [7, 0, 130, 1, 64, 33]
    lens = [7, 50, 1500, 640, 64, 2049]
    case(nq, lens, hq, hkv, d, page, block, topk, seed=3 + topk, slack=77)


@pytest.mark.parametrize("topk", [3, 64])
@pytest.mark.parametrize("n,length,hq,hkv,d,page,block", [
    (1000, 3333, 8, 2, 128, 64, 256), (777, 777, 4, 4, 64, 16, 64), (300, 5000, 12, 4, 128, 16, 512),
    (515, 2111, 7, 1, 64, 32, 128), (2048, 2048, 3, 1, 128, 128, 128)])
def test_a_long_chunk(n, length, hq, hkv, d, page, block, topk):
    case([n], [length], hq, hkv, d, page, block, topk, seed=n, with_idx=topk < 64)


def test_prefill_and_decode_steps_in_one_call():
    case([1, 600, 1, 1, 3, 1], [900, 2000, 17, 2300, 1200, 1], 8, 2, 128, 32, 128, 4, seed=8)


@pytest.mark.parametrize("topk", [50, 64])
def test_selection_of_every_block(topk):
    nq, lens = [3, 70, 0, 1, 33], [2500, 90, 5, 64, 1000]
    case(nq, lens, 8, 2, 64, 16, 64, topk, seed=31, slack=100)


@pytest.mark.parametrize("topk", [3, 1000])
def test_many_steps_beside_one_long_chunk(topk):
    lens = [700 + 13 * i for i in range(40)] + [1500]
    nq = [1 + i % 3 for i in range(40)] + [900]
    order = [40] + list(range(40)) if topk == 3 else list(range(41))
    case([nq[i] for i in order], [lens[i] for i in order], 8, 2, 64, 16, 64, topk, seed=9, with_idx=topk < 100)


@pytest.mark.parametrize("hq,hkv,d,block,topk", [(16, 4, 128, 512, 3), (16, 4, 64, 512, 2), (16, 4, 128, 64, 200),
                                                 (12, 4, 128, 128, 3), (16, 4, 64, 64, 200)])
def test_several_new_tokens_of_many_sequences(hq, hkv, d, block, topk):
    nq = [9 + 3 * (i % 2) for i in range(16)]
    nq[5] = 0
    lens = [400 + 97 * i for i in range(16)]
    case(nq, lens, hq, hkv, d, 32, block, topk, seed=41, with_idx=topk < 100)


def test_ties_go_to_the_lower_block():
    # equal keys in every block, and queries of zeros: every score ties
    c, ks, vs = filled([1024, 900], 2, 64, 16, 64, seed=4)
    for b, n in enumerate((1024, 900)):
        ks[b] = normal(5, 64, 2, 64).repeat(16, 1, 1)[:n]
    c.append(torch.cat(ks), torch.cat(vs), [0, 1024, 1924], [1024, 900])
    for q in (normal(6, 80, 4, 64), torch.zeros(80, 4, 64, dtype=BF, device="cuda")):
        got = attend(c, q, [50, 30], [1024, 900], 64, 4, with_idx=True)
        compare(got, expect(q, ks, vs, c, [50, 30], [1024, 900], 64, 4))
        assert (got[2][:, :, :3] == torch.arange(3, device="cuda")).all()


def test_scores_closer_than_fp32_holds():
    """Pooled keys that differ by one unit of fp32 in one place: only 64-bit scores tell them apart."""
    c, ks, vs = filled([64 * 40 + 5], 1, 128, 64, 64, seed=5)
    base = torch.randn(128, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    slots = c.table[0, :40].long()
    kb = base.repeat(40, 1)
    for i in range(40):
        kb[i, (37 * i) % 128] += float(torch.finfo(torch.float32).eps) * (i % 7 - 3) * base[(37 * i) % 128].abs()
    c.kbar[slots, 0] = kb
    q = normal(7, 5, 16, 128)
    got = attend(c, q, [5], [64 * 40 + 5], 64, 5, with_idx=True)
    compare(got, expect(q, ks, vs, c, [5], [64 * 40 + 5], 64, 5))


def test_odd_values_in_pooled_keys():
    """NaN scores count as -inf; infinite and huge ones are ordered like any other."""
    lens = [64 * 12 + 9]
    c, ks, vs = filled(lens, 1, 64, 16, 64, seed=6)
    slots = c.table[0, torch.arange(12, device="cuda") * 4 + 3].long()
    c.kbar[slots[2], 0, 5] = float("nan")
    c.kbar[slots[4], 0, :] = 1e30
    c.kbar[slots[5], 0, :] = 3e38
    c.kbar[slots[7], 0, 0] = float("inf")
    c.kbar[slots[9], 0, :] = 1e-42
    q = normal(8, 9, 4, 64)
    q[3] = q[3].abs() + 0.1
    q[5] = -q[5].abs() - 0.1
    got = attend(c, q, [9], lens, 64, 4, with_idx=True)
    assert ops.get_status() == ops.MOBA_OK
    compare(got, expect(q, ks, vs, c, [9], lens, 64, 4))


@pytest.mark.parametrize("n", [3, 400])
@pytest.mark.parametrize("d,noise,topk", [(64, 1e-2, 6), (128, 1e-4, 3), (128, 1e-6, 9)])
def test_scores_that_differ_little(n, d, noise, topk):
    """Pooled keys around a common one: the scores' differences reach down into fp32's last bits."""
    length = 64 * 70 + 11
    c, ks, vs = filled([length], 2, d, 64, 64, seed=25)
    g = torch.Generator("cuda").manual_seed(26)
    common = 3 * torch.randn(2, d, generator=g, device="cuda")
    c.kbar[c.table[0, :70].long()] = common * (1 + noise * torch.randn(70, 2, d, generator=g, device="cuda"))
    q = normal(27, n, 8, d)
    got = attend(c, q, [n], [length], 64, topk, with_idx=True)
    assert ops.get_status() == ops.MOBA_OK
    compare(got, expect(q, ks, vs, c, [n], [length], 64, topk))


@pytest.mark.parametrize("n", [4, 300])
@pytest.mark.parametrize("qexp,kexp", [(-80, 0), (0, -80), (-40, -62)])
def test_scores_whose_squares_vanish_in_fp32(n, qexp, kexp):
    length = 64 * 48 + 7
    c, ks, vs = filled([length], 2, 64, 64, 64, seed=21)
    slots = c.table[0, :48].long()
    c.kbar[slots] *= 2.0 ** kexp
    q = normal(22, n, 8, 64) * 2.0 ** qexp
    got = attend(c, q, [n], [length], 64, 4, with_idx=True)
    assert ops.get_status() == ops.MOBA_OK
    compare(got, expect(q, ks, vs, c, [n], [length], 64, 4))


@pytest.mark.parametrize("n", [1, 80])
@pytest.mark.parametrize("topk", [3, 100])
def test_a_block_of_scores_of_minus_infinity(n, topk):
    """A block whose keys are out of range, for rows that score -inf with all of them, has no weight."""
    lens = [64 * 6 + 30]
    c, ks, vs = filled(lens, 1, 64, 16, 64, seed=23)
    q = normal(24, n, 4, 64)
    q[..., 0] = q[..., 0].abs() + 0.1
    ks[0][64:128, :, 0] = -float("inf")
    pages = c.table[0, 4:8].long()
    c.k[pages, :, :, 0] = -float("inf")
    blocks = torch.arange(6, device="cuda")
    slots = c.table[0, blocks * 4 + 3].long()
    c.kbar[slots[1]] = 100.0 * q.double().mean((0, 1)).float()  # chosen by many rows all the same
    got = attend(c, q, [n], lens, 64, topk, with_idx=True)
    assert ops.get_status() == ops.MOBA_OK
    want = expect(q, ks, vs, c, [n], lens, 64, topk)
    assert all(x.isfinite().all() for x in want) and (topk == 100 or (got[2] == 1).any())
    compare(got, want)


def test_padding_rows_and_unwritten_memory_stay_out():
    """Pages hold NaN wherever nothing was appended; rows behind the last
    sequence keep what they hold."""
    nq, lens = [40, 1], [100, 77]
    c, ks, vs = filled(lens, 2, 64, 32, 64, seed=9)
    q = torch.cat([normal(1, 41, 4, 64), torch.full((20, 4, 64), float("nan"), dtype=BF, device="cuda")])
    out, lse = torch.full_like(q, 7.0), torch.full((61, 4), 7.0, device="cuda")
    idx = torch.full((61, 4, 2), 7, dtype=torch.int32, device="cuda")
    attend(c, q, nq, lens, 64, 2, out=out, lse=lse, idx=idx)
    assert (out[41:] == 7).all() and (lse[41:] == 7).all() and (idx[41:] == 7).all()
    compare((out[:41], lse[:41], idx[:41]), expect(q[:41], ks, vs, c, nq, lens, 64, 2))


@pytest.mark.parametrize("topk", [2, 40])
def test_bad_sequences_are_refused_on_the_device(topk):
    nq, lens = [3, 2, 1, 4], [200, 300, 150, 64]
    c, ks, vs = filled(lens, 2, 64, 16, 64, seed=10)
    q = normal(2, 10, 4, 64)
    want = expect(q, ks, vs, c, nq, lens, 64, topk)
    good = torch.ones(10, dtype=torch.bool, device="cuda")
    bad_lens = list(lens)
    bad_lens[1] = 1  # below its new tokens
    bad_lens[2] = c.mp * 16 + 1
    good[3:6] = False
    out, lse, idx = attend(c, q, nq, bad_lens, 64, topk, with_idx=True)
    assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    compare((out[good], lse[good], idx[good]), [t[good] for t in want])
    assert (out[~good] == 0).all() and (lse[~good] == -float("inf")).all() and (idx[~good] == -1).all()
    # offsets that decrease or leave the rows
    for cu in ([0, 3, 2, 2, 2], [0, 3, 5, 6, 11], [-1, 3, 5, 6, 10]):
        ops.paged_attn(q, c.k, c.v, c.kbar, c.table, i32(cu), i32(lens), 4, 64, topk)
        assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    # a page outside the pool
    for wrong in (-1, c.P, 2 ** 31 - 1):
        table = c.table.clone()
        table[0, 200 // 16] = wrong  # the page of the newest tokens
        out, lse, _ = ops.paged_attn(q, c.k, c.v, c.kbar, table, i32([0, 3, 5, 6, 10]), i32(lens), 4, 64, topk)
        assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
        assert (out[:3] == 0).all() and (lse[:3] == -float("inf")).all()
        compare((out[3:], lse[3:], None), [t[3:] for t in want])
    if topk == 2:  # the last page of a block, where its pooled key would be
        table = c.table.clone()
        table[1, 3] = c.P + 5
        out, lse, idx = ops.paged_attn(q, c.k, c.v, c.kbar, table, i32([0, 3, 5, 6, 10]), i32(lens), 4, 64, topk,
                                       with_idx=True)
        assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
        assert (out[3:5] == 0).all() and (lse[3:5] == -float("inf")).all() and (idx[3:5] == -1).all()
        compare((out[5:], lse[5:], idx[5:]), [t[5:] for t in want])


def test_workspace_stream_and_graph():
    nq, lens = [1, 20, 1], [1000, 500, 64]
    c, ks, vs = filled(lens, 2, 128, 32, 64, seed=11)
    q = normal(3, 22, 8, 128)
    size = ops.paged_attn_workspace_size(3, 22, 20, 8, 2, 128, 32, c.mp, 64, 3)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")  # needs no initialisation
    want = attend(c, q, nq, lens, 64, 3, with_idx=True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = attend(c, q, nq, lens, 64, 3, with_idx=True, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    with pytest.raises(RuntimeError):
        attend(c, q, nq, lens, 64, 3, workspace=ws[:size - 256])
    # two graphs that share a workspace, replayed one after the other with new inputs
    cu, ln = i32([0, 1, 21, 22]), i32(lens)
    outs = [(torch.empty_like(q), torch.empty(22, 8, device="cuda")) for _ in range(2)]
    graphs = []
    for (o, z), topk in zip(outs, (3, 2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.paged_attn(q, c.k, c.v, c.kbar, c.table, cu, ln, 20, 64, topk, out=o, lse=z, workspace=ws)
        graphs.append(g)
    for seed in (4, 5):
        q.copy_(normal(seed, 22, 8, 128))
        ws.fill_(0xEE)
        for g in graphs + graphs[::-1]:
            g.replay()
        for (o, z), topk in zip(outs, (3, 2)):
            compare((o, z, None), expect(q, ks, vs, c, nq, lens, 64, topk))


def test_offsets_beyond_32_bits():
    """The sequence's pages lie behind 2^32 elements of the pool."""
    hkv, page, d = 8, 128, 128
    P = (1 << 32) // (hkv * page * d) + 40
    k, v = (torch.empty(P, hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
    kbar = torch.empty(P, hkv, d, device="cuda")
    n, block = 700, 128
    c = Cache(1, 768, 1, d, page, block)
    c.k, c.v, c.kbar = k, v, kbar
    c.table = torch.arange(P - 1, P - 7, -1, dtype=torch.int32, device="cuda").view(1, 6).contiguous()
    ks, vs, q = [normal(1, n, hkv, d)], [normal(2, n, hkv, d)], normal(3, 5, 16, d)
    c.append(ks[0], vs[0], [0, n], [n])
    got = attend(c, q, [5], [n], block, 3, with_idx=True)
    assert ops.get_status() == ops.MOBA_OK
    compare(got, expect(q, ks, vs, c, [5], [n], block, 3))


@pytest.mark.parametrize("topk", [1, 3, 40])
def test_bad_sequences_in_long_chunks(topk):
    nq, lens = [200, 90, 150, 400], [300, 1000, 150, 900]
    c, ks, vs = filled(lens, 2, 64, 16, 64, seed=12)
    q = normal(2, 840, 4, 64)
    want = expect(q, ks, vs, c, nq, lens, 64, topk)
    cu = [0, 200, 290, 440, 840]
    good = torch.ones(840, dtype=torch.bool, device="cuda")
    good[200:440] = False
    out, lse, idx = ops.paged_attn(q, c.k, c.v, c.kbar, c.table, i32(cu), i32([300, 89, c.mp * 16 + 1, 900]), 400, 64,
                                   topk, with_idx=True)
    assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    compare((out[good], lse[good], idx[good]), [t[good] for t in want])
    assert (out[~good] == 0).all() and (lse[~good] == -float("inf")).all() and (idx[~good] == -1).all()
    # offsets that decrease, overlap, leave the rows, or give more than max_new
    for wrong in ([0, 400, 0, 400, 0], [0, 200, 290, 440, 841], [-1, 200, 290, 440, 840], [0, 401, 401, 401, 840]):
        ops.paged_attn(q, c.k, c.v, c.kbar, c.table, i32(wrong), i32([900] * 4), 400, 64, topk)
        assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    # a page outside the pool: the newest tokens' page of the last sequence
    table = c.table.clone()
    table[3, 899 // 16] = c.P
    out, lse, _ = ops.paged_attn(q, c.k, c.v, c.kbar, table, i32(cu), i32(lens), 400, 64, topk)
    assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    assert (out[836:] == 0).all() and (lse[836:] == -float("inf")).all()
    compare((out[:440], lse[:440], None), [t[:440] for t in want])
    # the context stays usable
    got = ops.paged_attn(q, c.k, c.v, c.kbar, c.table, i32(cu), i32(lens), 400, 64, topk, with_idx=True)
    assert ops.get_status() == ops.MOBA_OK
    compare(got, want)


@pytest.mark.parametrize("topk", [3, 1000])
@pytest.mark.parametrize("n,hq,hkv,d,page,block", [(1, 8, 8, 128, 64, 512), (1, 16, 8, 64, 16, 64),
                                                   (4, 32, 4, 128, 32, 128), (8, 24, 4, 64, 64, 128)])
def test_steps_over_long_caches(n, hq, hkv, d, page, block, topk):
    """Many key tiles to each of the GPU's SMs."""
    lens = [20000, 15001, 9000, 17, 12345, 19999]
    case([min(n, x) for x in lens], lens, hq, hkv, d, page, block, topk, seed=n + topk, with_idx=topk < 100)
