"""Attention of sequences that share prefixes against the definition in 64 bits, by each
sequence's own pages.  Tolerances as in test_gpu_paged_attn: joining the parts is fp32
arithmetic on fp32 sums, within the 2^-18 of exponentials and sums there."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_attn import expect
from .test_gpu_paged_cache import BF, built, i32, normal  # noqa: F401  (built: a fixture)

pytestmark = pytest.mark.gpu


class Forks:
    """Groups of sequences over one pool: a group is (shared tokens, [(new, own tokens with
    the new ones), ...]).  Pages in a random order, NaN wherever no token is; table rows
    end in -1."""

    def __init__(self, groups, hkv, d, page, seed=0, slack=0):
        assert all(p % page == 0 and n <= m for p, members in groups for n, m in members)
        g = torch.Generator().manual_seed(seed)
        need = sum(p // page + sum(-(-m // page) for _, m in members) for p, members in groups)
        order = torch.randperm(need + 3, generator=g).tolist()
        self.page, self.P = page, need + 3
        self.k = torch.full((self.P, hkv, page, d), float("nan"), dtype=BF, device="cuda")
        self.v = self.k.clone()
        self.kbar = None
        self.nq, self.lens, self.ks, self.vs, rows, self.cu_groups, self.prefixes = [], [], [], [], [], [0], []
        for i, (p, members) in enumerate(groups):
            head = [order.pop() for _ in range(p // page)]
            hk, hv = normal(seed + 11 * i + 1, p, hkv, d), normal(seed + 11 * i + 2, p, hkv, d)
            self._write(head, hk, hv)
            for j, (n, m) in enumerate(members):
                mine = [order.pop() for _ in range(-(-m // page))]
                k, v = normal(seed + 97 * i + 7 * j + 3, m, hkv, d), normal(seed + 97 * i + 7 * j + 4, m, hkv, d)
                self._write(mine, k, v)
                self.nq.append(n)
                self.lens.append(p + m)
                self.ks.append(torch.cat((hk, k)))
                self.vs.append(torch.cat((hv, v)))
                rows.append(head + mine)
            self.cu_groups.append(len(self.nq))
            self.prefixes.append(p)
        width = max(1, max(len(r) for r in rows)) + slack
        self.rows = rows
        self.table = i32([r + [-1] * (width - len(r)) for r in rows])

    def _write(self, pages, k, v):
        for x, pool in ((k, self.k), (v, self.v)):
            for i, p in enumerate(pages):
                part = x[i * self.page:(i + 1) * self.page]
                pool[p, :, :len(part)] = part.transpose(0, 1)

    @property
    def cu(self):
        cu = [0]
        for n in self.nq:
            cu.append(cu[-1] + n)
        return cu

    def call(self, q, **kw):
        a = dict(cu=self.cu, lens=self.lens, max_new=max(max(self.nq), 1), cu_groups=self.cu_groups, prefixes=self.prefixes)
        a.update({n: kw.pop(n) for n in list(kw) if n in a})
        return ops.paged_attn_shared(q, self.k, self.v, self.table, i32(a["cu"]), i32(a["lens"]), a["max_new"],
                                     i32(a["cu_groups"]), i32(a["prefixes"]), **kw)

    def expect(self, q):
        # the definition looks tokens up in ks and vs alone (no block is selected)
        return expect(q, self.ks, self.vs, self, self.nq, self.lens, 1 << 20, 1)


def compare(got, want, rows=slice(None)):
    out, lse, _, tol, ltol = want
    err = (got[0][rows].double() - out[rows]).abs()
    assert (err <= tol[rows]).all(), float((err - tol[rows]).max())
    err = (got[1][rows].double() - lse[rows]).abs()
    assert (err <= ltol[rows]).all(), float((err - ltol[rows]).max())


def case(groups, hq, hkv, d, page, seed=0, status=ops.MOBA_OK, slack=0, **kw):
    f = Forks(groups, hkv, d, page, seed, slack)
    q = normal(seed + 5, sum(f.nq), hq, d)
    got = f.call(q, **kw)
    assert ops.get_status() == status
    compare(got, f.expect(q))
    return f, q, got


HEADS = [(4, 4, 64, 16), (8, 2, 128, 32), (5, 1, 128, 64), (24, 8, 64, 128), (64, 1, 64, 16), (32, 2, 128, 256)]


@pytest.mark.parametrize("hq,hkv,d,page", HEADS)
def test_a_decode_step_of_forks(hq, hkv, d, page):
    case([(1280, [(1, 1 + 37 * i % 300) for i in range(9)])], hq, hkv, d, page)


@pytest.mark.parametrize("hq,hkv,d,page", HEADS)
def test_groups_of_uneven_sizes(hq, hkv, d, page):
    """Empty and single groups, groups that share nothing, new tokens of several at once."""
    groups = [(256, [(1, 1)]), (0, [(3, 70), (1, 1)]), (768, [(2, 100), (0, 0), (5, 5), (1, 260)]), (512, []),
              (1024, [(0, 9), (4, 64)]), (0, []), (256, [(1, 513), (2, 2), (3, 65)])]
    case(groups, hq, hkv, d, page, seed=3, slack=5)


@pytest.mark.parametrize("hq,hkv,d,page", HEADS)
def test_chunks_of_many_rows(hq, hkv, d, page):
    groups = [(512, [(130, 200), (1, 77), (64, 64), (0, 0)]), (0, [(90, 300)]), (1792, [(33, 40), (200, 513)])]
    case(groups, hq, hkv, d, page, seed=4, slack=2)


@pytest.mark.parametrize("seqs", [1, 2, 3, 33, 130, 300])
@pytest.mark.parametrize("prefix", [16, 112, 128, 144, 2032])
def test_prefixes_that_end_inside_a_tile(seqs, prefix):
    case([(prefix, [(1, 1 + i % 5) for i in range(seqs)])], 4, 2, 64, 16, seed=prefix + seqs)


def test_a_long_prefix_over_every_cta():
    case([(40960, [(1, 30), (2, 2), (1, 200)])], 8, 2, 128, 64, seed=6)
    case([(8192, [(2, 2)]), (4096, [(1, 1), (1, 4096)])], 6, 3, 128, 32, seed=7)


@pytest.mark.parametrize("d,page", [(64, 64), (128, 16)])
def test_groups_of_many_rows_beside_groups_of_few(d, page):
    """Units enough that groups of more than 16 rows go to the tensor cores, and few rows do
    not; prefixes that end inside a key tile; a group of more than 256 rows."""
    groups = [(3328 + page, [(1, 1 + i % 40) for i in range(40)]), (1984, [(2, 50)]), (512, [(1, 3)] * 3),
              (2560, [(2, 2 + i) for i in range(35)])]
    case(groups, 32, 8, d, page, seed=17)


def test_many_groups():
    """More groups and sequences than the plan's threads."""
    groups = [(16 * (i % 3), [(1, 1 + i % 4)] * (1 + i % 2)) for i in range(1300)]
    case(groups, 2, 1, 64, 16, seed=8)


def test_sequences_of_no_group_and_no_groups():
    f = Forks([(64, [(1, 30)]), (256, [(2, 5), (1, 1), (1, 90)]), (128, [(1, 1)])], 2, 64, 32, seed=9)
    q = normal(1, sum(f.nq), 6, 64)
    want = f.expect(q)
    for groups, prefixes in (([1, 4], [256]), ([], []), ([0], []), ([2, 4], [256]), ([1, 3], [224]), ([4, 4, 5], [96, 128])):
        got = f.call(q, cu_groups=groups or [0], prefixes=prefixes)
        assert ops.get_status() == ops.MOBA_OK
        compare(got, want)


def test_groups_that_are_wrong_share_nothing():
    """They are reported, and the sequences are attended by their own pages."""
    f = Forks([(256, [(2, 5), (1, 1), (1, 90)]), (64, [(1, 30), (3, 200)])], 2, 64, 32, seed=10, slack=3)
    q = normal(1, sum(f.nq), 6, 64)
    want = f.expect(q)
    many = 32 * f.table.shape[1]
    for groups, prefixes in (([0, 3, 5], [255, 64]), ([0, 3, 5], [256, -32]), ([0, 3, 5], [288, 64]),
                             ([0, 3, 5], [256, many + 32]), ([0, 3, 5], [256, 2 ** 31 - 32]), ([0, 6, 5], [256, 64]),
                             ([-1, 3, 5], [256, 64]), ([0, 3, 9], [256, 64]), ([3, 0, 5], [256, 64]),
                             ([5, 3, 0], [256, 64]), ([0, 2 ** 31 - 1, -2 ** 31], [256, 64])):
        got = f.call(q, cu_groups=groups, prefixes=prefixes)
        assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG, (groups, prefixes)
        compare(got, want)


@pytest.mark.parametrize("scale", [1, 50])
def test_refused_members_and_padding(scale):
    """A refused sequence's rows are cleared, its group shares nothing, the others stand; rows
    behind the last sequence are left as they were."""
    groups = [(256, [(2 * scale, 150), (3 * scale, 200), (1, 1)]), (128, [(1, 30), (4, 9)])]
    f = Forks(groups, 2, 128, 32, seed=11, slack=1)
    total = sum(f.nq)
    q = normal(1, total + 20, 8, 128)
    want = f.expect(q[:total])
    lens = list(f.lens)
    lens[1] = 3 * scale - 1  # fewer than its new tokens
    out, lse = torch.full_like(q, 7.0), torch.full((total + 20, 8), 7.0, device="cuda")
    f.call(q, lens=lens, out=out, lse=lse)
    assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    gone = slice(f.cu[1], f.cu[2])
    assert (out[gone] == 0).all() and (lse[gone] == -float("inf")).all()
    assert (out[total:] == 7).all() and (lse[total:] == 7).all()
    for rows in (slice(0, f.cu[1]), slice(f.cu[2], total)):
        compare((out, lse), want, rows)
    # offsets that lead out of the tensors, or nowhere
    for cu in ([-5, 2, 9, 10, 11, 15], [9, 8, 7, 6, 5, 4], [0, total + 99, 3, 2 ** 31 - 1, -2 ** 31, 7]):
        f.call(q, cu=cu, out=out, lse=lse)
        assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
        assert (out[total + 15:] == 7).all() or cu[1] > total


def test_pages_outside_the_pool():
    """Zeros and -inf for the rows that meet one (rows of its group may be among them)."""
    f = Forks([(256, [(1, 5), (1, 1), (1, 90)]), (64, [(1, 30), (3, 200)])], 2, 64, 32, seed=12)
    q = normal(1, sum(f.nq), 6, 64)
    want = f.expect(q)
    f.table[2, 9] = f.P  # the third sequence's own
    got = f.call(q)
    assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    assert (got[0][2] == 0).all() and (got[1][2] == -float("inf")).all()
    for rows in (slice(0, 2), slice(3, None)):
        compare(got, want, rows)
    f.table[2, 9] = f.rows[2][9]
    f.table[3:, 1] = -1  # of the second group's prefix
    got = f.call(q)
    assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    assert (got[0][3:] == 0).all() and (got[1][3:] == -float("inf")).all()
    compare(got, want, slice(0, 3))


def test_equal_calls_give_equal_bits_and_workspaces_hold():
    f = Forks([(2048, [(1, 1 + 50 * i) for i in range(20)])], 2, 128, 64, seed=13)
    q = normal(1, 20, 16, 128)
    want = f.call(q)
    need = ops.paged_attn_shared_workspace_size(20, 1, 20, 1, 16, 2, 128, 64, f.table.shape[1])
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        got = f.call(q, workspace=ws[:need])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (ws[need:] == 255).all() and ops.get_status() == ops.MOBA_OK
    with pytest.raises(RuntimeError):
        f.call(q, workspace=ws[:need - 256])


def test_a_side_stream_and_a_graph():
    """Captured with tables and groups that are rewritten in place."""
    f = Forks([(1024, [(1, 1 + 9 * i) for i in range(12)])], 2, 64, 16, seed=14)
    q = normal(1, 12, 8, 64)
    want = f.expect(q)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = f.call(q, stream=st)
    torch.cuda.synchronize()
    compare(got, want)
    cu, lens, groups, prefixes = i32(f.cu), i32(f.lens), i32([0, 12, 12]), i32([1024, 0])
    out, lse = torch.empty_like(q), torch.empty(12, 8, device="cuda")
    ws = torch.empty(ops.paged_attn_shared_workspace_size(12, 2, 12, 1, 8, 2, 64, 16, f.table.shape[1]),
                     dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.paged_attn_shared(q, f.k, f.v, f.table, cu, lens, 1, groups, prefixes, out=out, lse=lse, workspace=ws)
    for split, ps in (([0, 12, 12], [1024, 0]), ([0, 5, 12], [512, 1024]), ([3, 4, 11], [16, 1008]), ([0, 0, 0], [0, 0])):
        groups.copy_(i32(split))
        prefixes.copy_(i32(ps))
        out.zero_()
        g.replay()
        compare((out, lse), want)
    assert ops.get_status() == ops.MOBA_OK


def test_keys_of_every_size():
    """Logits far apart: the prefix or the own keys carry the whole weight."""
    for far, near in ((30.0, 0.01), (0.01, 30.0)):
        f = Forks([(512, [(1, 100), (2, 2), (1, 65)])], 1, 128, 32, seed=15)
        for b, (pages, length) in enumerate(zip(f.rows, f.lens)):
            f.ks[b][:512] *= far
            f.ks[b][512:] *= near
            for i, p in enumerate(pages):
                if i >= 512 // 32 or b == 0:
                    part = f.ks[b][i * 32:min((i + 1) * 32, length)]
                    f.k[p, :, :len(part)] = part.transpose(0, 1)
        q = normal(1, 4, 8, 128)
        got = f.call(q)
        assert ops.get_status() == ops.MOBA_OK
        compare(got, f.expect(q))


def test_no_new_tokens():
    f = Forks([(64, [(0, 5), (0, 9)])], 2, 64, 16, seed=16)
    out, lse = f.call(normal(1, 0, 4, 64))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    q = normal(1, 3, 4, 64)  # (rows of padding only)
    out, lse = torch.full_like(q, 7.0), torch.full((3, 4), 7.0, device="cuda")
    f.call(q, out=out, lse=lse)
    assert (out == 7).all() and (lse == 7).all() and ops.get_status() == ops.MOBA_OK


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("new,prefix", [((1, 1, 2), 512), ((2, 3, 13), 40960), ((70, 5, 40), 512)])
def test_keys_that_are_not_finite_show(value, new, prefix):
    """A NaN, or infinities that meet, in a key reach the rows that see it (a decode step, a group for
    the tensor cores, chunks; in the prefix and in the own keys); another group stands."""
    f = Forks([(prefix, [(n, 90) for n in new]), (512, [(1, 100), (2, 20)])], 2, 64, 32, seed=17)
    q = normal(1, sum(f.nq), 16, 64)
    q[..., 5] = q[..., 5].abs() + 0.1
    want = f.call(q)
    mine = sum(new)
    f.k[f.rows[0][3], 1, 4, 5] = value  # kv head 1: query heads 8 to 15
    out, lse = f.call(q)
    assert ops.get_status() == ops.MOBA_OK
    assert out[:mine, 8:].isnan().all() and lse[:mine, 8:].isnan().all()
    for a, b in ((out, want[0]), (lse, want[1])):
        assert torch.equal(a[:, :8], b[:, :8]) and torch.equal(a[mine:], b[mine:])
    f.k[f.rows[0][3], 1, 4, 5] = 0.0
    f.k[f.rows[1][prefix // 32], 0, 1, 5] = value  # a key of the second sequence alone
    out, lse = f.call(q)
    lo, hi = f.cu[1], f.cu[2]
    assert out[lo:hi, :8].isnan().all() and lse[lo:hi, :8].isnan().all()
    assert torch.equal(out[mine:], want[0][mine:]) and torch.equal(lse[mine:], want[1][mine:])


@pytest.mark.parametrize("count", [4, 1100])
@pytest.mark.parametrize("scale", [1, 40])
def test_a_group_whose_tables_have_changed(scale, count):
    """A row of the page table names another sequence's pages than when the groups were made:
    by their own pages, and reported."""
    f = Forks([(96, [(scale, 50 + i % 7) for i in range(count if scale == 1 else 4)]), (96, [(scale, 60), (1, 70)])],
              1, 64, 32, seed=18)
    q = normal(1, sum(f.nq), 4, 64)
    want = f.expect(q)
    n = len(f.nq)
    got = f.call(q, cu_groups=[0, n - 1, n], prefixes=[96, 96])  # one of the second group's among the first's
    assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    compare(got, want)
    got = f.call(q, cu_groups=[0, n], prefixes=[96])
    assert ops.get_status() == ops.MOBA_ERR_INVALID_ARG
    compare(got, want)
