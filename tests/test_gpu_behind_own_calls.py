"""Calls right behind calls of the framework whose results they read: such a call's first
kernel is there while the kernel that writes its operands still runs.  The same bits as with
copies of the operands and nothing running beside."""
import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_cache import BF, Cache, built, i32, normal  # noqa: F401  (built: a fixture)
from .test_gpu_paged_rope import same
from .test_gpu_paged_shared import Forks, compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
def test_weights_that_the_call_before_wrote(captured):
    """The norms' and the append's weights are the weights' gradient of the call before."""
    T, h, d, steps = 300, 6, 64, 40
    x = normal(1, T, 3 * h, d)
    w = 1 + 0.3 * normal(2, d).float()
    pos, freqs = torch.arange(T, dtype=torch.int32, device="cuda"), ops.rope_frequencies(d)
    dy = [normal(3 + i, T, h, d) for i in range(steps)]
    c = Cache(1, 512, h, d, 32, 64)
    tables = c.k, c.v, c.kbar, c.table, i32([0, T]), i32([T]), T, c.block, freqs
    dw, dx = torch.empty(d, device="cuda"), torch.empty(T, h, d, dtype=BF, device="cuda")
    want = []
    ws = torch.empty(ops.qk_norm_rope_bwd_workspace_size(T, h, 0, d), dtype=torch.uint8, device="cuda")

    def step(i):
        ops.qk_norm_rope_bwd(dy[i], None, x[:, :h], None, w, None, pos, freqs, dq=dx, dq_weight=dw, workspace=ws)
        y, _ = ops.qk_norm_rope(dx, None, dw, None, pos, freqs)
        ops.qk_norm_rope_bwd(dy[-1 - i], None, x[:, :h], None, w, None, pos, freqs, dq=dx, dq_weight=dw, workspace=ws)
        z = ops.paged_append_rope(dx, x[:, h:2 * h], x[:, 2 * h:], *tables, q_weight=dw, k_weight=dw)
        return y, z, c.k.clone(), c.kbar.clone()

    for i in range(steps):
        made = []
        for g in (dy[i], dy[-1 - i]):
            r = ops.qk_norm_rope_bwd(g, None, x[:, :h], None, w, None, pos, freqs)
            torch.cuda.synchronize()
            made.append((r[0].clone(), r[2].clone()))
            torch.cuda.synchronize()
        (x1, w1), (x2, w2) = made
        y = ops.qk_norm_rope(x1, None, w1, None, pos, freqs)[0]
        z = ops.paged_append_rope(x2, x[:, h:2 * h], x[:, 2 * h:], *tables, q_weight=w2, k_weight=w2)
        torch.cuda.synchronize()
        want.append((y, z, c.k.clone(), c.kbar.clone()))
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = [step(i) for i in range(steps)]
        for _ in range(2):
            g.replay()
    else:
        out = [step(i) for i in range(steps)]
    for a, b in zip(out, want):
        assert all(same(x, y) for x, y in zip(a, b))
    assert ops.get_status() == ops.MOBA_OK


@pytest.mark.parametrize("prefix", [512, 8192])
def test_shared_prefixes_behind_copies_of_their_operands(prefix):
    """A captured call whose operands are copied in right before it, replayed over workspaces of
    any contents (prefixes that are streamed, and ones for the tensor cores)."""
    f = Forks([(prefix, [(1, 1 + i % 40) for i in range(40)]), (64, [(1, 70), (1, 1)])], 8, 64, 16, seed=3)
    n = len(f.nq)
    live = [normal(1, n, 32, 64), f.table.clone(), i32(f.lens), i32([0, 40, 42]), i32([prefix, 64])]
    staged = [x.clone() for x in live]
    cu, out, lse = i32(f.cu), torch.empty_like(live[0]), torch.empty(n, 32, device="cuda")
    ws = torch.empty(ops.paged_attn_shared_workspace_size(n, 2, n, 1, 32, 8, 64, 16, f.table.shape[1]), dtype=torch.uint8, device="cuda")

    def call():
        for x, y in zip(live, staged):
            x.copy_(y)
        ops.paged_attn_shared(live[0], f.k, f.v, live[1], cu, live[2], 1, live[3], live[4], out=out, lse=lse, workspace=ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(12):
        staged[0].copy_(normal(10 + i, n, 32, 64))
        if i % 3 == 1:  # other pages for everybody: as if the sequences had changed places
            staged[1].copy_(f.table)
            staged[2].copy_(i32(f.lens))
        elif i % 3 == 2:
            staged[1][:40] = f.table[:40].flip(0)
            staged[2][:40] = i32(f.lens[:40][::-1])
        if i % 4 == 0:
            ws.fill_(i)
        want = ops.paged_attn_shared(staged[0], f.k, f.v, staged[1], cu, staged[2], 1, staged[3], staged[4])
        torch.cuda.synchronize()
        out.fill_(7.0)
        g.replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        call()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    compare(want, f.expect(staged[0]), slice(40, None))
    assert ops.get_status() == ops.MOBA_OK


@pytest.mark.parametrize("seqs", [3, 300])
def test_pooling_behind_copies_of_the_tables(seqs):
    """Steps that complete blocks, with page tables and lengths copied in right before them."""
    hkv, d, page, block = 4, 64, 16, 64
    freqs = ops.rope_frequencies(d)
    one, two = (Cache(seqs, 192, hkv, d, page, block, seed=5) for _ in range(2))
    first = normal(1, seqs * 126, 3 * hkv, d)
    cu = i32([126 * i for i in range(seqs + 1)])
    for c in (one, two):
        ops.paged_append_rope(first[:, :hkv], first[:, hkv:2 * hkv], first[:, 2 * hkv:], c.k, c.v, c.kbar, c.table, cu,
                              i32([126] * seqs), 126, block, freqs)
    step = i32(list(range(seqs + 1)))
    table, lens = one.table.clone(), i32([126] * seqs)
    x = normal(2, seqs, 3 * hkv, d)
    staged = [one.table.clone(), i32([126] * seqs), x.clone()]
    args = x[:, :hkv], x[:, hkv:2 * hkv], x[:, 2 * hkv:], one.k, one.v, one.kbar, table, step, lens, 1, block, freqs
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for a, b in zip((table, lens, x), staged):
            a.copy_(b)
        ops.paged_append_rope(*args)
    for n in range(127, 131):  # the block completed by the second of them
        order = torch.randperm(seqs, generator=torch.Generator().manual_seed(n)).cuda()
        staged[0].copy_(one.table[order])
        staged[1].fill_(n)
        staged[2].copy_(normal(n, seqs, 3 * hkv, d))
        torch.cuda.synchronize()
        g.replay()
        y = staged[2]
        torch.cuda.synchronize()
        ops.paged_append_rope(y[:, :hkv], y[:, hkv:2 * hkv], y[:, 2 * hkv:], two.k, two.v, two.kbar, staged[0], step, staged[1], 1,
                              block, freqs)
        torch.cuda.synchronize()
        for a, b in ((one.k, two.k), (one.v, two.v), (one.kbar, two.kbar)):
            assert same(a, b)
    assert not one.kbar[one.table[:, 7].long()].isnan().any() and ops.get_status() == ops.MOBA_OK


def test_two_caches_on_two_streams():
    """More calls on each than there are words for their tokens, side by side."""
    hkv, d, page, block, seqs, steps = 2, 64, 16, 64, 5, 1400
    freqs = ops.rope_frequencies(d)
    step = i32(list(range(seqs + 1)))
    lens = [i32([n + 1] * seqs) for n in range(steps)]
    x = normal(7, steps, seqs, 3 * hkv, d)

    def one(c, n):
        y = x[n]
        ops.paged_append_rope(y[:, :hkv], y[:, hkv:2 * hkv], y[:, 2 * hkv:], c.k, c.v, c.kbar, c.table, step, lens[n], 1, block,
                              freqs)

    caches = [Cache(seqs, steps, hkv, d, page, block, seed=9) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for n in range(steps):
        for c, st in zip(caches, streams):
            with torch.cuda.stream(st):
                one(c, n)
    torch.cuda.synchronize()
    for n in range(steps):
        one(caches[2], n)
    for c in caches[:2]:
        assert same(c.k, caches[2].k) and same(c.v, caches[2].v) and same(c.kbar, caches[2].kbar)
    assert ops.get_status() == ops.MOBA_OK


def test_two_graphs_on_one_workspace():
    """Replayed in turn: each makes its own plan there."""
    a = Forks([(8192, [(1, 1 + i) for i in range(40)]), (0, [(1, 50)])], 8, 64, 16, seed=4)
    b = Forks([(256, [(1, 9)] * 3), (4096, [(2, 20 + i) for i in range(24)])], 8, 64, 16, seed=5)
    need = max(ops.paged_attn_shared_workspace_size(len(f.nq), 2, sum(f.nq), max(f.nq), 32, 8, 64, 16, f.table.shape[1]) for f in (a, b))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    calls = []
    for f in (a, b):
        n = sum(f.nq)
        q, out, lse = normal(6, n, 32, 64), torch.empty(n, 32, 64, dtype=BF, device="cuda"), torch.empty(n, 32, device="cuda")
        args = q, f.k, f.v, f.table, i32(f.cu), i32(f.lens), max(f.nq), i32(f.cu_groups), i32(f.prefixes)
        want = ops.paged_attn_shared(*args)
        compare(want, f.expect(q))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.paged_attn_shared(*args, out=out, lse=lse, workspace=ws)
        calls.append((g, q, out, lse, want, args))
    for i in range(20):
        g, q, out, lse, want, _ = calls[i * 7 % 3 % 2]
        out.fill_(7.0)
        g.replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert ops.get_status() == ops.MOBA_OK
