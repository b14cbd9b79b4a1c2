"""The binding's calls in one step: the same bits as the calls step by step (a stream that is named
takes those), the caller's tensors, and what it leaves to them."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from long_context_sparse_moba_gb300 import ops

from .test_gpu_paged_cache import BF, built, i32, normal  # noqa: F401  (built: a fixture)
from .test_gpu_paged_shared import Forks

pytestmark = pytest.mark.gpu


def equal(a, b):
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    return len(a) == len(b) and all(x is y is None or (x.dtype is y.dtype and x.device == y.device and x.is_contiguous() and
                                                       torch.equal(x, y)) for x, y in zip(a, b))


def norm_case(T=5, hq=4, hk=2, d=64, wt=torch.float32, seed=1):
    x = normal(seed, T, hq + 2 * max(hk, 1), d)
    q, k = x[:, :hq], x[:, hq:hq + hk] if hk else None
    w = [(1 + 0.3 * normal(seed + i, d).float()).to(wt) for i in (1, 2)]
    return [q, k, w[0], w[1] if hk else None, i32([7 * i - 3 for i in range(T)]), ops.rope_frequencies(d)]


def append_case(page=16, d=64, bar=True):
    cu, lens = [0, 3, 3, 4], [40, 16, 64]
    k, v = (torch.zeros(20, 2, page, d, dtype=BF, device="cuda") for _ in range(2))
    kbar = torch.zeros(20, 2, d, device="cuda") if bar else None
    x = normal(3, 4, 8, d)
    table = i32([[3, 1, 7, -1, -1], [2, -1, -1, -1, -1], [9, 8, 4, 10, 15]])
    return [x[:, :4], x[:, 4:6], x[:, 6:], k, v, kbar, table, i32(cu), i32(lens), 3, 64, ops.rope_frequencies(d)]


def shared_case():
    f = Forks([(64, [(1, 9), (2, 20)]), (0, [(1, 30)])], 2, 64, 16)
    q = normal(5, 4, 8, 64)
    return [q, f.k, f.v, f.table, i32(f.cu), i32(f.lens), 2, i32(f.cu_groups), i32(f.prefixes)]


@pytest.mark.parametrize("T,hq,hk,d,wt", [(1, 1, 0, 64, BF), (5, 4, 2, 64, torch.float32), (300, 9, 3, 128, BF)])
def test_norms(T, hq, hk, d, wt):
    a = norm_case(T, hq, hk, d, wt)
    kw = dict(eps=1e-5, interleaved=True, magnitude=1.25)
    assert ops._native().qk_norm_rope(*a, 1e-5, True, 1.25, None, None) is not None
    st = torch.cuda.current_stream()
    want = ops.qk_norm_rope(*a, **kw, stream=st)
    assert equal(ops.qk_norm_rope(*a, **kw), want)
    qo = torch.empty(T, hq + 1, d, dtype=BF, device="cuda")[:, :hq]
    ko = torch.empty(T, hk, d, dtype=BF, device="cuda") if hk else None
    got = ops.qk_norm_rope(*a, **kw, q_out=qo, k_out=ko)
    assert got[0] is qo and got[1] is ko and torch.equal(qo, want[0])
    g = normal(8, T, hq, d), normal(9, T, hk, d) if hk else None
    assert ops._native().qk_norm_rope_bwd(*g, *a, 1e-5, True, 1.25, None, None, None, None, None) is not None
    want = ops.qk_norm_rope_bwd(*g, *a, **kw, stream=st)
    assert equal(ops.qk_norm_rope_bwd(*g, *a, **kw), want)
    ws = torch.empty(ops.qk_norm_rope_bwd_workspace_size(T, hq, hk, d), dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(x) if x is not None else None for x in want]
    got = ops.qk_norm_rope_bwd(*g, *a, **kw, dq=out[0], dk=out[1], dq_weight=out[2], dk_weight=out[3], workspace=ws)
    assert all(x is y for x, y in zip(got, out)) and equal(got, want)


@pytest.mark.parametrize("bar,norms,positions", [(True, True, False), (False, False, True), (True, False, False)])
def test_appending(bar, norms, positions):
    w = [normal(i, 64) for i in (1, 2)] if norms else [None, None]
    pos = i32([5, 6, 7, 8]) if positions else None
    results = []
    for native in (True, False):
        a = append_case(bar=bar)
        kw = dict(positions=pos, q_weight=w[0], k_weight=w[1])
        qo = torch.full((4, 4, 64), 7.0, dtype=BF, device="cuda")
        if native:
            assert ops._native().paged_append_rope(*append_case(bar=bar), pos, *w, 1e-6, False, 1.0, None) is not None
            assert ops.paged_append_rope(*a, **kw, q_out=qo) is qo
        else:
            ops.paged_append_rope(*a, **kw, q_out=qo, stream=torch.cuda.current_stream())
        results.append([qo, *a[3:6]])
    assert all(x is y is None or torch.equal(x, y) for x, y in zip(*results)) and ops.get_status() == ops.MOBA_OK


def test_shared_prefixes():
    a = shared_case()
    assert ops._native().paged_attn_shared(*a, None, None, None) is not None
    want = ops.paged_attn_shared(*a, stream=torch.cuda.current_stream())
    assert equal(ops.paged_attn_shared(*a), want)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(ops.paged_attn_shared_workspace_size(3, 2, 4, 2, 8, 2, 64, 16, a[3].shape[1]), dtype=torch.uint8,
                     device="cuda")
    got = ops.paged_attn_shared(*a, out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse and equal(got, want)


def test_what_it_leaves_to_the_other_steps():
    n = ops._native()
    one = norm_case()
    usual = [*one, 1e-6, False, 1.0, None, None]
    f64 = one[0].double()
    for i, x in ((0, one[0].cpu()), (0, f64), (0, one[0].transpose(0, 1)), (0, one[0][0]), (0, one[0][:0]), (1, one[1][:3]),
                 (1, None), (2, None), (2, one[2].to(BF)), (2, one[2][:32]), (3, None), (4, one[4].long()), (4, one[4][:2]),
                 (5, one[5].float()), (6, 1), (6, "x"), (6, float("nan")), (7, 1), (8, 1), (9, f64), (9, one[0][:2]), (10, one[1][:2]),
                 (9, one[1]), (0, "q"), (4, None)):
        a = list(usual)
        a[i] = x
        assert n.qk_norm_rope(*a) is None, (i, x)
    assert n.qk_norm_rope(*usual[:-1]) is None
    a = shared_case()
    for i, x in ((0, a[0][:, :, :32]), (0, a[0][:0]), (1, a[1][0]), (2, a[2][:5]), (3, a[3][:2]), (4, a[4][:2]), (6, 2 ** 40), (6, 0),
                 (6, 2.0), (7, a[7][:2]), (8, a[8][:1]), (9, a[0].float()), (10, a[0]), (11, a[0]), (11, a[0].view(-1).view(torch.uint8))):
        b = [*a, None, None, None]
        b[i] = x
        if i == 11 and x.dtype is torch.uint8:
            b[i] = x[:256]  # too small: refused by the entry point
        assert n.paged_attn_shared(*b) is None, (i, x)
    a = [*append_case(), None, None, None, 1e-6, False, 1.0, None]
    for i, x in ((0, a[0][:2]), (1, a[0]), (2, a[2][:, :1]), (3, a[3].float()), (5, a[5][:3]), (6, a[6].view(-1)), (7, a[7][:3]), (9, 0),
                 (10, 48), (11, a[11][:4]), (12, a[8]), (13, a[5][0, 0].half()), (15, 1), (17, float("inf")), (18, a[1])):
        b = list(a)
        b[i] = x
        assert n.paged_append_rope(*b) is None, (i, x)
    assert ops.get_status() == ops.MOBA_OK


def test_nothing_is_kept():
    a, b, c = norm_case(), append_case(), shared_case()
    g = [normal(8, 5, 4, 64), normal(9, 5, 2, 64)]
    out = [torch.empty(4, 4, 64, dtype=BF, device="cuda")]

    def calls():
        ops.qk_norm_rope(*a)
        ops.qk_norm_rope_bwd(*g, *a)
        ops.paged_append_rope(*b, q_out=out[0])
        ops.paged_attn_shared(*c)
        for bad in (dict(eps=0.0), dict(eps=1)):
            try:
                ops.qk_norm_rope(*a, **bad)
            except RuntimeError:
                pass

    calls()
    torch.cuda.synchronize()
    held = [x for x in (*a, *b, *c, *g, *out) if not isinstance(x, int)]
    counts, used = [sys.getrefcount(x) for x in held], torch.cuda.memory_allocated()
    for _ in range(50):
        calls()
    assert counts == [sys.getrefcount(x) for x in held] and used == torch.cuda.memory_allocated()


OUT_OF_MEMORY = """
import torch
from long_context_sparse_moba_gb300 import ops
q = torch.randn(7000, 32, 128, device="cuda").to(torch.bfloat16)  # (57 MB, and as much of results)
w, pos = torch.ones(128, device="cuda"), torch.arange(7000, dtype=torch.int32, device="cuda")
freqs = ops.rope_frequencies(128)
torch.cuda.empty_cache()
torch.cuda.set_per_process_memory_fraction(0.0001)
try:
    ops.qk_norm_rope(q, None, w, None, pos, freqs)
except torch.OutOfMemoryError:
    torch.cuda.set_per_process_memory_fraction(1.0)
    a = ops.qk_norm_rope(q, None, w, None, pos, freqs)[0]
    b = ops.qk_norm_rope(q, None, w, None, pos, freqs, stream=torch.cuda.current_stream())[0]
    print("raised", torch.equal(a, b), ops.get_status())
"""


def test_no_memory_is_an_error_like_any_other():
    """(In a process of its own, whose allocator has nothing kept.)"""
    run = subprocess.run([sys.executable, "-c", OUT_OF_MEMORY], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert run.returncode == 0 and run.stdout.split() == ["raised", "True", str(ops.MOBA_OK)], run.stdout + run.stderr


def test_threads_and_streams():
    """Calls at once by two threads, each on a stream of its own."""
    cases = [norm_case(T=200 + 100 * i, seed=10 + i) for i in range(2)]
    want = [ops.qk_norm_rope(*a) for a in cases]
    shared = shared_case()
    attn = ops.paged_attn_shared(*shared)
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(100):
                got, got2 = ops.qk_norm_rope(*cases[i]), ops.paged_attn_shared(*shared)
                if not equal(got, want[i]) or not equal(got2, attn):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and ops.get_status() == ops.MOBA_OK


def test_new_tensors_are_filled_where_torch_is_told_to():
    a = norm_case()
    assert ops._native().qk_norm_rope(*a, 1e-6, False, 1.0, None, None) is not None
    torch.use_deterministic_algorithms(True)
    try:
        assert ops._native().qk_norm_rope(*a, 1e-6, False, 1.0, None, None) is None
        x = shared_case()
        q = torch.cat((x[0], x[0]))  # (rows behind the last sequence)
        out, lse = ops.paged_attn_shared(q, *x[1:])
        assert out[4:].isnan().all() and lse[4:].isnan().all()
    finally:
        torch.use_deterministic_algorithms(False)


def test_captured_and_replayed():
    a, b, c = norm_case(T=40), append_case(), shared_case()
    g = normal(8, 40, 4, 64), normal(9, 40, 2, 64)
    call = lambda: (*ops.qk_norm_rope(*a), *ops.qk_norm_rope_bwd(*g, *a), ops.paged_append_rope(*b), *ops.paged_attn_shared(*c))
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for seed in (20, 30):
        for i, x in enumerate((a[0], a[1], g[0], g[1], b[0], c[0])):
            x.copy_(normal(seed + i, *x.shape))
        graph.replay()
        assert equal(got, call())
    assert ops.get_status() == ops.MOBA_OK


def test_modes_of_autograd():
    a = norm_case()
    a[0].requires_grad_(True)
    a[2] = torch.nn.Parameter(a[2])
    assert ops._native().qk_norm_rope(*a, 1e-6, False, 1.0, None, None) is not None
    plain = ops.qk_norm_rope(*a)
    assert not any(x.requires_grad or x.is_inference() for x in plain)
    with torch.inference_mode():
        got = ops.qk_norm_rope(*a)
        assert all(x.is_inference() for x in got) and equal(got, plain)


def test_captured_behind_copies_and_a_join():
    """The first kernel of a call behind a copy, a memset, and the join of two streams."""
    a, b, c = norm_case(T=40), append_case(), shared_case()
    g = normal(8, 40, 4, 64), normal(9, 40, 2, 64)
    calls = [lambda: ops.qk_norm_rope(*a), lambda: ops.qk_norm_rope_bwd(*g, *a), lambda: ops.paged_append_rope(*b),
             lambda: ops.paged_attn_shared(*c)]
    inputs = [(a[0], a[1]), g, (b[0], b[1]), (c[0], c[0])]
    for call, (x, y) in zip(calls, inputs):
        sx, sy, zero = x.clone(), y.clone(), torch.ones(1 << 20, device="cuda")
        call()
        torch.cuda.synchronize()
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for _ in range(20):
                    sy.mul_(-1.0)
                if y is not x:
                    y.copy_(sy)
            x.copy_(sx)
            zero.zero_()
            torch.cuda.current_stream().wait_stream(side)
            got = call()
            again = call()
        for i in range(3):
            sx.copy_(normal(60 + i, *x.shape))
            sy.copy_(normal(70 + i, *y.shape))
            graph.replay()
            want = call()
            assert equal(got, want) and equal(again, want)
    assert ops.get_status() == ops.MOBA_OK


def test_behind_kernels_that_write_their_operands():
    """Calls one after the other on a stream, each reading what the one before it wrote."""
    a = norm_case(T=3000, hq=8, hk=8, d=64)
    q, k = a[0].contiguous(), a[1].contiguous()
    step = lambda q, k, **kw: ops.qk_norm_rope(q, k, *a[2:], **kw)
    for _ in range(20):
        x, y = q, k
        for _ in range(10):
            x, y = step(x, y)
            x = x * 1.0
        torch.cuda.synchronize()
        z, w = q, k
        for _ in range(10):
            z, w = step(z, w)
            torch.cuda.synchronize()
        assert torch.equal(x, z) and torch.equal(y, w)
