"""Kernels that are brought in while the one before them on the stream drains (their source,
read as text): what they may rely on there is not something that a run shows."""
import os
import re

import pytest

from long_context_sparse_moba_gb300 import build


def source(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, name):
    """A function's body, its braces matched."""
    at = re.search(r"\b%s\([^;{]*\)(?: const)? \{" % re.escape(name), text)
    assert at, name
    depth, i = 1, at.end()
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[at.end():i - 1]


# first kernels of their calls: file, kernel, and what they call that reads operands
FIRST = [("moba_qk_norm.cu", "fwd_kernel", ["load_turns", "weight"]), ("moba_qk_norm.cu", "bwd_kernel", ["load_turns", "weight"]),
         ("moba_paged_rope.cu", "write_kernel", ["load_turns", "weight", "seq_now", "seq_of_row"]),
         ("moba_paged_shared.cu", "plan_spans_kernel", ["clear_refused"])]
HEADERS = ["moba_rope.cuh", "moba_paged.cuh", "moba_paged_attn.cuh"]


@pytest.mark.parametrize("file,kernel,calls", FIRST)
def test_first_kernels_take_nothing_for_constant(file, kernel, calls):
    """What wrote their operands may run while they are there: they wait before they read, let the
    next kernel in behind that, and read by plain loads (constant ones may be moved up)."""
    text = body(source(file), kernel)
    assert 0 <= text.find("after_previous()") < text.find("let_next()")
    headers = "".join(source(h) for h in HEADERS)
    for part in [text] + [body(headers, c) for c in calls]:
        assert "__ldg" not in part
    assert not re.search(r"\bc\.seq\(", text)  # (which reads constants)


def test_pooling_begins_by_the_writers_token_or_waits():
    """The kernel before it is ordered behind what wrote tables and older keys; this one is only by
    the token which that one releases behind its wait, or by waiting for its end."""
    write, pool = body(source("moba_paged_rope.cu"), "write_kernel"), body(source("moba_paged.cu"), "pool_kernel")
    assert write.find("after_previous()") < write.find("st_release(a.ready") < write.find("let_next()")
    begin = pool.find("ld_acquire(a.ready)")
    assert 0 < begin < pool.find("__syncthreads()") < pool.find("if (waited) after_previous()") < pool.find("seq_now")
    assert "__ldg" not in pool and "a.c.seq(" not in pool and "tile_of" not in pool
    assert "__ldg" not in body(source("moba_paged.cu"), "mean64")
    assert pool.rfind("if (!waited) after_previous();") < pool.find("*a.ready = 0")


def test_streaming_begins_by_the_plans_token_or_waits():
    """The kernel between it and the plan lets it in without ordering any memory."""
    text = source("moba_paged_shared.cu")
    plan, stream, merge = (body(text, n) for n in ("plan_spans_kernel", "stream_kernel", "merge_spans_kernel"))
    at = plan.find("st_release")
    assert plan.rfind("__syncthreads()") < at and plan.rfind("__syncthreads()") > plan.rfind("*a.head = h")
    begin = stream.find("ld_acquire")
    assert 0 < begin < stream.find("__syncthreads()") < stream.find("else after_previous()") < stream.find("a.head->spans")
    assert stream.rstrip().endswith("if (early) after_previous();")  # it ends behind the kernel before it
    assert "__ldg" not in stream and "__ldg" not in merge
    assert merge.find("after_previous()") < merge.find("a.head->ready = 0") < merge.find("return")
