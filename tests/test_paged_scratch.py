"""How the paged kernels read scratch that a kernel before them in the same call
writes.  Such a kernel may still run when its reader starts (programmatic dependent
launch), so the memory is not constant for the reader's life, which the read-only
data path (ld.global.nc: ``__ldg``, or a const ``__restrict__`` parameter) demands."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_sparse_moba_gb300", "csrc")


def code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def scratch_fields():
    """The pointers of Attn behind its "scratch" line."""
    with open(os.path.join(CSRC, "moba_paged_attn.cuh")) as f:
        text = f.read().split("struct Attn {")[1].split("\n};")[0].split("// scratch")[1]
    return set(re.findall(r"\*(\w+)", re.sub(r"//[^\n]*", "", text)))


def arguments(text, name):
    """The argument texts of every call of `name`."""
    for m in re.finditer(r"\b%s(?:<\w+>)?\(" % name, text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        yield text[m.end():at - 1]


def test_the_fields_are_found():
    assert {"tiles", "ublk", "umask", "own_off", "list", "tok", "sel", "part_h", "part_s", "counts"} <= scratch_fields()


def test_scratch_of_the_call_is_not_read_as_constant_data():
    fields, wrong = scratch_fields(), []
    for path in sorted(glob.glob(os.path.join(CSRC, "moba_paged*.cu*"))):
        text = code(path)
        for call in ("__ldg", "upper_index"):  # (upper_index reads its table with __ldg)
            for arg in arguments(text, call):
                wrong += [(os.path.basename(path), call, arg) for f in fields if re.search(r"\ba\.%s\b" % f, arg)]
        # a __restrict__ parameter may be read as constant data too
        for kernel in re.findall(r"__global__[^{;]*\)", text):
            assert "__restrict__" not in kernel, kernel
    assert not wrong, wrong
