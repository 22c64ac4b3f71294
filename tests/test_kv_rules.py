"""Rules that the KV-cache sources and their binding keep and that no run on a GPU can show: what the
instruction set leaves undefined works by chance in every test. No GPU is needed."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verification_78_gb300", "csrc")


def source(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_no_kernel_moves_registers_between_roles():
    """setmaxnreg is defined only where all four warps of a warpgroup execute the same one; the kernels'
    roles are single warps, so none of them may use it."""
    for name in sorted(os.listdir(CSRC)):
        assert "setmaxnreg" not in source(name), name


def test_queries_rotated_in_place_are_not_read_as_constants():
    """q_out may be q: the read-only path (__ldg) is defined only for memory that the kernel does not
    write."""
    text = source("spec_kv_append.cu")
    body = text[text.index("void append_queries("):text.index("kv_append_kernel(")]
    reads = re.findall(r"raw\[k\]\[[01]\] = ([^;]*src[^;]*);", body)
    assert len(reads) == 2
    for r in reads:
        assert "__ldg" not in r, r
