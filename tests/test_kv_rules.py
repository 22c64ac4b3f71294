"""Rules that the KV-cache sources and their binding keep and that no run on a GPU can show: what the
instruction set leaves undefined works by chance in every test. No GPU is needed."""

import os
import re
import types

import pytest
import torch

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


def _wrappers(sv):
    """Every wrapper that allocates, as a call on a given stream (operands of the smallest shapes)."""
    z = torch.zeros
    i32, bf = torch.int32, torch.bfloat16
    logits, rows = z(2, 3, 8), z(6, 8)
    toks, par = z(2, 3, dtype=i32), z(2, 3, dtype=i32)
    lens, table = z(2, dtype=i32), z(2, 4, dtype=i32)
    q = z(2, 3, 4, 64, dtype=bf)
    cache = types.SimpleNamespace(kv_heads=2, head_dim=64)
    hid = z(6, 16, dtype=bf)
    head = z(256, 16, dtype=bf)
    return {
        "verify_chain": lambda s: sv.verify_chain(logits, logits[:, :2], toks[:, :2], z(2, 3), 1.0, stream=s),
        "verify_tree": lambda s: sv.verify_tree(logits, par, toks, stream=s),
        "verify_tree_sample": lambda s: sv.verify_tree_sample(logits, logits, par, toks, z(2, 3), 1.0, stream=s),
        "verify_chain_lmhead": lambda s: sv.verify_chain_lmhead(hid, head, hid[:4], head, toks[:, :2], z(2, 3), 1.0, None, s),
        "probs": lambda s: sv.probs(rows, 1.0, stream=s),
        "sample": lambda s: sv.sample(rows, 1.0, z(6), stream=s),
        "topk": lambda s: sv.topk(rows, 2, stream=s),
        "tree_mask": lambda s: sv.tree_mask(par, s),
        "kv_append": lambda s: sv.kv_append(cache, table, lens, q[:, :, :2], q[:, :, :2], q=q, stream=s),
        "kv_attention": lambda s: sv.kv_attention(cache, table, lens, q, return_lse=True, stream=s),
        "kv_commit": lambda s: sv.kv_commit(cache, table, lens, par, lens, stream=s)}


NAMES = ("verify_chain", "verify_tree", "verify_tree_sample", "verify_chain_lmhead", "probs", "sample", "topk",
         "tree_mask", "kv_append", "kv_attention", "kv_commit")


@pytest.mark.parametrize("name", NAMES)
def test_wrappers_allocate_on_the_stream_of_the_call(monkeypatch, name):
    """A workspace that a wrapper makes and drops, and a status word that it zeroes, belong to the stream of
    the call: made on another one the memory is handed out again while the call still uses it, and the
    zeroing may come after the call's report."""
    from speculative_decoding_verification_78_gb300 import build
    build.build()
    import speculative_decoding_verification_78_gb300 as sv
    from speculative_decoding_verification_78_gb300 import _binding as b
    sv.load_library()
    call = _wrappers(sv)[name]
    given, current, made = object(), [None], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *_):
            current.pop()

    for fn in ("empty", "zeros", "empty_like"):
        def make(*a, _real=getattr(torch, fn), **kw):
            made.append(current[-1])
            return _real(*a, **kw)
        monkeypatch.setattr(torch, fn, make)
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(b, "_torch_stream", lambda s: s, raising=False)
    seen = []
    monkeypatch.setattr(b, "spec_" + name, lambda *a: seen.append(a[-1]) or 0)
    out = call(given)
    assert seen == [given] and isinstance(out, tuple)
    assert made and all(s is given for s in made), made
    del made[:]
    call(None)
    assert made and all(s is None for s in made)
