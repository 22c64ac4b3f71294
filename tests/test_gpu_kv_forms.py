"""GPU parity of the KV-cache operators in every form of their kernels: the row counts, head dims and types
that choose one, and the paths inside that random data seldom takes."""

import numpy as np
import pytest
import torch

import kv_ref as ref
import test_gpu_kv as kv
from test_gpu_kv import Case, check_attention, f64, rand16, rope_table, tree_words

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_78_gb300 as sv
    sv.load_library()
    return sv


# ------------------------------------------------------------------ scratch on the stream of the call

@pytest.mark.parametrize("raw", [False, True])
def test_scratch_of_a_call_on_another_stream(sv, raw):
    """The workspace that kv_attention makes for itself stays its own until the call has ended, whatever
    the current stream allocates meanwhile; and a reported status is not zeroed afterwards."""
    c = Case(91, [6000, 2500], 1, 2, 128, 64)
    q = rand16(c.rng, (2, 1, 8, 128), torch.bfloat16)
    want, wlse = check_attention(sv, c, q)
    table, lens = c.dev("table", "lens")
    cache = c.cache(sv)
    bad = table.clone()
    bad[0, 1] = -1
    size = sv.spec_kv_attention_workspace_bytes(2, 1, 8, 2, 128)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for pages, code in ((table, 0), (bad, sv.SPEC_ERR_PAGE)):
        with torch.cuda.stream(s):
            torch.cuda._sleep(100_000_000)   # about 50 ms: the call waits behind it
        out, lse, st = sv.kv_attention(cache, pages, lens, q, return_lse=True,
                                       stream=s.cuda_stream if raw else s)
        junk = [torch.full((n,), 0x3f, dtype=torch.uint8, device="cuda")
                for n in (size, size, out.numel() * 2, lse.numel() * 4, 4, 4) for _ in range(2)]
        torch.cuda.synchronize()
        assert int(st.item()) == code
        assert torch.equal(out[1], want[1]) and torch.equal(lse[1], wlse[1])
        if code == 0:
            assert torch.equal(out, want) and torch.equal(lse, wlse)
        assert all(bool((j == 0x3f).all()) for j in junk)
