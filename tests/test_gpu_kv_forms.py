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


# ------------------------------------------------------------------ references that rise

@pytest.mark.parametrize("G", [16, 32])
def test_a_row_whose_reference_rises_leaves_the_others_sums(sv, G):
    """Rows share tiles with one whose scores rise by more than 2^7 a tile, so that every tile is weighed
    twice. What the first time added to the others' sums is taken off again to half a unit of the sum: of
    6 tiles a group at most 3.5 x 2^-24, 2^-21.7 of a base-2 logarithm, which is held in steps of 2^-18 (the
    values' scale is 2^70): at most one row in 13 may show it, and one in 8 is let pass."""
    B, Hkv, D, page, tiles = 19, 8, 64, 64, 12
    n = 128 * tiles
    rng = np.random.default_rng(G)
    k = np.zeros((B, n, Hkv, D), np.float32)
    k[..., 1:] = rng.integers(-8, 9, (B, 1, Hkv, D - 1))   # every token the same but for dim 0
    k[..., 0] = (np.arange(n) // 128)[None, :, None]
    pages = B * n // page

    def pool(x):   # [B, n, Hkv, D] -> pages in order
        x = x.reshape(pages, page, Hkv, D).transpose(0, 2, 1, 3)
        return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(kv.E4)

    v = pool(rng.integers(-8, 9, k.shape).astype(np.float32))
    one = torch.ones(pages, Hkv, device="cuda")
    cache = sv.KVCache(pool(k), v, one, one * 2.0 ** 70)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(B, -1)
    lens = torch.full((B,), n - 1, dtype=torch.int32, device="cuda")
    q = rand16(rng, (B, 1, Hkv * G, D), torch.bfloat16, 0.05)
    q[..., 0] = 0
    lses = []
    for rising in (0.0, 16.0):
        r = q.clone()
        r[:, :, ::G] = 0
        r[:, :, ::G, 0] = rising
        _, lse, st = sv.kv_attention(cache, table, lens, r, scale=1.0, return_lse=True)
        assert int(st.item()) == 0
        lses.append(lse.view(-1, G)[:, 1:])
    assert bool(torch.isfinite(lses[0]).all())
    differ = float((lses[0] != lses[1]).float().mean())
    assert differ <= 1 / 8, differ


def test_an_empty_batch(sv):
    cache = sv.new_kv_cache(4, 2, 64, 16)
    before = cache.k.view(torch.uint8).clone()
    table = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    lens = torch.empty(0, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 3, 8, 64, dtype=torch.bfloat16, device="cuda")
    q, st = sv.kv_append(cache, table, lens, x[:, :, :2], x[:, :, :2], q=x)
    out, lse, st = sv.kv_attention(cache, table, lens, q, return_lse=True, status=st)
    new, st = sv.kv_commit(cache, table, lens, torch.empty(0, 3, dtype=torch.int32, device="cuda"), lens, status=st)
    assert int(st.item()) == 0
    assert (q.shape, out.shape, lse.shape, new.shape) == (x.shape, x.shape, x.shape[:3], lens.shape)
    assert torch.equal(cache.k.view(torch.uint8), before)
