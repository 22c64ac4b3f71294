"""The KV-cache calls without a GPU: what the library refuses before anything is enqueued, and
what the binding refuses before a pointer reaches the library."""

import ctypes

import pytest
import torch

FAKE = 0x100000   # a 256-byte aligned fake device address: never dereferenced here


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_78_gb300 import build as b
    b.build()
    import speculative_decoding_verification_78_gb300 as sv
    sv.load_library()
    return sv


def _cache(sv, **kw):
    c = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=100, page_size=64, kv_heads=2,
             head_dim=128)
    c.update(kw)
    return sv.SpecKVCache(*(c[f] for f, _ in sv.SpecKVCache._fields_))


def _append(sv, cache=None, **kw):
    c = dict(table=FAKE, pps=4, lens=FAKE, new=None, B=2, N=3, k=FAKE, ks=256, v=FAKE, vs=256,
             q=FAKE, qs=512, qh=4, qo=FAKE + 4096, dtype=1, rope=FAKE, rows=100, dim=64, inter=0,
             pos=None, mask=None, status=FAKE, stream=None)
    c.update(kw)
    return sv.load_library().spec_kv_append(ctypes.byref(cache or _cache(sv)), *c.values())


def _attend(sv, cache=None, **kw):
    c = dict(table=FAKE, pps=4, lens=FAKE, new=None, B=2, N=3, q=FAKE, qs=512, qh=4, dtype=1,
             scale=0.1, mask=None, out=FAKE, lse=None, status=FAKE, ws=FAKE, wsb=1 << 30, stream=None)
    c.update(kw)
    return sv.load_library().spec_kv_attention(ctypes.byref(cache or _cache(sv)), *c.values())


def _commit(sv, cache=None, **kw):
    c = dict(layers=1, table=FAKE, pps=4, lens=FAKE, B=2, N=8, path=FAKE, acc=FAKE, out=FAKE + 256,
             status=FAKE, stream=None)
    c.update(kw)
    return sv.load_library().spec_kv_commit(ctypes.byref(cache or _cache(sv)), *c.values())


@pytest.mark.parametrize("bad", [dict(head_dim=96), dict(page_size=48), dict(page_size=8),
                                 dict(kv_heads=0), dict(kv_heads=1025), dict(num_pages=0),
                                 dict(num_pages=1 << 24)])
def test_cache_shapes(sv, bad):
    for call in (_append, _attend, _commit):
        assert call(sv, _cache(sv, **bad)) == sv.SPEC_ERR_SHAPE


def test_cache_pointers(sv):
    for call in (_append, _attend, _commit):
        for f in ("k", "v", "k_scale", "v_scale"):
            assert call(sv, _cache(sv, **{f: None})) == sv.SPEC_ERR_NULL
            assert call(sv, _cache(sv, **{f: FAKE + 2})) == sv.SPEC_ERR_ALIGN
        assert call(sv, table=None) == sv.SPEC_ERR_NULL
        assert call(sv, lens=None) == sv.SPEC_ERR_NULL
        assert call(sv, status=None) == sv.SPEC_ERR_NULL
        assert call(sv, lens=FAKE + 1) == sv.SPEC_ERR_ALIGN
        assert call(sv, pps=0) == sv.SPEC_ERR_SHAPE
        assert call(sv, pps=1 << 24) == sv.SPEC_ERR_SHAPE
        assert call(sv, B=-1) == sv.SPEC_ERR_SHAPE
        assert call(sv, N=0) == sv.SPEC_ERR_SHAPE
        assert call(sv, B=0) == sv.SPEC_OK


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=0), -4), (dict(dtype=7), -4), (dict(N=(1 << 20) + 1), -2), (dict(ks=255), -2),
    (dict(ks=260), -2), (dict(vs=128), -2), (dict(qs=256), -2), (dict(qh=-1), -2),
    (dict(dim=24), -2), (dict(dim=144), -2), (dict(rows=0), -2), (dict(N=1025, mask=FAKE), -2),
    (dict(k=None), -1), (dict(v=None), -1), (dict(q=None), -1), (dict(qo=None), -1),
    (dict(rope=None), -1), (dict(k=FAKE + 8), -6), (dict(q=FAKE + 8), -6), (dict(pos=FAKE + 2), -6),
    (dict(q=FAKE + 4096, qs=1024), -2)])
def test_append_refusals(sv, bad, code):
    assert _append(sv, **bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=0), -4), (dict(qh=3), -2), (dict(qh=0), -2), (dict(qs=256), -2),
    (dict(scale=float("nan")), -2), (dict(scale=float("inf")), -2), (dict(N=1025, mask=FAKE), -2),
    (dict(q=None), -1), (dict(out=None), -1), (dict(ws=None), -1), (dict(wsb=16), -5),
    (dict(ws=FAKE + 8), -6), (dict(out=FAKE + 2), -6), (dict(lse=FAKE + 2), -6),
    (dict(B=1 << 30, pps=1 << 20), -2)])
def test_attention_refusals(sv, bad, code):
    assert _attend(sv, **bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(layers=0), -2), (dict(N=1025), -2), (dict(path=None), -1), (dict(acc=None), -1),
    (dict(out=None), -1), (dict(out=FAKE), -2), (dict(path=FAKE + 1), -6)])
def test_commit_refusals(sv, bad, code):
    assert _commit(sv, **bad) == code


def test_attention_workspace(sv):
    n = sv.spec_kv_attention_workspace_bytes(4, 6, 32, 8, 128)
    assert n > 0
    # bounded whatever the batch: a few partial results for each SM, and a word for each sequence
    assert sv.spec_kv_attention_workspace_bytes(4096, 64, 64, 8, 128) < 64 << 20
    for bad in ((-1, 6, 32, 8, 128), (4, 0, 32, 8, 128), (4, 6, 30, 8, 128), (4, 6, 32, 0, 128),
                (4, 6, 32, 8, 96), (4, 6, 0, 8, 128)):
        assert sv.spec_kv_attention_workspace_bytes(*bad) == 0


def test_binding_refuses_host_and_misshapen_tensors(sv):
    shape = (10, 2, 64, 128)
    k = torch.empty(shape, dtype=torch.uint8)
    s = torch.ones(10, 2)
    with pytest.raises(ValueError, match="device tensor"):
        sv.KVCache(k, k, s, s)
    with pytest.raises(TypeError):
        sv.KVCache(k.float(), k, s, s)
    with pytest.raises(ValueError):
        sv.KVCache(k, k, s[:5], s)
    with pytest.raises(ValueError):
        sv.KVCache(k[0], k[0], s, s)

    from speculative_decoding_verification_78_gb300 import _binding as b
    x = torch.empty(2, 3, 4, 128, dtype=torch.bfloat16)
    for bad in (x.float(), x[..., :64], x[:, :, :2]):
        with pytest.raises((TypeError, ValueError)):
            b._tokens(bad, "q", 2, 3, 4, 128, torch.bfloat16)
    with pytest.raises(ValueError):
        b._kv_shared(torch.empty(3, 4, dtype=torch.int32), torch.empty(2, dtype=torch.int32), None,
                     None, None, 2, 3)
    with pytest.raises(TypeError):
        b._kv_shared(torch.empty(2, 4, dtype=torch.int64), torch.empty(2, dtype=torch.int32), None,
                     None, None, 2, 3)
