"""What the KV-cache calls take and what they refuse, at the limits: on the host, nothing is launched (a
workspace that is too small ends each accepted call)."""

import pytest
import torch

from test_kv_host import FAKE, _append, _attend, _cache, _commit, sv   # noqa: F401


@pytest.mark.parametrize("N,most", [(1, 255), (16, 255), (17, 255), (32, 255), (33, 255), (128, 255),
                                    (129, 255), (256, 255), (257, 127), (512, 127), (513, 85)])
def test_attention_tiles_in_31_bits(sv, N, most):   # noqa: F811
    """2^22 tiles of 128 slots, 2 key heads, one query head each: row tiles of 16, 32, 128 or 256."""
    cache = _cache(sv, page_size=128)
    call = lambda B: _attend(sv, cache, N=N, B=B, pps=1 << 22, qh=2, qs=256, wsb=16)
    assert call(most) == sv.SPEC_ERR_WORKSPACE
    assert call(most + 1) == sv.SPEC_ERR_SHAPE
    assert call((1 << 31) - 1) == sv.SPEC_ERR_SHAPE


@pytest.mark.parametrize("shape,code", [
    (dict(B=16, N=32768, qh=32, qs=4096, pps=4096), -5),        # 16 prompts of 32768 of up to 262144 tokens
    (dict(B=1, N=1 << 20, qh=32, qs=4096, pps=1 << 14), -5),    # a million tokens in one piece
    (dict(B=1, N=1 << 20, qh=8 * 2047, qs=8 * 2047 * 128, pps=1), -5),
    (dict(B=1, N=1 << 20, qh=8 * 2048, qs=8 * 2048 * 128, pps=1), -2)])
def test_long_prompts_are_taken(sv, shape, code):   # noqa: F811
    assert _attend(sv, _cache(sv, kv_heads=8), wsb=16, **shape) == code


@pytest.mark.parametrize("layers", [None, 3])
@pytest.mark.parametrize("bad", ["v", "k_scale", "v_scale", "v layers", "scale layers", "none"])
def test_cache_of_mixed_layouts(sv, layers, bad):   # noqa: F811
    """Values and scales in another order than the keys have as many elements, but lie elsewhere."""
    lead = () if layers is None else (layers,)
    k = torch.zeros(*lead, 10, 2, 64, 128, dtype=torch.uint8)
    s = torch.ones(*lead, 10, 2)
    swap = lambda t, a, b: t.transpose(a, b).contiguous()
    args = {"v": (k, swap(k, -3, -2), s, s), "k_scale": (k, k, swap(s, -2, -1), s),
            "v_scale": (k, k, s, swap(s, -2, -1)), "v layers": (k, k.flatten(0, 1), s, s),
            "scale layers": (k, k, s, s.flatten()), "none": (k, None, s, s)}[bad]
    with pytest.raises(ValueError, match="beside k"):
        sv.KVCache(*args)
    with pytest.raises(ValueError, match="device tensor"):   # as it should lie
        sv.KVCache(k, k, s, s)


def test_an_empty_batch_has_no_tensors(sv):   # noqa: F811
    """B = 0 does nothing, and torch gives empty tensors no address: only the cache and the status are
    asked for."""
    none = dict(B=0, table=None, lens=None)
    assert _append(sv, k=None, v=None, q=None, qo=None, **none) == sv.SPEC_OK
    assert _attend(sv, q=None, out=None, **none) == sv.SPEC_OK
    assert _commit(sv, path=None, acc=None, out=None, **none) == sv.SPEC_OK
    for call in (_append, _attend, _commit):
        assert call(sv, _cache(sv, k=None), B=0) == sv.SPEC_ERR_NULL
        assert call(sv, B=0, status=None) == sv.SPEC_ERR_NULL
        assert call(sv, B=0, N=0) == sv.SPEC_ERR_SHAPE
        assert call(sv, B=0, lens=FAKE + 1) == sv.SPEC_ERR_ALIGN
    assert _attend(sv, B=0, wsb=16) == sv.SPEC_ERR_WORKSPACE
