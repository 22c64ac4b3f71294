"""The page and beam calls without a GPU: what the library refuses before anything is enqueued."""

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
    c = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=100, page_size=64, kv_heads=2, head_dim=128)
    c.update(kw)
    return ctypes.byref(sv.SpecKVCache(*(c[f] for f, _ in sv.SpecKVCache._fields_)))


def _call(name, defaults):
    def call(sv, cache=None, **kw):
        assert set(kw) <= set(defaults)
        return getattr(sv.load_library(), name)(cache or _cache(sv), *{**defaults, **kw}.values())
    return call


WS = dict(ws=FAKE, wsb=1 << 20, stream=None)
reserve = _call("spec_kv_reserve", dict(refs=FAKE, table=FAKE, pps=4, lens=FAKE, new=None, B=2, N=3, granted=FAKE,
                                        status=FAKE, **WS))
trim = _call("spec_kv_trim", dict(refs=FAKE, table=FAKE, pps=4, lens=FAKE, B=2, window=10, sinks=4, status=FAKE,
                                  stream=None))
free = _call("spec_kv_free", dict(refs=FAKE, table=FAKE, pps=4, lens=FAKE, ended=None, B=2, status=FAKE, stream=None))
fork = _call("spec_kv_fork", dict(layers=1, refs=FAKE, table=FAKE, pps=4, lens=FAKE, B=2, parents=FAKE, C=3, release=0,
                                  out=FAKE + 4096, lens_out=FAKE + 4096, status=FAKE, **WS))
compact = _call("spec_kv_compact", dict(layers=1, refs=FAKE, table=FAKE, pps=4, B=2, map=FAKE, live=FAKE, status=FAKE,
                                        **WS))
ALL = [reserve, trim, free, fork, compact]


@pytest.mark.parametrize("call", ALL)
def test_common_refusals(sv, call):
    for bad in (dict(head_dim=96), dict(page_size=48), dict(kv_heads=0), dict(num_pages=0), dict(num_pages=1 << 24)):
        assert call(sv, _cache(sv, **bad)) == sv.SPEC_ERR_SHAPE
    for f in ("k", "v", "k_scale", "v_scale"):
        assert call(sv, _cache(sv, **{f: None})) == sv.SPEC_ERR_NULL
    for name in ("refs", "table", "status"):
        assert call(sv, **{name: None}) == sv.SPEC_ERR_NULL
        assert call(sv, **{name: FAKE + 2}) == sv.SPEC_ERR_ALIGN
    assert call(sv, pps=0) == sv.SPEC_ERR_SHAPE
    assert call(sv, B=-1) == sv.SPEC_ERR_SHAPE
    assert call(sv, B=sv.SPEC_MAX_SEQS + 1) == sv.SPEC_ERR_SHAPE
    if call is not compact:
        assert call(sv, lens=None) == sv.SPEC_ERR_NULL


@pytest.mark.parametrize("call,bad,code", [
    (reserve, dict(N=0), -2), (reserve, dict(N=(1 << 20) + 1), -2), (reserve, dict(granted=None), -1),
    (reserve, dict(granted=FAKE + 2), -6), (reserve, dict(new=FAKE + 1), -6), (reserve, dict(ws=None), -1),
    (reserve, dict(ws=FAKE + 8), -6), (reserve, dict(wsb=100), -5),
    (trim, dict(window=0), -2), (trim, dict(window=-1), -2), (trim, dict(sinks=-1), -2),
    (free, dict(ended=FAKE + 2), -6),
    (fork, dict(layers=0), -2), (fork, dict(C=-1), -2), (fork, dict(C=8193), -2), (fork, dict(parents=None), -1),
    (fork, dict(out=None), -1), (fork, dict(lens_out=None), -1), (fork, dict(parents=FAKE + 2), -6),
    (fork, dict(out=FAKE), -2), (fork, dict(out=FAKE + 16), -2), (fork, dict(out=FAKE - 16), -2),
    (fork, dict(lens_out=FAKE + 4), -2), (fork, dict(wsb=100), -5), (fork, dict(ws=None), -1),
    (compact, dict(layers=0), -2), (compact, dict(map=None), -1), (compact, dict(live=None), -1),
    (compact, dict(map=FAKE + 2), -6), (compact, dict(wsb=100), -5)])
def test_refusals(sv, call, bad, code):
    assert call(sv, **bad) == code


def test_empty_calls(sv):
    for call in (reserve, trim, free):
        assert call(sv, B=0, table=None, lens=None) == sv.SPEC_OK
    assert fork(sv, C=0, parents=None, out=None, lens_out=None) == sv.SPEC_OK


def test_workspaces(sv):
    assert sv.spec_kv_pages_workspace_bytes(100, 5) >= 16 + 800
    assert sv.spec_kv_pages_workspace_bytes(1, 8192) >= 20 * 8192
    for bad in ((0, 5), (10, -1), (10, 8193)):
        assert sv.spec_kv_pages_workspace_bytes(*bad) == 0
    assert sv.spec_beam_workspace_bytes(2, 4, 32000, sv.SPEC_F32) >= 2 * 4 * 32 * 8
    for bad in ((-1, 4, 100, 0), (1, 0, 100, 0), (1, 65, 100, 0), (1, 4, 0, 0), (1, 4, (1 << 20) + 1, 0), (1, 4, 100, 2)):
        assert sv.spec_beam_workspace_bytes(*bad) == 0


def _select(sv, **kw):
    c = dict(logits=FAKE, dtype=1, scores=FAKE, done=None, pad=0, B=2, K=4, V=1000, n=8, tokens=FAKE + 64,
             parents=FAKE + 64, out=FAKE + 64, status=FAKE, ws=FAKE, wsb=1 << 20, stream=None)
    c.update(kw)
    return sv.load_library().spec_beam_select(*c.values())


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=2), -4), (dict(B=-1), -2), (dict(K=0), -2), (dict(K=65), -2), (dict(n=0), -2), (dict(n=65), -2),
    (dict(V=0), -2), (dict(V=(1 << 20) + 1), -2), (dict(pad=-1), -2), (dict(pad=1000), -2),
    (dict(B=1 << 24, K=64, V=1 << 20), -2), (dict(logits=None), -1), (dict(scores=None), -1),
    (dict(tokens=None), -1), (dict(parents=None), -1), (dict(out=None), -1), (dict(status=None), -1),
    (dict(ws=None), -1), (dict(logits=FAKE + 1), -6), (dict(dtype=0, logits=FAKE + 2), -6),
    (dict(done=FAKE + 2), -6), (dict(ws=FAKE + 8), -6), (dict(out=FAKE), -2), (dict(wsb=8), -5)])
def test_select_refusals(sv, bad, code):
    assert _select(sv, **bad) == code


def test_select_outputs_over_inputs(sv):
    far = dict(logits=FAKE, scores=FAKE + 4096, done=FAKE + 8192, tokens=FAKE + 12288, parents=FAKE + 16384,
               out=FAKE + 20480, wsb=1)   # (refused for its workspace, after the outputs were found fine)
    assert _select(sv, **far) == sv.SPEC_ERR_WORKSPACE
    for name in ("tokens", "parents", "out"):
        for at in (4096 - 60, 4096, 4096 + 28, 8192 + 4):
            assert _select(sv, **{**far, name: FAKE + at}) == sv.SPEC_ERR_SHAPE
    assert _select(sv, **{**far, "out": FAKE + 4096 + 32}) == sv.SPEC_ERR_WORKSPACE


def test_reorder_refusals(sv):
    lib = sv.load_library()

    def call(states, parents=FAKE, R=4, C=4, status=FAKE, count=None):
        arr = (sv.SpecState * max(1, len(states)))(*states)
        return lib.spec_beam_reorder(arr, len(states) if count is None else count, parents, R, C, status, None)

    a = (FAKE, FAKE + 4096, 64)
    assert call([a], C=0) == sv.SPEC_OK
    assert call([], count=0) == sv.SPEC_ERR_SHAPE
    assert call([a] * 9) == sv.SPEC_ERR_SHAPE
    assert call([(FAKE, FAKE + 4096, 0)]) == sv.SPEC_ERR_SHAPE
    assert call([(FAKE, FAKE + 4096, 1 << 61)]) == sv.SPEC_ERR_SHAPE
    assert call([a], R=-1) == sv.SPEC_ERR_SHAPE
    assert call([a], parents=None) == sv.SPEC_ERR_NULL
    assert call([a], status=None) == sv.SPEC_ERR_NULL
    assert call([a], parents=FAKE + 2) == sv.SPEC_ERR_ALIGN
    assert call([(None, FAKE, 64)]) == sv.SPEC_ERR_NULL
    assert call([(FAKE, None, 64)]) == sv.SPEC_ERR_NULL
    assert call([(FAKE, FAKE + 255, 64)]) == sv.SPEC_ERR_SHAPE                      # over its input
    assert call([a, (FAKE + 8192, FAKE + 64, 64)]) == sv.SPEC_ERR_SHAPE             # over the other's input
    assert call([a, (FAKE + 8192, FAKE + 4096 + 128, 64)]) == sv.SPEC_ERR_SHAPE     # over the other's output


def test_binding_refusals(sv):
    from speculative_decoding_verification_78_gb300 import _binding as b
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError):
        b.spec_beam_select(torch.zeros(3, 4), None, None, 0, 1, None, None, None, None, None)
    with pytest.raises(ValueError, match="device tensor"):
        b.spec_beam_select(torch.zeros(1, 3, 4), None, None, 0, 1, None, None, None, None, None)
    with pytest.raises(ValueError):
        b.spec_beam_reorder([i32(3, 2)], i32(4), [i32(4, 3)], i32(1))
    with pytest.raises(ValueError, match="device tensor"):
        b.spec_beam_reorder([i32(3, 2)], i32(4), [i32(4, 2)], i32(1))
    with pytest.raises(ValueError):
        b.spec_beam_reorder([], i32(4), [], i32(1))
    with pytest.raises(TypeError):
        b.spec_beam_reorder([i32(3, 2)], i32(4).long(), [i32(4, 2)], i32(1))


def test_status_texts(sv):
    assert "free page" in sv.spec_status_string(sv.SPEC_ERR_NO_PAGE)
    assert "given back" in sv.spec_status_string(sv.SPEC_ERR_REFS)


def _window(sv, cache=None, **kw):
    c = dict(table=FAKE, pps=4, lens=FAKE, new=None, B=2, N=3, q=FAKE, qs=512, qh=4, dtype=1, scale=0.1, mask=None,
             window=10, sinks=2, out=FAKE, lse=None, status=FAKE, ws=FAKE, wsb=1 << 30, stream=None)
    c.update(kw)
    return sv.load_library().spec_kv_attention_window(cache or _cache(sv), *c.values())


@pytest.mark.parametrize("bad,code", [
    (dict(window=0), -2), (dict(window=-5), -2), (dict(sinks=-1), -2), (dict(mask=FAKE, window=2), -2),
    (dict(dtype=0), -4), (dict(qh=3), -2), (dict(q=None), -1), (dict(out=None), -1), (dict(ws=None), -1),
    (dict(wsb=16), -5), (dict(N=1025, mask=FAKE, window=2000), -2), (dict(scale=float("nan")), -2)])
def test_window_refusals(sv, bad, code):
    assert _window(sv, **bad) == code


def test_window_of_a_tree_and_empty_batch(sv):
    assert _window(sv, mask=FAKE, window=3, B=0, table=None, lens=None) == sv.SPEC_OK
    with pytest.raises(ValueError, match="window"):
        sv.kv_attention(None, None, None, None, sinks=3)
