"""GPU tests of attention with a sliding window and sinks over the paged cache, against the plain fp64 form.

Tolerances as in test_gpu_kv (the roundings are the same: the output's, the weights' to fp16, the scores')."""

import numpy as np
import pytest
import torch

import kv_ref as ref
from test_gpu_kv import E4, HALF, Case, f64, rand16, tree_words

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_78_gb300 as sv
    sv.load_library()
    return sv


def seen(n0, N, n, window, sinks, bits=None):
    """[N, n0 + n] truth values by the definition; bits [N, N] of a tree."""
    t, i = np.arange(n0 + n)[None], np.arange(N)[:, None]
    depth = i if bits is None else np.maximum(0, bits.sum(1, keepdims=True) - 1)
    new = t - n0 <= i
    if bits is not None:
        new = np.concatenate([np.ones((N, n0), bool), bits[:, :n]], 1)
    return new & ((t < sinks) | (t > n0 + depth - window)) & (i < n)


def forget(c, window, sinks):
    """Table entries of pages behind the window of the first new token are -1, as kv_trim leaves them; the
    slots of other pages that no query sees hold NaN, scales too."""
    used = set()
    for b in range(c.B):
        for j in range(c.table.shape[1]):
            lo, hi = j * c.page, (j + 1) * c.page
            if c.table[b, j] < 0:
                continue
            if lo >= sinks and hi <= int(c.lens[b]) - window + 1:
                c.table[b, j] = -1
            else:
                used.add(int(c.table[b, j]))
                for t in range(lo, hi):
                    if t >= sinks and t <= int(c.lens[b]) - window:
                        for x in c.pool:
                            x[:, c.table[b, j], :, t - lo] = 0x7f
    for p in set(range(c.pool[0].shape[1])) - used:
        for x, s in zip(c.pool, c.scale):
            x[:, p] = 0xff
            s[:, p] = np.nan


def check(sv, c, q, window, sinks, words=None, new_lens=None, **kw):
    cache = c.cache(sv)
    table, lens = c.dev("table", "lens")
    nl = None if new_lens is None else torch.tensor(new_lens, dtype=torch.int32).cuda()
    out, lse, st = sv.kv_attention(cache, table, lens, q, mask=words, new_lens=nl, return_lse=True,
                                   window=window, sinks=sinks, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    scale = c.D ** -0.5
    qd, o, l = f64(q), f64(out), f64(lse)
    for b in range(c.B):
        n = c.N if new_lens is None else new_lens[b]
        n0 = int(c.lens[b])
        see = seen(n0, c.N, n, window, sinks, None if words is None else ref.mask_bits(words[b].cpu().numpy(), c.N))
        some = see.any(0)   # slots that nobody sees may hold anything
        at = np.flatnonzero(some)
        k, v = (ref.E4M3[p[0][c.table[b][at // c.page], :, at % c.page]] *
                s[0][c.table[b][at // c.page]][:, :, None].astype(np.float64) for p, s in zip(c.pool, c.scale))
        want, wl, avg, big, spread = ref.attention(qd[b], k, v, see[:, some], scale)
        d = big * (c.D + 8) * 2.0 ** -24 + spread * 2.0 ** -17 + 2.0 ** -20
        tol = HALF[q.dtype] * np.abs(want) + (2.0 ** -11 + 2 * d[..., None]) * avg + 1e-30
        err = np.abs(o[b] - want)
        assert (err <= tol).all(), (b, float(np.nanmax(err / tol)), np.argwhere(~(err <= tol))[:4])
        fin = np.isfinite(wl)
        assert (np.isneginf(l[b]) == ~fin).all()
        le = np.abs(l[b][fin] - wl[fin])
        lt = d[fin] + 2.0 ** -22 * np.abs(wl[fin]) + 2.0 ** -20
        assert (le <= lt).all(), (b, float((le / lt).max()))
    return out, lse


WINDOWS = [(1, 0), (1, 1), (7, 0), (64, 4), (127, 5), (128, 0), (129, 16), (130, 130), (300, 1), (257, 300),
           (5000, 0), (5000, 7)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("G,Hkv,D,page,dtype", [(4, 2, 128, 64, BF16), (1, 3, 64, 16, F16), (20, 1, 128, 128, BF16)])
def test_one_token(sv, G, Hkv, D, page, dtype, window, sinks):
    lens = [0, 1, 5, 63, 64, 127, 128, 129, 255, 256, 300, 513, 700, 1025]
    c = Case(window + sinks, lens, 1, Hkv, D, page)
    forget(c, window, sinks)
    check(sv, c, rand16(c.rng, (c.B, 1, Hkv * G, D), dtype), window, sinks)


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("N,G,D,page,dtype", [(5, 2, 64, 32, BF16), (6, 4, 128, 16, F16), (17, 5, 128, 64, BF16),
                                              (33, 4, 64, 16, F16), (70, 4, 128, 128, BF16)])
def test_chains(sv, N, G, D, page, dtype, window, sinks):
    lens = [0, 3, 100, 127, 260, 511, 640]
    c = Case(N + window, lens, N, 2, D, page)
    forget(c, window, sinks)
    check(sv, c, rand16(c.rng, (c.B, N, 2 * G, D), dtype), window, sinks)


@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 4), (128, 130), (513, 20), (10000, 1)])
@pytest.mark.parametrize("N,G,D,dtype", [(600, 1, 64, BF16), (333, 4, 128, F16), (1000, 2, 128, BF16)])
def test_pieces_of_prompts(sv, N, G, D, dtype, window, sinks):
    """New tokens past the window of each other; whole tiles that some rows do not see, at both ends."""
    c = Case(N, [0, 77, 300], N, 1, D, 32)
    forget(c, window, sinks)
    check(sv, c, rand16(c.rng, (c.B, N, G, D), dtype), window, sinks, new_lens=[N, N - 70, 1])


@pytest.mark.parametrize("window,sinks", [(64, 0), (64, 3), (130, 64), (129, 200), (4000, 5)])
@pytest.mark.parametrize("N,G,D,page,dtype", [(7, 2, 128, 16, BF16), (13, 2, 64, 64, F16), (30, 4, 128, 64, BF16),
                                              (64, 4, 64, 32, F16), (64, 5, 128, 128, BF16)])
def test_trees(sv, N, G, D, page, dtype, window, sinks):
    lens = [0, 1, 130, 500, 777]
    c = Case(N + sinks, lens, N, 2, D, page)
    words = tree_words(c.rng, c.B, N, sv)
    words[1, N - 1] = 0   # a node that sees no new token, nor itself
    forget(c, window, sinks)
    check(sv, c, rand16(c.rng, (c.B, N, 2 * G, D), dtype), window, sinks, words=words)


def test_empty_sequences(sv):
    """No tokens, padding only, and a masked-out row of an empty sequence: zeros and -inf."""
    c = Case(1, [0, 40, 0, 200], 3, 2, 64, 16)
    words = tree_words(c.rng, 4, 3, sv)
    words[0, 2] = 0
    q = rand16(c.rng, (4, 3, 4, 64), BF16)
    out, lse = check(sv, c, q, 9, 2, words=words)
    assert out[0, 2].eq(0).all() and lse[0, 2].eq(-np.inf).all()
    out, lse = check(sv, c, q, 9, 2, new_lens=[0, 0, 2, 3])
    assert out[:2].eq(0).all() and lse[:2].eq(-np.inf).all()


@pytest.mark.parametrize("N,G,dtype", [(1, 4, BF16), (8, 4, F16), (40, 4, BF16), (200, 2, F16)])
def test_a_window_past_everything_changes_nothing(sv, N, G, dtype):
    c = Case(2, [0, 50, 300, 1000], N, 2, 128, 64)
    cache, (table, lens) = c.cache(sv), c.dev("table", "lens")
    q = rand16(c.rng, (4, N, 2 * G, 128), dtype)
    want = sv.kv_attention(cache, table, lens, q, return_lse=True)
    for window, sinks in ((2000, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 5000)):
        got = sv.kv_attention(cache, table, lens, q, return_lse=True, window=window, sinks=sinks)
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_nan_reaches_those_that_see_it(sv):
    """A NaN key, value or query; and one that has left the window."""
    N, window, sinks = 40, 64, 2
    c = Case(3, [200, 200, 200], N, 2, 128, 64, junk=False)
    for b, (side, t) in enumerate(((0, 150), (1, 170), (1, 1))):
        c.pool[side][0, c.table[b, t // 64], 1, t % 64, 5] = 0x7f
    q = rand16(c.rng, (3, N, 4, 128), BF16)
    q[2, 7, 0, 3] = np.nan
    cache, (table, lens) = c.cache(sv), c.dev("table", "lens")
    out, lse, st = sv.kv_attention(cache, table, lens, q, window=window, sinks=sinks, return_lse=True)
    nan = out.isnan().any(-1).cpu().numpy()   # [B, N, heads]
    want = np.zeros_like(nan)
    for b, t in enumerate((150, 170, 1)):
        want[b, :, 2:] = np.array([t < sinks or t > 200 + i - window for i in range(N)])[:, None]
    want[2, 7, 0] = True
    np.testing.assert_array_equal(nan, want)
    assert int(st.item()) == 0


def test_bad_pages(sv):
    """A page number past the pool, in the window and behind it."""
    c = Case(4, [300, 300], 2, 1, 64, 16, junk=False)
    c.table[0, 2] = 9999    # slots 32 .. 47: behind the window, not a sink
    c.table[1, 17] = 9999   # slots 272 .. 287: seen
    cache, (table, lens) = c.cache(sv), c.dev("table", "lens")
    q = rand16(c.rng, (2, 2, 4, 64), BF16)
    out, _, st = sv.kv_attention(cache, table[:1].contiguous(), lens[:1], q[:1].contiguous(), window=100, sinks=4)
    assert int(st.item()) == 0 and not out.isnan().any()
    out, _, st = sv.kv_attention(cache, table, lens, q, window=100, sinks=4)
    assert int(st.item()) == sv.SPEC_ERR_PAGE and not out[0].isnan().any() and out[1].isnan().all()
    lens[0] = -3
    out, _, st = sv.kv_attention(cache, table, lens, q, window=10, sinks=4)
    assert int(st.item()) == sv.SPEC_ERR_LENGTH and out[0].isnan().all() and not out[1].isnan().any()


def test_in_a_graph_with_other_lengths(sv):
    c = Case(5, [700, 20, 300], 4, 2, 128, 64, junk=False)
    cache, (table, lens) = c.cache(sv), c.dev("table", "lens")
    q = rand16(c.rng, (3, 4, 8, 128), BF16)
    ws = sv.new_attention_workspace(3, 4, 8, 2, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = sv.kv_attention(cache, table, lens, q, window=200, sinks=3, workspace=ws, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _, st = sv.kv_attention(cache, table, lens, q, window=200, sinks=3, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0])
    for new in ([3, 600, 700], [0, 0, 5], [500, 512, 130]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        want = sv.kv_attention(cache, table, lens, q, window=200, sinks=3)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and int(st.item()) == 0


def test_far_slots(sv):
    """A window at the end of a long sequence of which only the sinks' and the window's pages exist."""
    page, n = 128, 1 << 22
    c = Case(6, [10], 3, 1, 64, page, junk=False)
    table = np.full((1, n // page + 2), -1, np.int32)
    keep = [0] + list(range((n - 500) // page, n // page + 1))
    pages = len(keep) + 1
    c.pool = [c.codes((1, pages, 1, page, 64)) for _ in range(2)]
    c.scale = [np.full((1, pages, 1), 2.0 ** -6, np.float32) for _ in range(2)]
    for p, j in enumerate(keep):
        table[0, j] = p
    c.table, c.lens = table, np.array([n], np.int32)
    q = rand16(c.rng, (1, 3, 4, 64), BF16)
    cache, (d_table, lens) = c.cache(sv), c.dev("table", "lens")
    out, lse, st = sv.kv_attention(cache, d_table, lens, q, window=490, sinks=5, return_lse=True)
    assert int(st.item()) == 0
    slots = np.array(list(range(5)) + list(range(n - 489, n + 3)))
    k, v = (ref.E4M3[p[0][table[0][slots // page], :, slots % page]] * 2.0 ** -6 for p in c.pool)
    pos = n + np.arange(3)[:, None]
    see = (slots[None] < 5) | ((slots[None] > pos - 490) & (slots[None] <= pos))
    want, wl, avg, big, spread = ref.attention(f64(q)[0], k, v, see, 64 ** -0.5)
    d = big * 72 * 2.0 ** -24 + spread * 2.0 ** -17 + 2.0 ** -20
    tol = HALF[BF16] * np.abs(want) + (2.0 ** -11 + 2 * d[..., None]) * avg
    assert (np.abs(f64(out)[0] - want) <= tol).all()


def test_trim_leaves_what_attention_reads(sv):
    """kv_trim and then windowed attention: the same bits as before the pages went."""
    c = Case(7, [500, 129, 64, 1000], 1, 2, 64, 16, junk=False)
    cache, (table, lens) = c.cache(sv), c.dev("table", "lens")
    q = rand16(c.rng, (4, 1, 4, 64), BF16)
    refs = sv.new_page_refs(cache)
    refs[table.flatten().long()] = 1
    lens += 1   # the new token is in the cache
    want = sv.kv_attention(cache, table, lens - 1, q, window=100, sinks=20, return_lse=True)
    before = int((refs > 0).sum())
    _, st = sv.kv_trim(cache, refs, table, lens - 1, window=100, sinks=20)
    sv.kv_reserve(cache, refs, table, lens - 1, 1)   # (the slot of the new token itself, where it began a page)
    assert int(st.item()) == 0 and int((refs > 0).sum()) < before - 80
    out, lse, st = sv.kv_attention(cache, table, lens - 1, q, window=100, sinks=20, return_lse=True)
    sel = torch.tensor([0, 1, 3], device="cuda")   # (sequence 2's token began a page, which is another one now)
    assert torch.equal(out[sel], want[0][sel]) and torch.equal(lse[sel], want[1][sel])
